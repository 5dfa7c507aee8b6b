"""The gated delta rule over prompts, its gradients and its single-token form
against float64, token by token: lengths around a chunk, odd heads, strides,
carried states, sequences that end early or are empty."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import causal_conv_backward_gb300 as m  # noqa: E402
import delta_reference as ref  # noqa: E402
from ssm_reference import check, to64  # noqa: E402

BF16, FP16, F32 = torch.bfloat16, torch.float16, torch.float32
NAN = float("nan")


@pytest.fixture(scope="module", autouse=True)
def cuda_ready():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from causal_conv_backward_gb300 import build
    build.build()


def rand(*shape, dtype=BF16, scale=1.0, seed=0, add=0.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (add + scale * torch.randn(shape, generator=g, device="cuda")).to(dtype)


def lens(lengths):
    return None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")


def inputs(S, B, H, G, K, V, dtype=BF16, what="dbsf", layout="dense", lengths=None):
    """Tensors by name, and the same with nothing behind the lengths (which the
    library does not read: NaN there). `what`: d decay, b its bias, s a state,
    f gradient of the final state."""
    t = dict(q=rand(S, B, G, K, dtype=dtype, seed=1, add=0.3), k=rand(S, B, G, K, dtype=dtype, seed=2, add=0.3),
             v=rand(S, B, H, V, dtype=dtype, seed=3), delta=rand(S, B, H, dtype=dtype, seed=4) if "d" in what else None,
             beta=rand(S, B, H, dtype=dtype, seed=5), A=-torch.exp(rand(H, dtype=F32, seed=6)) if "d" in what else None,
             delta_bias=rand(H, dtype=F32, seed=7, add=-2.0) if "b" in what else None,
             state=rand(B, H, V, K, dtype=F32, seed=8, scale=0.3) if "s" in what else None)
    gy, gf = rand(S, B, H, V, dtype=dtype, seed=9), rand(B, H, V, K, dtype=F32, seed=10, scale=0.3) if "f" in what else None
    clean = dict(t)
    if lengths is not None:
        for name in ("q", "k", "v", "delta", "beta"):
            if t[name] is not None:
                t[name] = t[name].clone()
                for b, n in enumerate(lengths):
                    t[name][max(0, n):, b] = NAN
    if layout == "joined":      # q, k, v side by side in one projection's rows, delta and beta in another's
        row = torch.cat([t[n].flatten(2) for n in ("q", "k", "v")], 2)
        t["q"], t["k"], t["v"] = (row[..., :G * K].view(S, B, G, K), row[..., G * K:2 * G * K].view(S, B, G, K),
                                  row[..., 2 * G * K:].view(S, B, H, V))
    elif layout == "odd":
        for n in ("q", "k", "v", "delta", "beta"):
            if t[n] is not None:
                wide = torch.full((*t[n].shape[:-1], t[n].shape[-1] + 3), NAN, dtype=dtype, device="cuda")
                wide[..., 1:-2] = t[n]
                t[n] = wide[..., 1:-2]
        wide = torch.full((*gy.shape[:-1], V + 1), NAN, dtype=dtype, device="cuda")
        wide[..., 1:] = gy
        gy = wide[..., 1:]
    elif layout == "batch":     # [B,S,...] in memory
        for n in ("q", "k", "v", "delta", "beta"):
            if t[n] is not None:
                t[n] = t[n].transpose(0, 1).contiguous().transpose(0, 1)
        gy = gy.transpose(0, 1).contiguous().transpose(0, 1)
    return t, clean, gy, gf


FORMS = dict(delta_softplus=True, beta_sigmoid=True, qk_norm=True)


def reference(clean, lengths, forms=FORMS, scale=None):
    d = {k: to64(v, grad=True) for k, v in clean.items()}
    y, final = ref.delta_rule(d["q"], d["k"], d["v"], d["delta"], d["beta"], d["A"], d["delta_bias"], forms["delta_softplus"],
                              forms["beta_sigmoid"], forms["qk_norm"], scale, lengths, d["state"])
    return d, y, final


def run(S, B, H, G, K, V, dtype=BF16, what="dbsf", layout="dense", lengths=None, forms=FORMS, scale=None):
    t, clean, gy, gf = inputs(S, B, H, G, K, V, dtype, what, layout, lengths)
    leaves, ry, rf = reference(clean, lengths, forms, scale)
    args = [t[k] for k in ("q", "k", "v", "delta", "beta", "A", "delta_bias")]
    kw = dict(forms, lengths=lens(lengths), state=t["state"], scale=scale)
    y, final = m.gated_delta(*args, return_state=True, **kw)
    # sums over K, and over the tokens of a chunk and what its products pass on
    terms = K + 256
    check(y, ry, terms, "y")
    check(final, rf, terms, "final state")
    assert torch.equal(m.gated_delta(*args, **kw), y)
    got = m.gated_delta_backward(gy, *args, grad_final_state=gf, **kw)
    loss = (ry * to64(gy)).sum() + ((rf * to64(gf)).sum() if gf is not None else 0)
    names = [k for k in got._fields if clean[k] is not None]
    for k, want in zip(names, torch.autograd.grad(loss, [leaves[k] for k in names], allow_unused=True)):
        per = {"q": V * H // G + 256, "k": V * H // G + 256, "delta": K * V, "beta": V + 256, "A": S * B * 64, "delta_bias": S * B * 64}.get(k, K + 256)
        check(getattr(got, k), want if want is not None else torch.zeros_like(leaves[k]), per, k)
    for k in got._fields:
        assert (getattr(got, k) is None) == (clean[k] is None)
    if lengths is not None:
        for b, n in enumerate(lengths):
            assert not y[max(0, n):, b].any()
            for k in ("q", "k", "v", "delta", "beta"):
                g = getattr(got, k)
                assert g is None or not g[max(0, n):, b].any(), k


# lengths around one, a group and a chunk of tokens
@pytest.mark.parametrize("S", [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 200])
@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_lengths_of_the_prompt(S, dtype):
    run(S, 2, 2, 1, 32, 16, dtype)


# keys and values on both sides of the kernels' widths, shared heads
@pytest.mark.parametrize("K,V", [(1, 1), (3, 5), (16, 130), (33, 64), (64, 64), (65, 16), (96, 40), (100, 63), (127, 65), (128, 128), (128, 200), (64, 257)])
@pytest.mark.parametrize("H,G", [(3, 3), (4, 1)])
def test_heads(K, V, H, G):
    run(70, 1, H, G, K, V)


@pytest.mark.parametrize("what", ["", "d", "db", "s", "f", "dsf"])
@pytest.mark.parametrize("S", [9, 130])
def test_what_is_given(what, S):
    run(S, 2, 4, 2, 24, 24, what=what)


@pytest.mark.parametrize("softplus", [True, False])
@pytest.mark.parametrize("sigmoid", [True, False])
@pytest.mark.parametrize("norm", [True, False])
def test_forms(softplus, sigmoid, norm):
    S, B, H, G, K, V = 80, 1, 2, 2, 16, 16
    forms = dict(delta_softplus=softplus, beta_sigmoid=sigmoid, qk_norm=norm)
    t, clean, gy, gf = inputs(S, B, H, G, K, V)
    for d in (t, clean):
        if not softplus:
            d["delta"], d["delta_bias"] = d["delta"].abs(), d["delta_bias"].abs()
        if not sigmoid:
            d["beta"] = (d["beta"] * 0.1).abs()
        if not norm:                        # lengths near one, so that the states stay bounded
            d["q"], d["k"] = d["q"] * 0.2, d["k"] * 0.2
    leaves, ry, rf = reference(clean, None, forms, 0.7)
    args = [t[k] for k in ("q", "k", "v", "delta", "beta", "A", "delta_bias")]
    kw = dict(forms, scale=0.7, state=t["state"])
    y, final = m.gated_delta(*args, return_state=True, **kw)
    check(y, ry, K + 256, "y")
    check(final, rf, K + 256, "final state")
    got = m.gated_delta_backward(gy, *args, grad_final_state=gf, **kw)
    loss = (ry * to64(gy)).sum() + (rf * to64(gf)).sum()
    for k, want in zip(got._fields, torch.autograd.grad(loss, [leaves[k] for k in got._fields])):
        check(getattr(got, k), want, S * 64, k)


@pytest.mark.parametrize("layout", ["joined", "odd", "batch"])
@pytest.mark.parametrize("lengths", [None, [70, 0, 33]])
def test_layouts(layout, lengths):
    run(70, 3, 4, 2, 64, 64, layout=layout, lengths=lengths)


@pytest.mark.parametrize("S,lengths", [(1, [0, 1]), (64, [64, 63]), (130, [130, 65, 64, 1, 0]), (200, [-3, 500, 128, 129])])
@pytest.mark.parametrize("K,V", [(40, 24), (128, 128)])
def test_sequences_that_end_early(S, lengths, K, V):
    run(S, len(lengths), 2, 1, K, V, lengths=lengths)


def test_prompt_in_two_parts_is_the_prompt():
    S, B, H, G, K, V = 150, 2, 2, 2, 64, 32
    t, _, _, _ = inputs(S, B, H, G, K, V, what="dbs")
    toks, rest = ("q", "k", "v", "delta", "beta"), ("A", "delta_bias")
    whole, final = m.gated_delta(*[t[k] for k in toks + rest], state=t["state"], return_state=True, **FORMS)
    for cut in (1, 64, 77, 149):
        a, s = m.gated_delta(*[t[k][:cut] for k in toks], *[t[k] for k in rest], state=t["state"], return_state=True, **FORMS)
        b, s = m.gated_delta(*[t[k][cut:] for k in toks], *[t[k] for k in rest], state=s, return_state=True, **FORMS)
        both = torch.cat([a, b])
        check(both, whole.double(), 2 * K + 256, "y")
        check(s, final.double(), 2 * K + 256, "state")


# ------------------------------------------------------------------ single tokens
@pytest.mark.parametrize("K,V", [(1, 1), (32, 16), (33, 20), (64, 64), (100, 70), (128, 128), (128, 300)])
@pytest.mark.parametrize("slots", [None, [4, -1, 0], [7, 2, 5]])
@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_step(K, V, slots, dtype):
    B, H, G, rows = 3, 4, 2, 6
    t, _, _, _ = inputs(1, B, H, G, K, V, dtype, "db")
    cache = rand(rows, H, V, K, dtype=F32, seed=11, scale=0.3)
    before = cache.clone()
    one = {k: v[0] for k, v in t.items() if k in ("q", "k", "v", "delta", "beta")}
    y = m.gated_delta_step(*one.values(), cache, t["A"], t["delta_bias"], slots=lens(slots), **FORMS)
    at = list(range(B)) if slots is None else slots
    touched = [r for r in at if 0 <= r < rows]
    for b, r in enumerate(at):
        if not 0 <= r < rows:
            assert not y[b].any()
            continue
        d = {k: to64(v) for k, v in one.items()}
        ry, rf = ref.delta_rule(*[d[k][None, b:b + 1] for k in ("q", "k", "v", "delta", "beta")], to64(t["A"]), to64(t["delta_bias"]),
                                state=to64(before[r:r + 1]))
        check(y[b], ry[0, 0], K, "y")
        check(cache[r], rf[0], K, "state")
    for r in range(rows):
        if r not in touched:
            assert torch.equal(cache[r], before[r])


def test_steps_continue_a_prompt():
    """A prompt and then single tokens, with layouts of a running program."""
    S, B, H, G, K, V, new = 70, 3, 4, 2, 128, 64, 5
    t, clean, _, _ = inputs(S + new, B, H, G, K, V, what="db")
    lengths = [S, 11, 0]
    _, ry, rf = reference(clean, [n + new for n in lengths])
    toks = ("q", "k", "v", "delta", "beta")
    _, state = m.gated_delta(*[t[k][:S] for k in toks], t["A"], t["delta_bias"], lengths=lens(lengths), return_state=True, **FORMS)
    rows = torch.arange(B, device="cuda")
    for i in range(new):
        at = lens(lengths).long() + i
        y = m.gated_delta_step(*[t[k][at, rows] for k in toks], state, t["A"], t["delta_bias"], **FORMS)
        check(y, torch.stack([ry[n + i, b] for b, n in enumerate(lengths)]), K + 256, "y")
    check(state, rf, K + 256, "state")


def test_step_without_decay_and_by_strides():
    B, H, G, K, V = 3, 2, 1, 48, 40
    t, _, _, _ = inputs(1, B, H, G, K, V, what="", layout="odd")
    state = rand(B, H, V, K, dtype=F32, seed=11)
    d = {k: to64(t[k]) for k in ("q", "k", "v", "beta")}
    ry, rf = ref.delta_rule(d["q"], d["k"], d["v"], None, d["beta"], state=to64(state))
    y = m.gated_delta_step(t["q"][0], t["k"][0], t["v"][0], None, t["beta"][0], state, **FORMS)
    check(y, ry[0], K, "y")
    check(state, rf, K, "state")


# ------------------------------------------------------------------ in a program
def test_same_bits_every_time_and_in_a_graph():
    t, _, gy, gf = inputs(300, 2, 4, 2, 128, 128)
    args = [t[k] for k in ("q", "k", "v", "delta", "beta", "A", "delta_bias")]
    kw = dict(FORMS, state=t["state"], lengths=lens([300, 131]))

    def both():
        return (*m.gated_delta(*args, return_state=True, **kw), *m.gated_delta_backward(gy, *args, grad_final_state=gf, **kw))

    first = both()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        again = both()
    for _ in range(2):
        for x in again:
            x.fill_(NAN)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_a_step_in_a_graph_moves_the_cache_on():
    t, _, _, _ = inputs(1, 4, 4, 2, 128, 128, what="db")
    one = [t[k][0] for k in ("q", "k", "v", "delta", "beta")]
    cache = rand(4, 4, 128, 128, dtype=F32, seed=11, scale=0.3)
    want, start = cache.clone(), cache.clone()
    ys = [m.gated_delta_step(*one, want, t["A"], t["delta_bias"], **FORMS) for _ in range(3)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = m.gated_delta_step(*one, cache, t["A"], t["delta_bias"], **FORMS)
    cache.copy_(start)
    for i in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, ys[i])
    assert torch.equal(cache, want)


@pytest.mark.parametrize("A,delta", [(-1.0, 30.0), (-16.0, 300.0), (-1e-4, -30.0), (0.0, 1.0)])
def test_decays_at_both_ends(A, delta):
    """States that are gone after a token, and states that never fade."""
    S, B, H, G, K, V = 150, 1, 2, 1, 32, 32
    t, clean, gy, gf = inputs(S, B, H, G, K, V, what="dsf")
    for d in (t, clean):
        d["A"] = torch.full((H,), A, device="cuda")
        d["delta"] = (rand(S, B, H, seed=4) * 0.1 + delta).to(BF16)
    leaves, ry, rf = reference(clean, None)
    args = [t[k] for k in ("q", "k", "v", "delta", "beta", "A", "delta_bias")]
    y, final = m.gated_delta(*args, state=t["state"], return_state=True, **FORMS)
    check(y, ry, K + 256, "y")
    check(final, rf, K + 256, "final state")
    got = m.gated_delta_backward(gy, *args, state=t["state"], grad_final_state=gf, **FORMS)
    names = ("q", "k", "v", "beta", "state")
    loss = (ry * to64(gy)).sum() + (rf * to64(gf)).sum()
    for k, want in zip(names, torch.autograd.grad(loss, [leaves[k] for k in names])):
        check(getattr(got, k), want, K + 256, k)


def test_repeated_keys():
    """The same key again and again, b near one: each token overwrites the one before."""
    S, B, H, G, K, V = 130, 1, 2, 1, 64, 32
    t, clean, gy, gf = inputs(S, B, H, G, K, V)
    for d in (t, clean):
        d["k"] = d["k"][:1].expand(S, B, G, K)
        d["beta"] = torch.full((S, B, H), 6.0, dtype=BF16, device="cuda")
    leaves, ry, rf = reference(clean, None)
    args = [t[k] for k in ("q", "k", "v", "delta", "beta", "A", "delta_bias")]
    y, final = m.gated_delta(*args, state=t["state"], return_state=True, **FORMS)
    check(y, ry, K + 256, "y")
    check(final, rf, K + 256, "final state")
    got = m.gated_delta_backward(gy, *args, state=t["state"], grad_final_state=gf, **FORMS)
    loss = (ry * to64(gy)).sum() + (rf * to64(gf)).sum()
    for k, want in zip(got._fields, torch.autograd.grad(loss, [leaves[k] for k in got._fields])):
        check(getattr(got, k), want, S * 64, k)


@pytest.mark.parametrize("S", [1, 17, 64, 100, 300])
@pytest.mark.parametrize("K,V", [(64, 64), (128, 72)])
def test_pairs_behind_a_token_cancel(S, K, V):
    """The first token's decay multiplies an empty state: its gradient is a sum
    of terms that cancel, all of the first chunk's pairs (t, i) in t's row less
    those in i's column. The kernel adds them up as integers for each of 16 warps
    and joins four warps' rows of two kinds and four columns per token, each
    rounded by less than 2^-16 of a unit, and a unit is 2^-24 of the largest pair
    at most: 64 * 12 * 2^-40 < 2^-30 of the largest pair is left."""
    B, H, G = 2, 4, 2
    t, _, gy, _ = inputs(S, B, H, G, K, V, what="db")
    g = m.gated_delta_backward(gy, **t, **FORMS)
    heads = lambda x: to64(x).repeat_interleave(H // G, 2)
    q, k = (x / (x.pow(2).sum(-1, keepdim=True) + 1e-6).sqrt() for x in (heads(t["q"]), heads(t["k"])))
    q, v, gy, b = q * K ** -0.5, to64(t["v"]), to64(gy), to64(t["beta"]).sigmoid()
    log_a = to64(t["A"]) * torch.nn.functional.softplus(to64(t["delta"]) + to64(t["delta_bias"]))
    a = log_a.exp()[..., None, None]
    state, u = torch.zeros(B, H, V, K, dtype=torch.float64, device=q.device), []
    for i in range(S):
        state = a[i] * state
        u.append(b[i, ..., None] * (v[i] - torch.einsum("bhvk,bhk->bhv", state, k[i])))
        state = state + torch.einsum("bhv,bhk->bhvk", u[i], k[i])
    u, grad, du = torch.stack(u), torch.zeros_like(state), [None] * S
    for i in reversed(range(S)):
        grad = grad + torch.einsum("bhv,bhk->bhvk", gy[i], q[i])
        du[i] = torch.einsum("bhvk,bhk->bhv", grad, k[i])
        grad = a[i] * (grad - torch.einsum("bhv,bhk->bhvk", b[i, ..., None] * du[i], k[i]))
    n = min(S, 64)
    c = log_a[:n].cumsum(0)
    decay = torch.exp(c[:, None] - c[None]) * torch.ones(n, n, device=q.device).tril(-1)[..., None, None]
    dots = lambda x, y: torch.einsum("tbhd,ibhd->tibh", x[:n], y[:n])
    pairs = torch.maximum((dots(gy, u) * dots(q, k)).abs(), (b[:n, None] * dots(torch.stack(du), u) * dots(k, k)).abs())
    most = torch.nan_to_num(pairs * decay, nan=0.0).amax((0, 1))
    assert (to64(g.delta[0]).abs() <= 2.0 ** -30 * 1.01 * most * to64(t["A"]).abs()).all()
    assert S == 1 or g.delta[1:].count_nonzero() > 0
