"""The short convolution and the selective scan on the GPU against their
definitions in 64 bits: sizes around tiles, chunks and vectors, lengths from
zero up, strides, groups, carried states, gradients (by the formula and by
differences), caches, streams, refusals. Every buffer the binding allocates
sits between guard regions and starts out as NaN."""
import ctypes

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import causal_conv_backward_gb300 as m  # noqa: E402
import ssm_reference as ref  # noqa: E402
from causal_conv_backward_gb300 import _ssm  # noqa: E402
from parity import check_guards, guarded_full  # noqa: E402

BF16, FP16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def cuda_ready():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from causal_conv_backward_gb300 import build
    build.build()


@pytest.fixture(autouse=True)
def guards(monkeypatch):
    """Outputs and workspaces come from guarded buffers full of NaN patterns."""
    made = []

    class Guarded:
        def __getattr__(self, name):
            return getattr(torch, name)

        @staticmethod
        def empty(shape, dtype=None, device=None):
            shape = (shape,) if isinstance(shape, int) else shape
            made.append(guarded_full(shape, dtype, 0xFF, device))
            return made[-1]

    _ssm._load()
    monkeypatch.setattr(_ssm, "_torch", Guarded())
    yield
    torch.cuda.synchronize()
    check_guards(*made)


def rand(*shape, dtype=BF16, scale=1.0, seed=0):
    g = torch.Generator().manual_seed(seed + 7919 * sum(shape))
    return (scale * torch.randn(shape, generator=g)).to(dtype).cuda()


def as_strided(t, layout):
    """The same values in another memory order."""
    if layout == "dense":
        return t
    if layout == "slice":       # part of a wider tensor, rows 16-byte aligned
        wide = torch.full((*t.shape[:-1], t.shape[-1] + 24), float("nan"), dtype=t.dtype, device=t.device)
        wide[..., 16:16 + t.shape[-1]] = t
        return wide[..., 16:16 + t.shape[-1]]
    if layout == "odd":         # rows on odd elements
        wide = torch.full((*t.shape[:-1], t.shape[-1] + 3), float("nan"), dtype=t.dtype, device=t.device)
        wide[..., 1:1 + t.shape[-1]] = t
        return wide[..., 1:1 + t.shape[-1]]
    assert layout == "batch first"
    return t.transpose(0, 1).contiguous().transpose(0, 1)


def lens(values):
    return None if values is None else torch.tensor(values, dtype=torch.int32, device="cuda")


def poison(t, lengths):
    """NaN past every sequence's end."""
    if lengths is not None:
        S = t.shape[0]
        for b, n in enumerate(lengths.tolist()):
            t[max(0, min(S, n)):, b] = float("nan")
    return t


# ------------------------------------------------------------------ short convolution
CONV = [  # S, B, H, W, dtype, lengths, state, bias, silu, layout
    (1, 1, 1, 1, BF16, None, False, False, True, "dense"),
    (1, 3, 8, 4, FP16, None, True, True, True, "dense"),
    (2, 2, 64, 8, BF16, None, True, True, True, "slice"),
    (7, 2, 130, 3, BF16, [7, 0], True, True, False, "dense"),
    (8, 1, 384, 4, FP16, None, False, True, True, "batch first"),
    (33, 3, 132, 4, BF16, [1, 33, 2], True, True, True, "slice"),
    (40, 2, 67, 5, FP16, [40, 99], False, False, True, "odd"),
    (64, 2, 96, 2, BF16, [-5, 63], True, True, True, "dense"),
    (65, 1, 100, 6, BF16, None, True, True, True, "batch first"),
    (129, 2, 72, 7, FP16, [128, 3], True, False, False, "odd"),
    (600, 1, 40, 4, BF16, [513], True, True, True, "slice"),
    (700, 2, 512, 8, BF16, None, False, True, True, "dense"),
]


@pytest.mark.parametrize("S,B,H,W,dtype,lengths,state,bias,silu,layout", CONV)
def test_short_conv(S, B, H, W, dtype, lengths, state, bias, silu, layout):
    ln = lens(lengths)
    x0 = rand(S, B, H, dtype=dtype, seed=1)
    x = poison(as_strided(x0, layout).clone() if layout == "dense" else as_strided(x0, layout), ln)
    w, b = rand(W, H, dtype=dtype, scale=W ** -0.5, seed=2), rand(H, dtype=dtype, seed=3) if bias else None
    s0 = rand(B, W - 1, H, dtype=dtype, seed=4) if state else None
    act = "silu" if silu else None
    y, final = m.short_conv(x, w, b, activation=act, lengths=ln, state=s0, return_state=True)
    leaves = [ref.to64(t, grad=True) for t in (x0, w, b, s0)]
    ry, rf = ref.conv(leaves[0], leaves[1], leaves[2], silu, lengths, leaves[3])
    ref.check(y, ry, W, "y")
    assert torch.equal(final.cpu().double(), rf.detach())           # rows are copied
    again = m.short_conv(x, w, b, activation=act, lengths=ln, state=s0)
    assert torch.equal(again, y)

    gy = poison(rand(S, B, H, dtype=dtype, seed=5), ln)
    gf = rand(B, W - 1, H, dtype=dtype, seed=6)
    got = m.short_conv_backward(gy, x, w, b, activation=act, lengths=ln, state=s0, grad_final_state=gf)
    gy64 = ref.to64(torch.nan_to_num(gy, nan=0.0))
    loss = (ry * gy64).sum() + (rf * ref.to64(gf)).sum()
    want = torch.autograd.grad(loss, [t for t in leaves if t is not None], allow_unused=True)
    want = iter([v if v is not None else torch.zeros_like(t) for v, t in zip(want, [t for t in leaves if t is not None])])
    for name, leaf, g in zip(("x", "weight", "bias", "state"), leaves, (got.x, got.weight, got.bias, got.state)):
        if leaf is None:
            assert g is None
            continue
        ref.check(g, next(want), W if name in ("x", "state") else S * B, name)


@pytest.mark.parametrize("which", [0, 1, 2, 3])
def test_short_conv_gradient_by_differences(which):
    S, B, H, W = 37, 2, 24, 4
    t = [rand(S, B, H, seed=1), rand(W, H, scale=0.5, seed=2), rand(H, seed=3), rand(B, W - 1, H, seed=4)]
    ln, gy, gf = lens([37, 20]), rand(S, B, H, seed=5), rand(B, W - 1, H, seed=6)
    got = m.short_conv_backward(gy, t[0], t[1], t[2], lengths=ln, state=t[3], grad_final_state=gf)
    leaves = [ref.to64(v) for v in t]

    def loss():
        y, f = ref.conv(leaves[0], leaves[1], leaves[2], True, [37, 20], leaves[3])
        return (y * ref.to64(gy)).sum() + (f * ref.to64(gf)).sum()

    by_diff, by_grad, scale = ref.differences(loss, leaves[which], (got.x, got.weight, got.bias, got.state)[which])
    # each gradient value is off by at most u of itself; the difference by eps^2 of third derivatives
    assert abs(by_diff - by_grad) <= 2.0 ** -8 * scale + 1e-5 * (1 + abs(by_diff))


@pytest.mark.parametrize("B,H,W,dtype,rows,slots,layout", [
    (1, 1, 1, BF16, 1, None, "dense"), (1, 8, 4, FP16, 1, None, "dense"), (3, 64, 2, BF16, 7, [6, 0, 3], "slice"),
    (5, 130, 4, BF16, 6, [5, -1, 0, 6, 2], "odd"), (4, 96, 8, FP16, 4, [3, 2, 1, 0], "dense"), (2, 2048, 3, BF16, 5, None, "dense"),
])
def test_short_conv_step(B, H, W, dtype, rows, slots, layout):
    x, w, b = rand(B, H, dtype=dtype, seed=1), rand(W, H, dtype=dtype, scale=0.5, seed=2), rand(H, dtype=dtype, seed=3)
    cache = rand(rows, W - 1, H, dtype=dtype, seed=4)
    before = cache.clone()
    y = m.short_conv_step(as_strided(x, layout), cache, w, b, slots=lens(slots))
    for i in range(B):
        r = i if slots is None else slots[i]
        if not 0 <= r < rows:
            assert not y[i].any()
            continue
        ry, rf = ref.conv(ref.to64(x[i])[None, None], ref.to64(w), ref.to64(b), True, None, ref.to64(before[r:r + 1]))
        ref.check(y[i], ry[0, 0], W, "y")
        assert torch.equal(cache[r].cpu().double(), rf[0])
        before[r] = cache[r]
    assert torch.equal(before, cache)       # no other row moved


# ------------------------------------------------------------------ selective scan
def scan_inputs(S, B, H, N, G, dtype, opts, layout, lengths, seed=0):
    t = {"u": rand(S, B, H, dtype=dtype, seed=seed + 1), "delta": rand(S, B, H, dtype=dtype, scale=0.5, seed=seed + 2),
         "A": -torch.exp(rand(H, N, dtype=F32, seed=seed + 3)), "B": rand(S, B, G, N, dtype=dtype, seed=seed + 4),
         "C": rand(S, B, G, N, dtype=dtype, seed=seed + 5)}
    t["D"] = rand(H, dtype=F32, seed=seed + 6) if "D" in opts else None
    t["z"] = rand(S, B, H, dtype=dtype, seed=seed + 7) if "z" in opts else None
    t["delta_bias"] = rand(H, dtype=F32, seed=seed + 8) - 2 if "b" in opts else None
    t["state"] = rand(B, H, N, dtype=F32, seed=seed + 9) if "s" in opts else None
    clean = dict(t)
    for k in ("u", "delta", "B", "C", "z"):
        if t[k] is not None:
            t[k] = poison(as_strided(t[k].clone(), layout), lengths)
    return t, clean


SCAN = [  # S, B, H, N, G, dtype, options (D, z, delta_bias, state, softplus p), layout, lengths
    (1, 1, 1, 1, 1, BF16, "", "dense", None),
    (1, 2, 8, 16, 1, FP16, "Dzbsp", "dense", None),
    (2, 1, 64, 16, 1, BF16, "Dzbp", "slice", None),
    (31, 2, 65, 16, 1, BF16, "Dzbsp", "dense", [31, 0]),
    (32, 1, 128, 16, 2, BF16, "zbsp", "batch first", None),
    (33, 3, 130, 16, 2, FP16, "Dzbsp", "odd", [33, 1, 32]),
    (40, 2, 20, 4, 1, BF16, "Dp", "dense", [40, 77]),
    (65, 2, 36, 8, 3, BF16, "Dzbsp", "slice", [-1, 64]),
    (70, 1, 300, 3, 1, FP16, "Dzbsp", "dense", None),
    (50, 2, 33, 13, 3, BF16, "Dzbsp", "odd", [50, 17]),
    (97, 1, 70, 32, 1, BF16, "Dzbsp", "dense", None),
    (130, 2, 24, 20, 2, FP16, "Dzbsp", "slice", [129, 66]),
    (130, 1, 40, 64, 1, BF16, "Dzbsp", "dense", [128]),
    (66, 1, 18, 33, 2, BF16, "zs", "odd", None),
    (300, 1, 16, 16, 1, BF16, "Dzbsp", "dense", [290]),
    (517, 2, 10, 16, 5, FP16, "Dzbsp", "slice", [517, 129]),
]


def reference_scan(clean, opts, lengths):
    leaves = {k: ref.to64(v, grad=True) for k, v in clean.items()}
    y, f = ref.scan(leaves["u"], leaves["delta"], leaves["A"], leaves["B"], leaves["C"], leaves["D"], leaves["z"],
                    leaves["delta_bias"], "p" in opts, lengths, leaves["state"])
    return leaves, y, f


@pytest.mark.parametrize("S,B,H,N,G,dtype,opts,layout,lengths", SCAN)
def test_selective_scan(S, B, H, N, G, dtype, opts, layout, lengths):
    ln = lens(lengths)
    if "p" not in opts:
        opts_scale = 0.2    # raw steps of either sign: decays stay near 1
    t, clean = scan_inputs(S, B, H, N, G, dtype, opts, layout, ln)
    if "p" not in opts:
        for d in (t, clean):
            d["delta"] = (d["delta"] * opts_scale).to(dtype)
            d["A"] = d["A"] * opts_scale
    args = [t[k] for k in ("u", "delta", "A", "B", "C", "D", "z", "delta_bias")]
    kw = dict(delta_softplus="p" in opts, lengths=ln, state=t["state"])
    leaves, ry, rf = reference_scan(clean, opts, lengths)
    y, final = m.selective_scan(*args, **kw, return_state=True)
    ref.check(y, ry, N + 64, "y")
    ref.check(final, rf, N + 64, "final state")
    assert torch.equal(m.selective_scan(*args, **kw), y)

    gy, gf = poison(rand(S, B, H, dtype=dtype, seed=20), ln), rand(B, H, N, dtype=F32, seed=21)
    got = m.selective_scan_backward(gy, *args, **kw, grad_final_state=gf)
    loss = (ry * ref.to64(torch.nan_to_num(gy, nan=0.0))).sum() + (rf * ref.to64(gf)).sum()
    names = [k for k in got._fields if leaves[k] is not None]
    want = torch.autograd.grad(loss, [leaves[k] for k in names], allow_unused=True)
    for k, v in zip(names, want):
        v = torch.zeros_like(leaves[k]) if v is None else v
        terms = {"B": H // G + 64, "C": H // G + 64, "A": S * B, "D": S * B, "delta_bias": S * B}.get(k, 4 * N + 64)
        ref.check(getattr(got, k), v, terms, k)
    for k in got._fields:
        assert (getattr(got, k) is None) == (leaves[k] is None), k
    again = m.selective_scan_backward(gy, *args, **kw, grad_final_state=gf)
    for a, b in zip(got, again):
        assert a is None or torch.equal(a, b)


@pytest.mark.parametrize("which", ["u", "delta", "A", "B", "C", "D", "z", "delta_bias", "state"])
def test_selective_scan_gradient_by_differences(which):
    S, B, H, N, G, opts, lengths = 45, 2, 12, 16, 2, "Dzbsp", [45, 30]
    t, clean = scan_inputs(S, B, H, N, G, BF16, opts, "dense", None)
    gy, gf, ln = rand(S, B, H, seed=20), rand(B, H, N, dtype=F32, seed=21), lens(lengths)
    got = m.selective_scan_backward(gy, *[t[k] for k in ("u", "delta", "A", "B", "C", "D", "z", "delta_bias")],
                                    delta_softplus=True, lengths=ln, state=t["state"], grad_final_state=gf)
    leaves = {k: ref.to64(v) for k, v in clean.items()}

    def loss():
        y, f = ref.scan(*[leaves[k] for k in ("u", "delta", "A", "B", "C", "D", "z", "delta_bias")], True, lengths,
                        leaves["state"])
        return (y * ref.to64(gy)).sum() + (f * ref.to64(gf)).sum()

    by_diff, by_grad, scale = ref.differences(loss, leaves[which], getattr(got, which), eps=1e-5)
    u = 2.0 ** -8 if which in ("u", "delta", "B", "C", "z") else 2.0 ** -16
    assert abs(by_diff - by_grad) <= u * scale + 1e-5 * (1 + abs(by_diff))


def test_long_sequence_of_few_channels_is_cut_and_joined():
    """One sequence of 3000 tokens and 8 channels: many chunks; the end state of
    a prompt cut in two calls is the one of the whole."""
    S, H, N = 3000, 8, 16
    t, clean = scan_inputs(S, 1, H, N, 1, BF16, "Dzbsp", "dense", None)
    t["A"] *= 0.01      # long memory: chunks far back still count
    clean["A"] = t["A"]
    names = ("u", "delta", "A", "B", "C", "D", "z", "delta_bias")
    y, f = m.selective_scan(*[t[k] for k in names], delta_softplus=True, state=t["state"], return_state=True)
    _, ry, rf = reference_scan(clean, "p", None)
    ref.check(y, ry, N + S, "y")
    ref.check(f, rf, N + S, "final state")
    cut = 1717
    a = {k: v[:cut] if k in ("u", "delta", "B", "C", "z") else v for k, v in t.items()}
    b = {k: v[cut:] if k in ("u", "delta", "B", "C", "z") else v for k, v in t.items()}
    y1, f1 = m.selective_scan(*[a[k] for k in names], delta_softplus=True, state=t["state"], return_state=True)
    y2, f2 = m.selective_scan(*[b[k] for k in names], delta_softplus=True, state=f1, return_state=True)
    ref.check(torch.cat([y1, y2]), ry, N + S, "y of two calls")
    ref.check(f2, rf, N + S, "final state of two calls")


@pytest.mark.parametrize("B,H,N,G,dtype,opts,rows,slots,layout", [
    (1, 1, 1, 1, BF16, "", 1, None, "dense"), (1, 8, 16, 1, FP16, "Dzbp", 1, None, "dense"),
    (3, 66, 16, 2, BF16, "Dzbp", 7, [6, 0, 3], "slice"), (5, 130, 13, 1, BF16, "zbp", 6, [5, -1, 0, 6, 2], "odd"),
    (4, 96, 32, 4, FP16, "Dp", 4, [3, 2, 1, 0], "dense"), (2, 10, 64, 1, BF16, "Dzb", 5, None, "dense"),
    (2, 300, 4, 3, BF16, "Dzbp", 2, None, "slice"), (2, 30, 7, 3, FP16, "Dzbp", 2, [1, 0], "odd"),
])
def test_selective_scan_step(B, H, N, G, dtype, opts, rows, slots, layout):
    t, clean = scan_inputs(1, B, H, N, G, dtype, opts, layout, None)
    one = {k: v[0] if v is not None and k in ("u", "delta", "B", "C", "z") else v for k, v in t.items()}
    cache = rand(rows, H, N, dtype=F32, seed=40)
    before = cache.clone()
    y = m.selective_scan_step(one["u"], one["delta"], cache, one["A"], one["B"], one["C"], one["D"], one["z"],
                              one["delta_bias"], delta_softplus="p" in opts, slots=lens(slots))
    for i in range(B):
        r = i if slots is None else slots[i]
        if not 0 <= r < rows:
            assert not y[i].any()
            continue
        row = {k: ref.to64(v[:, i:i + 1] if v is not None and k in ("u", "delta", "B", "C", "z") else v) for k, v in clean.items()}
        ry, rf = ref.scan(*[row[k] for k in ("u", "delta", "A", "B", "C", "D", "z", "delta_bias")], "p" in opts, None,
                          ref.to64(before[r:r + 1]))
        ref.check(y[i], ry[0, 0], N, "y")
        ref.check(cache[r], rf[0], N, "state")
        before[r] = cache[r]
    assert torch.equal(before, cache)


def test_steps_continue_a_prompt():
    """A prompt and then single tokens give what the whole sequence gives."""
    S, cut, B, H, W, N = 20, 13, 2, 40, 4, 16
    x, w, b = rand(S, B, H, seed=1), rand(W, H, scale=0.5, seed=2), rand(H, seed=3)
    whole = m.short_conv(x, w, b)
    y, win = m.short_conv(x[:cut], w, b, return_state=True)
    parts = [y] + [m.short_conv_step(x[i], win, w, b)[None] for i in range(cut, S)]
    assert torch.equal(torch.cat(parts), whole)
    t, _ = scan_inputs(S, B, H, N, 1, BF16, "Dzbp", "dense", None)
    names = ("u", "delta", "A", "B", "C", "D", "z", "delta_bias")
    y, f = m.selective_scan(*[t[k] for k in names], delta_softplus=True, return_state=True)
    p = {k: v[:cut] if k in ("u", "delta", "B", "C", "z") else v for k, v in t.items()}
    y1, st = m.selective_scan(*[p[k] for k in names], delta_softplus=True, return_state=True)
    outs = [y1]
    for i in range(cut, S):
        o = {k: v[i] if k in ("u", "delta", "B", "C", "z") else v for k, v in t.items()}
        outs.append(m.selective_scan_step(o["u"], o["delta"], st, o["A"], o["B"], o["C"], o["D"], o["z"],
                                          o["delta_bias"], delta_softplus=True)[None])
    ref.check(torch.cat(outs), y.double(), 16, "y")
    ref.check(st, f.double(), 16, "state")


def test_broadcast_rows():
    """Zero strides: one row of B, C and z for every token and sequence."""
    S, B, H, N = 37, 2, 70, 16
    t, clean = scan_inputs(S, B, H, N, 1, BF16, "Dzbp", "dense", None)
    for k in ("B", "C", "z"):
        one = t[k][:1, :1]
        t[k], clean[k] = one.expand_as(t[k]), one.expand_as(t[k]).contiguous()
    names = ("u", "delta", "A", "B", "C", "D", "z", "delta_bias")
    _, ry, _ = reference_scan(clean, "p", None)
    ref.check(m.selective_scan(*[t[k] for k in names], delta_softplus=True), ry, N + 64, "y")


def test_infinite_and_extreme_values_stay_where_they_are():
    """Large steps forget everything, very negative ones keep it; an infinite
    input reaches later tokens of its channel only."""
    S, H, N = 40, 64, 16
    t, clean = scan_inputs(S, 1, H, N, 1, BF16, "Dbp", "dense", None)
    t["delta"][10] = 300.0          # exp(dt A) underflows
    t["delta"][20] = -300.0         # dt = 0
    names = ("u", "delta", "A", "B", "C", "D", "z", "delta_bias")
    y = m.selective_scan(*[t[k] for k in names], delta_softplus=True)
    clean["delta"] = t["delta"]
    _, ry, _ = reference_scan(clean, "p", None)
    ref.check(y, ry, N + 64, "y")
    t["u"][25, 0, 3] = float("inf")
    y2 = m.selective_scan(*[t[k] for k in names], delta_softplus=True)
    assert not torch.isfinite(y2[25:, 0, 3]).any()
    keep = torch.ones(H, dtype=torch.bool, device="cuda")
    keep[3] = False
    assert torch.equal(y2[:, :, keep], y[:, :, keep]) and torch.equal(y2[:25], y[:25])


def test_other_stream():
    """Work on a side stream, its tensors freed and reused meanwhile."""
    S, B, H, N = 256, 2, 128, 16
    t, _ = scan_inputs(S, B, H, N, 1, BF16, "Dzbp", "dense", None)
    names = ("u", "delta", "A", "B", "C", "D", "z", "delta_bias")
    want = m.selective_scan(*[t[k] for k in names], delta_softplus=True)
    x, w = rand(S, B, H, seed=1), rand(4, H, seed=2)
    want_y = m.short_conv(x, w)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for handle in (side, side.cuda_stream):
        got = m.selective_scan(*[t[k] for k in names], delta_softplus=True, stream=handle)
        got_y = m.short_conv(x, w, stream=handle)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(got, want) and torch.equal(got_y, want_y)


def test_capture_in_a_graph():
    """A decode step in a CUDA graph: the cache moves on at every replay."""
    B, H, W, N = 2, 64, 4, 16
    x, w, win = rand(B, H, seed=1), rand(W, H, seed=2), rand(B, W - 1, H, seed=3)
    t, _ = scan_inputs(1, B, H, N, 1, BF16, "Dzbp", "dense", None)
    st = rand(B, H, N, dtype=F32, seed=9)
    o = {k: v[0] if v is not None and k in ("u", "delta", "B", "C", "z") else v for k, v in t.items()}

    def step(win, st, y1, y2):
        m.short_conv_step(x, win, w, y=y1)
        m.selective_scan_step(o["u"], o["delta"], st, o["A"], o["B"], o["C"], o["D"], o["z"], o["delta_bias"],
                              delta_softplus=True, y=y2)

    w2, s2, y1, y2 = win.clone(), st.clone(), torch.empty_like(x), torch.empty_like(x)
    for _ in range(3):
        step(w2, s2, y1, y2)
    want = [v.clone() for v in (w2, s2, y1, y2)]
    w3, s3 = win.clone(), st.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(w3, s3, y1, y2)
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    for a, b in zip(want, (w3, s3, y1, y2)):
        assert torch.equal(a, b)


# ------------------------------------------------------------------ refusals
def test_refusals():
    S, B, H, W, N = 4, 2, 16, 4, 16
    x, w, b = rand(S, B, H), rand(W, H), rand(H)
    for bad in (x.cpu(), x[0], x.transpose(0, 2)):
        with pytest.raises(ValueError):
            m.short_conv(bad, w)
    with pytest.raises(TypeError):
        m.short_conv(x.float(), w)
    with pytest.raises(TypeError):
        m.short_conv(x, w.half())
    for kw in (dict(bias=b[1:]), dict(state=rand(B, W, H)), dict(lengths=torch.zeros(3, dtype=torch.int32, device="cuda")),
               dict(activation="relu"), dict(lengths=torch.zeros(B, dtype=torch.int32)), dict(y=rand(S, B, 2 * H)[:, :, :H])):
        with pytest.raises(ValueError):
            m.short_conv(x, w, **kw)
    with pytest.raises(TypeError):
        m.short_conv(x, w, lengths=torch.zeros(B, dtype=torch.int64, device="cuda"))
    with pytest.raises(m.Mcc1dError):
        m.short_conv(x, rand(9, H))
    with pytest.raises(ValueError):
        m.short_conv_step(x[0], rand(1, W - 1, H), w)
    with pytest.raises(ValueError):
        m.short_conv_backward(x[:3], x, w)
    t, _ = scan_inputs(S, B, H, N, 1, BF16, "Dzbsp", "dense", None)
    names = ("u", "delta", "A", "B", "C", "D", "z", "delta_bias")
    good = [t[k] for k in names]
    for i, bad in ((1, t["delta"][:3]), (3, t["B"][..., :8]), (4, t["C"].transpose(2, 3)), (5, t["D"][1:]), (2, t["A"][:8])):
        with pytest.raises(ValueError):
            m.selective_scan(*good[:i], bad, *good[i + 1:])
    for i, bad in ((1, t["delta"].half()), (2, t["A"].bfloat16()), (7, t["delta_bias"].double())):
        with pytest.raises(TypeError):
            m.selective_scan(*good[:i], bad, *good[i + 1:])
    with pytest.raises(ValueError):
        m.selective_scan(*good, state=t["state"][:1])
    with pytest.raises(ValueError):
        m.selective_scan_backward(t["u"][:2], *good)
    with pytest.raises(m.Mcc1dError):       # three groups do not divide 16 channels
        m.selective_scan(*good[:3], rand(S, B, 3, N), rand(S, B, 3, N), *good[5:])
    with pytest.raises(m.Mcc1dError):       # more states than the library takes
        m.selective_scan(*good[:2], rand(H, 65, dtype=F32), rand(S, B, 1, 65), rand(S, B, 1, 65), *good[5:])
    with pytest.raises(TypeError):
        m.selective_scan_step(t["u"][0], t["delta"][0], t["state"].half(), t["A"], t["B"][0], t["C"][0])
    with pytest.raises(ValueError):
        m.selective_scan_step(t["u"][0], t["delta"][0], t["state"][:1], t["A"], t["B"][0], t["C"][0])
    assert ctypes.sizeof(m.ScanArgs) > 0


def test_offsets_past_32_bits():
    """More than 2^31 elements: the last tokens agree with the same tokens run
    alone from the carried window and state."""
    S, H, N, last = 540_000, 4096, 4, 50
    assert S * H > 2 ** 31
    g = torch.Generator(device="cuda").manual_seed(0)
    x = torch.randn(S, 1, H, generator=g, device="cuda", dtype=BF16)
    w, b = rand(4, H, seed=2), rand(H, seed=3)
    y = torch.empty(S, 1, H, device="cuda", dtype=BF16)     # too large for guards to be worth it
    m.short_conv(x, w, b, y=y)
    _, window = m.short_conv(x[:S - last], w, b, return_state=True, y=torch.empty_like(y[:S - last]))
    assert torch.equal(window, x[S - last - 3:S - last].transpose(0, 1))
    assert torch.equal(m.short_conv(x[S - last:], w, b, state=window), y[S - last:])
    delta, A, Bm = x.sub_(1.0), -torch.exp(rand(H, N, dtype=F32)), rand(last, 1, 1, N).repeat(S // last, 1, 1, 1)
    _, state = m.selective_scan(y[:S - last], delta[:S - last], A, Bm[:S - last], Bm[:S - last], delta_softplus=True,
                                return_state=True, y=torch.empty_like(y[:S - last]))
    tail = slice(S - last, S)
    want, f = m.selective_scan(y[tail], delta[tail], A, Bm[tail], Bm[tail], delta_softplus=True, state=state, return_state=True)
    got, f2 = m.selective_scan(y, delta, A, Bm, Bm, delta_softplus=True, return_state=True, y=torch.empty_like(y))
    ref.check(got[tail], want.double(), N + 64, "y")
    ref.check(f2, f.double(), N + 64, "state")
