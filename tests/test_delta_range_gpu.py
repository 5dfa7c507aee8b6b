"""The gated delta rule where a state grows or fades by many powers of two within
a chunk, and where values, states or gradients are much smaller than others of
their chunk: every token against float64 relative to its own size."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import causal_conv_backward_gb300 as m  # noqa: E402
import delta_reference as ref  # noqa: E402
from ssm_reference import rounding, to64  # noqa: E402
from test_delta_gpu import BF16, F32, cuda_ready, rand  # noqa: E402,F401

FORMS = dict(delta_softplus=False, beta_sigmoid=True, qk_norm=True)


def near(got, want, terms, size, what):
    """ssm_reference.check's bound (16 2^-24 (8 + sqrt(terms)) of a typical value, and
    the final rounding), the typical value taken from `size` in place of the
    largest of all."""
    dtype, got, want = got.dtype, to64(got), want.detach()
    assert torch.isfinite(got).all(), f"{what}: not finite"
    tol = 16 * 2.0 ** -24 * (8 + terms ** 0.5) * size.detach() + torch.zeros_like(want)
    if dtype is not F32:
        u, step = rounding(dtype)
        tol = tol + u * want.abs() + step
    off = (got - want).abs() / tol.clamp(min=1e-300)
    assert not (off > 1).any(), f"{what}: {int((off > 1).sum())} of {off.numel()} off, worst {float(off.max()):.3g} of the tolerance"


def of_row(want):
    """A token's own size: the largest along its last axis."""
    return want.abs().amax(-1, keepdim=True)


def of_neighbours(want):
    """The size of a gate's gradient, which is one number and may cancel to nothing:
    the largest of its head within eight tokens."""
    w = want.detach().abs().permute(1, 2, 0)
    return torch.nn.functional.max_pool1d(w, 17, 1, 8).permute(2, 0, 1)


def inputs(steps, B=2, H=2, G=1, K=32, V=24, seed=0):
    """`steps`: log2 of each token's decay. Heads and sequences differ by a tenth of it."""
    S = len(steps)
    t = dict(q=rand(S, B, G, K, seed=seed + 1), k=rand(S, B, G, K, seed=seed + 2), v=rand(S, B, H, V, seed=seed + 3))
    x = torch.tensor(steps, device="cuda", dtype=F32)[:, None, None] * 0.6931472
    t["delta"] = (x * (1 - 0.1 * torch.rand(S, B, H, device="cuda", generator=torch.Generator(device="cuda").manual_seed(seed + 4)))).to(BF16)
    t["beta"] = rand(S, B, H, seed=seed + 5)
    t["A"] = torch.ones(H, device="cuda")
    t["state"] = rand(B, H, V, K, dtype=F32, seed=seed + 6)
    return t, rand(S, B, H, V, seed=seed + 7), rand(B, H, V, K, dtype=F32, seed=seed + 8)


def exact(t):
    d = {k: to64(v, grad=True) for k, v in t.items()}
    y, final = ref.delta_rule(d["q"], d["k"], d["v"], d["delta"], d["beta"], d["A"], None, False, True, True, state=d["state"])
    return d, y, final


OUT, STATES, TOKENS = ("y", "final"), ("grad v", "grad state"), ("grad q", "grad k", "grad delta", "grad beta", "grad A")


def run(t, gy, gf, what):
    S, B, H, V = t["v"].shape
    K = t["k"].shape[-1]
    args = [t[k] for k in ("q", "k", "v", "delta", "beta", "A")]
    leaves, ry, rf = exact(t)
    y, final = m.gated_delta(*args, state=t["state"], return_state=True, **FORMS)
    if "y" in what:
        near(y, ry, K + 256, of_row(ry), "y")
    if "final" in what:
        near(final, rf, K + 256, rf.abs().amax((-1, -2), keepdim=True), "final state")
    if not any(k.startswith("grad") for k in what):
        return
    got = m.gated_delta_backward(gy if gy is not None else torch.zeros_like(t["v"]), *args, state=t["state"], grad_final_state=gf, **FORMS)
    loss = ((ry * to64(gy)).sum() if gy is not None else 0) + ((rf * to64(gf)).sum() if gf is not None else 0)
    names = ("q", "k", "v", "delta", "beta", "A", "state")
    want = dict(zip(names, torch.autograd.grad(loss, [leaves[k] for k in names], allow_unused=True)))
    want = {k: torch.zeros_like(leaves[k]) if w is None else w for k, w in want.items()}
    gates = {k: of_neighbours(want[k]) for k in ("delta", "beta")}
    size = {"q": of_row(want["q"]), "k": of_row(want["k"]), "v": of_row(want["v"]), "state": want["state"].abs().amax((-1, -2), keepdim=True), **gates,
            "A": (gates["delta"] * to64(t["delta"]).abs()).sum((0, 1))}
    terms = {"delta": K * V, "beta": K * V, "A": S * B * 64, "state": K + 256}
    for k in names:
        if "grad " + k in what:
            near(getattr(got, k), want[k], terms.get(k, 2 * V * K + 256), size[k], "grad " + k)


def growing(S, log2, K, V):
    """States that grow by 2^log2 in 64 tokens, up to what fp32 holds."""
    t, gy, gf = inputs([log2 / 64] * S, K=K, V=V)
    if log2 > 100:        # sums of some terms below the types' largest value
        gy, gf = gy * 2.0 ** -10, gf * 2.0 ** -10
        t["v"], t["state"] = t["v"] * 2.0 ** -10, t["state"] * 2.0 ** -10
    return t, gy, gf


GROWTH = pytest.mark.parametrize("S,log2", [(16, 30), (200, 5), (200, 10), (200, 17), (200, 30), (96, 60), (64, 100), (64, 120)])
SHAPES = pytest.mark.parametrize("K,V", [(32, 24), (128, 72)])
GRADIENTS = pytest.mark.parametrize("part", [STATES, TOKENS], ids=["states", "tokens"])


@GROWTH
@SHAPES
def test_growth(S, log2, K, V):
    run(*growing(S, log2, K, V), OUT)


PATHS = {"down and up": [-1.5] * 32 + [1.5] * 32, "up and down": [1.5] * 32 + [-1.5] * 32, "in turn": [8.0, -8.0] * 32,
         "one step up": [0.0] * 30 + [40.0] + [0.0] * 33, "one step down": [0.0] * 30 + [-40.0] + [0.0] * 33,
         "gone after each token": [-60.0] * 64}


@pytest.mark.parametrize("path", PATHS)
def test_growth_and_decay_in_one_chunk(path):
    run(*inputs(PATHS[path] + [0.0] * 20), OUT)


@GROWTH
@SHAPES
@GRADIENTS
def test_gradients_of_growth(S, log2, K, V, part):
    run(*growing(S, log2, K, V), part)


@pytest.mark.parametrize("path", PATHS)
@GRADIENTS
def test_gradients_of_growth_and_decay_in_one_chunk(path, part):
    run(*inputs(PATHS[path] + [0.0] * 20), part)


# what is left of a state or of a gradient after 200 tokens: 2^-20 to 2^-100 of it
RATES = [-0.1, -0.3, -0.5]


@pytest.mark.parametrize("rate", RATES)
@SHAPES
@pytest.mark.parametrize("where", ["last chunk", "last token", "final state"])
@GRADIENTS
def test_gradients_that_come_from_the_end_only(rate, K, V, where, part):
    t, gy, gf = inputs([rate] * 200, K=K, V=V)
    if where == "final state":
        return run(t, None, gf, part)
    gy[:192 if where == "last chunk" else 199] = 0
    run(t, gy, None, part)


@pytest.mark.parametrize("S,rate", [(40, -2.0), (64, -1.5)])
@GRADIENTS
def test_gradients_of_a_final_state_that_has_faded_in_a_chunk(S, rate, part):
    t, _, gf = inputs([rate] * S)
    run(t, None, gf, part)


@pytest.mark.parametrize("rate", RATES)
@SHAPES
@pytest.mark.parametrize("first", [0, 1, 40])
def test_values_that_end(rate, K, V, first):
    """Nothing but the carried state, or the first tokens' values, is left to read."""
    t, gy, gf = inputs([rate] * 200, K=K, V=V)
    t["v"][first:] = 0
    run(t, gy, gf, OUT)


@pytest.mark.parametrize("rate", [-0.5, -1.0, -2.0])
def test_states_that_fade_to_nothing(rate):
    """Below what fp32 holds, and on from there with values again."""
    t, gy, gf = inputs([rate] * 600)
    t["v"][:500] = 0
    leaves, ry, rf = exact(t)
    y, final = m.gated_delta(*[t[k] for k in ("q", "k", "v", "delta", "beta", "A")], state=t["state"], return_state=True, **FORMS)
    late = ry[500:]
    near(y[500:], late, 32 + 256, of_row(late), "y")
    near(final, rf, 32 + 256, rf.abs().amax((-1, -2), keepdim=True), "final state")
    assert (to64(y[:500]) - ry[:500].detach()).abs().max() < 2.0 ** -8 * float(ry[:500].detach().abs().max())


@pytest.mark.parametrize("what", ["one key", "any keys"])
@pytest.mark.parametrize("S", [64, 150])
def test_keys_that_decays_hold(what, S):
    """Keys that are not divided by their lengths: b |k|^2 = 6 turns a state along
    the key round to five times itself, 2^148 in a chunk of one key, and the decay
    of 1/8 a token holds it."""
    t, gy, gf = inputs([-3.0] * S)
    t["k"] = (t["k"].float() / t["k"].float().norm(dim=-1, keepdim=True) * 6 ** 0.5).to(BF16)
    if what == "one key":
        t["k"] = t["k"][:1].expand_as(t["k"])
    t["beta"], forms = torch.ones_like(t["beta"]), dict(delta_softplus=False, beta_sigmoid=False, qk_norm=False)
    K, V = 32, 24
    args = [t[k] for k in ("q", "k", "v", "delta", "beta", "A")]
    d = {k: to64(v, grad=True) for k, v in t.items()}
    ry, rf = ref.delta_rule(d["q"], d["k"], d["v"], d["delta"], d["beta"], d["A"], None, False, False, False, state=d["state"])
    y, final = m.gated_delta(*args, state=t["state"], return_state=True, **forms)
    near(y, ry, K + 256, of_row(ry), "y")
    near(final, rf, K + 256, rf.abs().amax((-1, -2), keepdim=True), "final state")
    got = m.gated_delta_backward(gy, *args, state=t["state"], grad_final_state=gf, **forms)
    names = ("q", "k", "v", "state")
    for k, want in zip(names, torch.autograd.grad((ry * to64(gy)).sum() + (rf * to64(gf)).sum(), [d[k] for k in names])):
        near(getattr(got, k), want, 2 * V * K + 256, of_row(want) if k != "state" else want.abs().amax((-1, -2), keepdim=True), "grad " + k)


@SHAPES
@pytest.mark.parametrize("part", [OUT, STATES], ids=["outputs", "states"])
@pytest.mark.parametrize("size", [100, 110, 116, 120])
def test_states_near_the_largest(K, V, part, size):
    """States and gradients some 2^5 to 2^26 below fp32's largest value: what bounds
    their rows passes it, the rows themselves do not."""
    t, gy, gf = inputs([-0.01] * 200, K=K, V=V)
    if part is OUT:
        t["v"], t["state"] = t["v"] * 2.0 ** size, t["state"] * 2.0 ** size
    else:
        gy, gf = gy * 2.0 ** size, gf * 2.0 ** size
    run(t, gy, gf, part)
