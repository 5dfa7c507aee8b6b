"""Values at the edges of the short convolution and the selective scan: what a
mask, a padding lane or a padding row covers leaves nothing behind, whatever
stands there, and finite results come out of large intermediate ones."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import causal_conv_backward_gb300 as m  # noqa: E402
import ssm_reference as ref  # noqa: E402
from test_ssm_gpu import BF16, F32, cuda_ready, guards, lens, rand, reference_scan, scan_inputs  # noqa: E402,F401
from test_ssm_long_gpu import leaf, scan64, scan_bwd_chunks  # noqa: E402

SCAN_ARGS = ("u", "delta", "A", "B", "C", "D", "z", "delta_bias")
INF = float("inf")


# N = 4, 16, 64: one, four and sixteen lanes per channel, blocks of 256, 64 and 16 channels
@pytest.mark.parametrize("N,H,G", [(4, 5, 1), (16, 5, 1), (16, 6, 2), (64, 3, 1)])
def test_growing_states_leave_the_groups_other_channels_alone(N, H, G):
    """A > 0 with small steps: every state grows a little, and lanes past the
    group's last channel, whose steps are not small, add nothing."""
    S, B = 40, 2
    t, clean = scan_inputs(S, B, H, N, G, BF16, "Dzsp", "dense", None)
    for d in (t, clean):
        d["A"] = 60 + 0.1 * rand(H, N, dtype=F32, seed=30)
        d["delta"] = (-6.9 + 0.1 * rand(S, B, H, dtype=F32, seed=31)).to(BF16)   # steps near 0.001
    args = [t[k] for k in SCAN_ARGS]
    gy, gf = rand(S, B, H, seed=20), rand(B, H, N, dtype=F32, seed=21)
    leaves, ry, rf = reference_scan(clean, "p", None)
    got = m.selective_scan_backward(gy, *args, delta_softplus=True, state=t["state"], grad_final_state=gf)
    loss = (ry * ref.to64(gy)).sum() + (rf * ref.to64(gf)).sum()
    names = [k for k in got._fields if leaves[k] is not None]
    for k, want in zip(names, torch.autograd.grad(loss, [leaves[k] for k in names])):
        terms = {"B": H // G + 64, "C": H // G + 64, "A": S * B, "D": S * B}.get(k, 4 * N + 64)
        ref.check(getattr(got, k), want, terms, k)


@pytest.mark.parametrize("H,W", [(64, 4), (66, 6), (33, 4)])
@pytest.mark.parametrize("activation", ["silu", None])
def test_conv_sequence_without_tokens_adds_nothing(H, W, activation):
    """Whatever the window of a length of zero holds, the weights' gradients
    are those of the other sequences."""
    S, B = 21, 3
    x, w, b, gy = rand(S, B, H, seed=1), rand(W, H, scale=0.5, seed=2), rand(H, seed=3), rand(S, B, H, seed=4)
    state, ln = rand(B, W - 1, H, seed=5), lens([21, 0, 13])
    clean = m.short_conv_backward(gy, x, w, b, activation=activation, lengths=ln, state=state)
    state[1, :, ::2], state[1, :, 1::2] = INF, float("nan")
    got = m.short_conv_backward(gy, x, w, b, activation=activation, lengths=ln, state=state)
    for k in ("x", "weight", "bias", "state"):
        assert torch.equal(getattr(got, k), getattr(clean, k)), k


@pytest.mark.parametrize("H,W", [(64, 4), (66, 6), (33, 4)])
def test_conv_infinite_last_token_meets_its_own_taps_only(H, W):
    """Without an activation x(n-1) reaches one row of grad_weight; the rows
    past the length give the same result as no rows there."""
    S, n = 40, 21
    x, w, gy = rand(S, 1, H, seed=1), rand(W, H, scale=0.5, seed=2), rand(S, 1, H, seed=4)
    x[n - 1, 0, 3] = INF
    got = m.short_conv_backward(gy, x, w, activation=None, lengths=lens([n]))
    want = m.short_conv_backward(gy[:n], x[:n], w, activation=None)
    assert want.weight.isinf().sum() == 1 and torch.isfinite(want.weight[:W - 1]).all()
    assert torch.equal(got.weight, want.weight)
    assert torch.equal(got.x[:n], want.x) and not got.x[n:].any()


@pytest.mark.parametrize("bad", [INF, float("nan")])
def test_conv_gradient_past_the_end_is_zero_for_any_weight(bad):
    S, H, W, n = 40, 64, 4, 21
    x, w, gy = rand(S, 1, H, seed=1), rand(W, H, scale=0.5, seed=2), rand(S, 1, H, seed=4)
    w[:, 5] = bad
    got = m.short_conv_backward(gy, x, w, lengths=lens([n]))
    assert not got.x[n:].any()


@pytest.mark.parametrize("S,lengths", [(20, None), (21, None), (48, [37])])
def test_infinite_last_input_leaves_grad_A_finite(S, lengths):
    """grad_A sums g(t) a(t) h(t-1): the state after the last token is not in
    it, though it stands in the rows that fill the last tile."""
    H, N = 6, 16
    t, clean = scan_inputs(S, 1, H, N, 1, BF16, "Dp", "dense", None)
    n = S if lengths is None else lengths[0]
    for d in (t, clean):
        d["u"][n - 1, 0, 2] = INF
    gy = rand(S, 1, H, seed=20)
    leaves, ry, _ = reference_scan(clean, "p", lengths)
    want = torch.autograd.grad((ry[:n] * ref.to64(gy)[:n]).sum(), leaves["A"])[0]
    assert torch.isfinite(want).all()
    got = m.selective_scan_backward(gy, *[t[k] for k in SCAN_ARGS], delta_softplus=True, lengths=lens(lengths))
    ref.check(got.A, want, S, "A")


@pytest.mark.parametrize("N", [4, 16, 64])
def test_empty_states_stay_empty_through_any_growth(N):
    """Zero inputs first (padding on the left), with A > 0 and steps so large
    that the growth over a chunk is past fp32: the states stay zero until the
    first input, and what follows is as if it stood alone."""
    S, H, first, G = 260, 10, 215, 1
    t, clean = scan_inputs(S, 1, H, N, G, BF16, "Dzp", "dense", None)
    for d in (t, clean):
        d["A"] = 1 + 0.1 * rand(H, N, dtype=F32, seed=30)
        d["u"][:first] = 0
        d["delta"][:first] = 30.0        # e^(30 A) per token
        d["delta"][first:] = -4.0
    args = [t[k] for k in SCAN_ARGS]
    alone = {k: v[first:] if v is not None and k in ("u", "delta", "B", "C", "z") else v for k, v in clean.items()}
    leaves, ry, rf = reference_scan(alone, "p", None)
    y, final = m.selective_scan(*args, delta_softplus=True, return_state=True)
    assert not y[:first].any()
    ref.check(y[first:], ry, N + 64, "y")
    ref.check(final, rf, N + 64, "final state")
    gy = rand(S, 1, H, seed=20)
    got = m.selective_scan_backward(gy, *args, delta_softplus=True)
    names = ("u", "delta", "B", "C", "z")
    for k, want in zip(names, torch.autograd.grad((ry * ref.to64(gy[first:])).sum(), [leaves[k] for k in names])):
        ref.check(getattr(got, k)[first:], want, {"B": H + 64, "C": H + 64}.get(k, 4 * N + 64), k)


def test_empty_states_stay_empty_in_chunks_of_several_tiles():
    """The same where the first input stands in a chunk's second tile."""
    S, B, H, N, first = 450, 128, 7, 16, 215
    tiles, chunks = scan_bwd_chunks(S, B, H, N, 1)
    per = -(-tiles // chunks)
    assert first // 16 % per > 0
    t, clean = scan_inputs(S, B, H, N, 1, BF16, "Dzbsp", "dense", None)
    t["A"] = 1 + 0.1 * rand(H, N, dtype=F32, seed=30)
    t["u"][:first] = 0
    t["delta"][:first] = 30.0
    t["delta"][first:] = -4.0
    t["state"].zero_()
    args, cut = [t[k] for k in SCAN_ARGS], ("u", "delta", "B", "C", "z")
    leaves = {k: leaf(v[first:] if k in cut else v) for k, v in t.items()}
    ry, rf = scan64(leaves, None)
    y, final = m.selective_scan(*args, delta_softplus=True, return_state=True)
    assert not y[:first].any()
    ref.check(y[first:], ry, N + S, "y")
    ref.check(final, rf, N + S, "final state")
    gy = rand(S, B, H, seed=20)
    got = m.selective_scan_backward(gy, *args, delta_softplus=True)
    for k, want in zip(cut, torch.autograd.grad((ry * gy[first:].double()).sum(), [leaves[k] for k in cut])):
        ref.check(getattr(got, k)[first:], want, {"B": H + S, "C": H + S}.get(k, 4 * N + S), k)


def test_given_outputs():
    """On an input they are refused; beside one, in the same buffer, they are not."""
    S, B, H, W = 20, 2, 64, 4
    two = torch.cat([rand(1, S, B, H, seed=1), torch.zeros(1, S, B, H, dtype=BF16, device="cuda")])
    x, y, w, win = two[0], two[1], rand(W, H, seed=2), rand(B, W - 1, H, seed=3)
    want = m.short_conv(x, w)
    for bad in (x, two.view(-1)[H:H + S * B * H].view(S, B, H)):
        with pytest.raises(m.Mcc1dError):
            m.short_conv(x, w, y=bad)
    assert m.short_conv(x, w, y=y) is y and torch.equal(y, want)
    with pytest.raises(m.Mcc1dError):
        m.short_conv_step(x[0], win, w, y=x[0])
    with pytest.raises(m.Mcc1dError):
        m.short_conv_step(x[0], win, w, y=win[0, :B])
    t, _ = scan_inputs(S, B, H, 16, 1, BF16, "Dzbp", "dense", None)
    for k in ("u", "delta", "z"):
        with pytest.raises(m.Mcc1dError):
            m.selective_scan(*[t[k] for k in SCAN_ARGS], delta_softplus=True, y=t[k])
    assert torch.equal(x, two[0]) and torch.equal(m.short_conv(x, w), want)


def test_scan_of_more_than_2_31_group_rows():
    """One channel per group, S B G above 2^31; inputs constant over time, so
    that the last tokens are at the fixed point of h = a h + dt u B."""
    S, H = (1 << 19) + 3, 4096
    u, delta, Bm, Cm = rand(1, 1, H, seed=1), rand(1, 1, H, scale=0.5, seed=2), rand(1, 1, H, 1, seed=3), rand(1, 1, H, 1, seed=4)
    A = -1 - rand(H, 1, dtype=F32, seed=5).abs()
    y = torch.empty(S, 1, H, dtype=BF16, device="cuda")
    m.selective_scan(u.expand(S, 1, H), delta.expand(S, 1, H), A, Bm.expand(S, 1, H, 1), Cm.expand(S, 1, H, 1), delta_softplus=True, y=y)
    dt = torch.logaddexp(delta.double(), torch.zeros_like(delta).double())
    a, b, c = torch.exp(dt * A[:, 0].double()), dt * u.double() * Bm[..., 0].double(), Cm[..., 0].double()
    t = torch.arange(1, 41, device="cuda").double().view(-1, 1, 1)
    ref.check(y[:40], (1 - a ** t) / (1 - a) * b * c, 40, "first tokens")
    ref.check(y[-40:], (b / (1 - a) * c).expand(40, 1, H), 40, "last tokens")
