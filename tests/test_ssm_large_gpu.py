"""Backwards over more than 2^31 elements: with a gradient on the last tokens
only, their results are those of the tail of the sequence, in float64."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import causal_conv_backward_gb300 as m  # noqa: E402
import ssm_reference as ref  # noqa: E402
from test_ssm_gpu import BF16, F32, cuda_ready, rand  # noqa: E402,F401
from test_ssm_long_gpu import conv64, leaf, scan64  # noqa: E402

S, H, FROM, LOSS = 540_000, 4096, 800, 50     # the tail, and its last tokens, which have a gradient


def big(seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(S, 1, H, generator=g, device="cuda", dtype=BF16).mul_(scale)


def last(seed):
    gy = torch.zeros(S, 1, H, device="cuda", dtype=BF16)
    gy[-LOSS:] = rand(LOSS, 1, H, seed=seed)
    return gy


def test_conv():
    assert S * H > 2 ** 31
    x, w, b, gy = big(0), rand(4, H, scale=0.5, seed=1), rand(H, seed=2), last(3)
    got = m.short_conv_backward(gy, x, w, b)
    tail = slice(S - FROM, S)
    leaves = [leaf(t) for t in (x[tail], w, b)]
    y, _ = conv64(*leaves, True, None, None)
    for k, want in zip(("x", "weight", "bias"), torch.autograd.grad((y * gy[tail].double()).sum(), leaves)):
        g = getattr(got, k)
        ref.check(g[tail] if k == "x" else g, want, 4 if k == "x" else FROM, k)
    assert not got.x[:S - FROM].any()


def test_scan():
    N = 4
    # memories short enough that the tail's states and gradients are its own
    t = {"u": big(0), "delta": big(1, 0.5), "A": -1 - rand(H, N, dtype=F32, seed=2).abs(),
         "B": rand(S, 1, 1, N, seed=3), "C": rand(S, 1, 1, N, seed=4), "D": rand(H, dtype=F32, seed=5), "z": big(6),
         "delta_bias": rand(H, dtype=F32, seed=7)}
    gy = last(8)
    got = m.selective_scan_backward(gy, *t.values(), delta_softplus=True)
    tail, long = slice(S - FROM, S), ("u", "delta", "B", "C", "z")
    leaves = {k: leaf(v[tail] if k in long else v) for k, v in t.items()}
    y, _ = scan64({**leaves, "state": torch.zeros(1, H, N, dtype=torch.float64, device="cuda")}, None)
    for k, want in zip(leaves, torch.autograd.grad((y * gy[tail].double()).sum(), list(leaves.values()))):
        g = getattr(got, k)
        ref.check(g[tail] if k in long else g, want, H + FROM if k in ("B", "C") else FROM, k)
