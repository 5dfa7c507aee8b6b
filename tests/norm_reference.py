"""The block's norms in 64 bits from their definitions; gradients by
differentiating the same lines (torch autograd in float64). Test
infrastructure: nothing of it runs in the library."""
import torch


def rms(x, eps):
    return x / torch.sqrt(x.square().mean(-1, keepdim=True) + eps)


def gated(x, z, w, eps):
    y = rms(x, eps) * w
    return y if z is None else y * z * torch.sigmoid(z)


def residual(x, r, w, post=None, scale=None, eps=1e-6):
    """y and h."""
    m = x if post is None else rms(x, eps) * post
    h = r + (m if scale is None else scale * m)
    return rms(h, eps) * w, h


def check(got, want, size, D=None, what=""):
    """|got - want| within the final rounding and the fp32 arithmetic behind it.

    A 16-bit output is rounded once: half a step of it. What is rounded comes
    out of a few roundings of the terms that `size` bounds (|terms|, of the
    shape of the output or broadcast to it) and of sums of D products of
    threads and shuffles (depth under 64): 96 2^-24 of size covers both; the
    gate's exponential and reciprocal add under 8 2^-24 of it."""
    got, want = got.detach().cpu(), want.detach().cpu()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    dtype, got = got.dtype, got.double()
    assert torch.isfinite(got).all(), f"{what}: not finite"
    tol = 104 * 2.0 ** -24 * size.detach().cpu().double() + torch.zeros_like(want)
    if dtype is torch.bfloat16:
        tol = tol + 2.0 ** -8 * want.abs() + 2.0 ** -133
    elif dtype is torch.float16:
        tol = tol + 2.0 ** -11 * want.abs() + 2.0 ** -24
    bad = (got - want).abs() > tol
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} off, worst "
                           f"{float(((got - want).abs() / tol.clamp(min=1e-300)).max()):.3g} of the tolerance")
