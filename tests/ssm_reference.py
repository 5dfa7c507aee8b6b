"""The short convolution and the selective scan in 64 bits, token by token, from
their definitions; gradients by differentiating the same lines (torch autograd
in float64, CPU). Test infrastructure: nothing of it runs in the library."""
import torch


def rounding(dtype):
    """Unit roundoff of a 16-bit type, and its smallest step."""
    return (2.0 ** -8, 2.0 ** -133) if dtype is torch.bfloat16 else (2.0 ** -11, 2.0 ** -24)


def check(got, want, terms, what=""):
    """|got - want| within the final rounding and the fp32 sums behind it.

    A 16-bit output is rounded once: u |want| (or half a subnormal step). What
    is rounded is an fp32 sum of `terms` products (tokens, states, channels):
    its error is at most depth 2^-24 sum|products|, the depth of the sums kept
    under 16 by partial sums plus the few roundings of each product, and the
    sum of |products| about sqrt(terms) times a typical value of the result
    where signs are mixed, hence 16 2^-24 (8 + sqrt(terms)) max|want|."""
    dtype = got.dtype
    got, want = got.detach().cpu().double(), want.detach().cpu().double()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    assert torch.isfinite(got).all(), f"{what}: not finite"
    if not want.numel():
        return
    fp32 = 16 * 2.0 ** -24 * (8 + terms ** 0.5) * want.abs().max()
    tol = fp32 + torch.zeros_like(want)
    if dtype is not torch.float32:
        u, step = rounding(dtype)
        tol = tol + u * want.abs() + step
    bad = (got - want).abs() > tol
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} off, worst "
                           f"{float(((got - want).abs() / tol.clamp(min=1e-300)).max()):.3g} of the tolerance")


def _len(lengths, b, S):
    return S if lengths is None else max(0, min(S, int(lengths[b])))


def conv(x, w, bias=None, silu=True, lengths=None, state=None):
    """y [S,B,H] and the final window [B,W-1,H]."""
    S, B, H = x.shape
    W = w.shape[0]
    ys, finals = [], []
    for b in range(B):
        n = _len(lengths, b, S)
        past = state[b] if state is not None else torch.zeros(W - 1, H, dtype=x.dtype)
        rows = torch.cat([past, x[:n, b]])
        out = []
        for t in range(n):
            pre = (rows[t:t + W] * w).sum(0)
            if bias is not None:
                pre = pre + bias
            out.append(pre * torch.sigmoid(pre) if silu else pre)
        y = torch.stack(out) if n else torch.zeros(0, H, dtype=x.dtype)
        ys.append(torch.cat([y, torch.zeros(S - n, H, dtype=x.dtype)]))
        finals.append(rows[n:n + W - 1])
    return torch.stack(ys, 1), torch.stack(finals)


def scan(u, delta, A, B, C, D=None, z=None, delta_bias=None, softplus=True, lengths=None, state=None):
    """y [S,B,H] and the final state [B,H,N]."""
    S, nb, H = u.shape
    G, N = B.shape[2], B.shape[3]
    ys, finals = [], []
    for b in range(nb):
        n = _len(lengths, b, S)
        h = state[b] if state is not None else torch.zeros(H, N, dtype=u.dtype)
        out = []
        for t in range(n):
            dt = delta[t, b] if delta_bias is None else delta[t, b] + delta_bias
            if softplus:
                dt = torch.logaddexp(dt, torch.zeros_like(dt))
            Bt, Ct = (m[t, b].repeat_interleave(H // G, 0) for m in (B, C))
            h = torch.exp(dt[:, None] * A) * h + (dt * u[t, b])[:, None] * Bt
            y = (h * Ct).sum(1)
            if D is not None:
                y = y + D * u[t, b]
            if z is not None:
                y = y * z[t, b] * torch.sigmoid(z[t, b])
            out.append(y)
        y = torch.stack(out) if n else torch.zeros(0, H, dtype=u.dtype)
        ys.append(torch.cat([y, torch.zeros(S - n, H, dtype=u.dtype)]))
        finals.append(h)
    return torch.stack(ys, 1), torch.stack(finals)


def to64(t, grad=False):
    """A float64 CPU copy (None stays None)."""
    if t is None:
        return None
    c = t.detach().cpu().double()
    return c.requires_grad_(grad)


def differences(loss, leaf, got, eps=1e-4, seed=0):
    """(central difference of `loss` along a random direction of `leaf`,
    <got, direction>, sum |got direction|): the last scales what rounding the
    gradient's values may cost."""
    g = torch.Generator().manual_seed(seed)
    d = torch.randn(leaf.shape, generator=g, dtype=torch.float64)
    with torch.no_grad():
        keep = leaf.data.clone()
        leaf.data = keep + eps * d
        up = float(loss())
        leaf.data = keep - eps * d
        down = float(loss())
        leaf.data = keep
    got = got.detach().cpu().double()
    return (up - down) / (2 * eps), float((got * d).sum()), float((got * d).abs().sum())
