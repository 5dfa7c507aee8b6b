"""The gated delta rule in 64 bits, token by token, from its definition;
gradients by differentiating the same lines (torch autograd in float64, CPU).
Test infrastructure: nothing of it runs in the library."""
import torch

EPS = 1e-6


def unit(t):
    return t / torch.sqrt(t.square().sum(-1, keepdim=True) + EPS)


def delta_rule(q, k, v, delta, beta, A=None, bias=None, softplus=True, sigmoid=True, norm=True, scale=None, lengths=None,
               state=None):
    """y [S,B,H,V] and the final state [B,H,V,K]."""
    S, B, G, K = q.shape
    H, V = v.shape[2:]
    scale = K ** -0.5 if scale is None else scale
    if norm:
        q, k = unit(q), unit(k)
    q, k = (t.repeat_interleave(H // G, 2) for t in (q, k))
    if delta is not None:
        dt = delta if bias is None else delta + bias
        if softplus:
            dt = torch.logaddexp(dt, torch.zeros_like(dt))
        a = torch.exp(dt * A)
    else:
        a = torch.ones_like(beta)
    b = torch.sigmoid(beta) if sigmoid else beta
    ys, finals = [], []
    for n in range(B):
        length = S if lengths is None else max(0, min(S, int(lengths[n])))
        h = state[n] if state is not None else torch.zeros(H, V, K, dtype=q.dtype)
        out = []
        for t in range(length):
            h = h * a[t, n][:, None, None]
            u = b[t, n][:, None] * (v[t, n] - (h * k[t, n][:, None]).sum(-1))
            h = h + u[:, :, None] * k[t, n][:, None]
            out.append((h * q[t, n][:, None]).sum(-1) * scale)
        y = torch.stack(out) if out else torch.zeros(0, H, V, dtype=q.dtype)
        ys.append(torch.cat([y, torch.zeros(S - length, H, V, dtype=q.dtype)]))
        finals.append(h)
    return torch.stack(ys, 1), torch.stack(finals)
