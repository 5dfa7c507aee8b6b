"""What the gated delta rule and the block's norms are measured on.

Together with the short convolution they are a whole layer, on the library's
[S,B,...] layout:

  delta          S_t = a_t S_{t-1} + u_t k_t^T,  u_t = b_t (v_t - a_t S_{t-1} k_t),  y_t = S_t q_t
                 per head, with a_t = exp(A softplus(delta_t + delta_bias)), b_t = sigmoid(beta_t),
                 q and k divided by their lengths, over whole prompts; its gradients
  delta_step     the same for one new token of every sequence, states kept in a
                 cache of slots and updated in place
  gated_norm     y = x / rms(x) weight silu(z), per head, behind the mixer; its gradients
  residual_norm  h = residual + scale (x / rms(x) post_weight),  y = h / rms(h) weight,
                 between a block and the next; its gradients

listed() and draw() give the cases, prepare() their inputs, run() one pass in
the plain form (own false) or through the library (own true), exact() the same
values from the definitions in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
DEVICE = "cuda"
EPS = 1e-6


# ------------------------------------------------------------------ cases
def _case(name, op, S, B, H, dtype, G=0, K=0, V=0, lengths=False, slots=False, carry=False, wide=False, post=False):
    """One case. H heads of V values (delta, gated_norm), or rows of H (residual_norm).
    `carry`: prompts continue from a state and hand one on (the backward then also
    takes the gradient of the state that was handed on). `lengths`: right-padded
    sequences of their own lengths. `slots`: the rows of a step are spread over a
    larger cache, one of them a padding row. `wide`: the residual stream is fp32.
    `post`: the branch has a norm and a scale of its own before the sum."""
    c = {"op": op, "S": S, "B": B, "H": H, "dtype": dtype, "G": G, "K": K, "V": V, "lengths": lengths, "slots": slots,
         "carry": carry, "wide": wide, "post": post}
    return dict(c, name=name) if name else c


def listed():
    return [
        # a short odd prompt of two sequences, few heads: latency counts
        _case("delta_s61_b2_h4_bf16", "delta", 61, 2, 4, "bf16", G=2, K=64, V=64),
        # the prompt of a serving batch: unequal lengths, from and to a state
        _case("delta_s4096_b8_h16_bf16", "delta", 4096, 8, 16, "bf16", G=16, K=128, V=128, lengths=True, carry=True),
        # one long document with few heads: the long axis is all there is to share out
        _case("delta_s65536_b1_h6_fp16", "delta", 65536, 1, 6, "fp16", G=6, K=64, V=64, carry=True),
        # the backward of a small training step, odd length, two value heads to a key head
        _case("delta_bwd_s509_b2_h6_fp16", "delta_bwd", 509, 2, 6, "fp16", G=3, K=64, V=64),
        # a training step's backward over 16 K tokens, value heads sharing q and k
        _case("delta_bwd_s2048_b8_h16_bf16", "delta_bwd", 2048, 8, 16, "bf16", G=8, K=128, V=128),
        # decoding one sequence
        _case("delta_step_b1_h16_bf16", "delta_step", 1, 1, 16, "bf16", G=16, K=128, V=128),
        # decoding a large batch out of a larger cache
        _case("delta_step_b256_h16_bf16", "delta_step", 1, 256, 16, "bf16", G=8, K=128, V=128, slots=True),
        # behind the mixer over a serving batch's prompts
        _case("gated_norm_s4096_b8_h16_bf16", "gated_norm", 4096, 8, 16, "bf16", V=128),
        # its gradients in a training step over 16 K tokens
        _case("gated_norm_bwd_s2048_b8_h32_fp16", "gated_norm_bwd", 2048, 8, 32, "fp16", V=64),
        # between two blocks while one sequence is decoded
        _case("residual_norm_b1_h2048_bf16", "residual_norm", 1, 1, 2048, "bf16", wide=True),
        # between two blocks over prompts of 64 K tokens
        _case("residual_norm_s8192_b8_h4096_bf16", "residual_norm", 8192, 8, 4096, "bf16", post=True),
        # its gradients in a training step over 16 K tokens, fp32 residual stream
        _case("residual_norm_bwd_s2048_b8_h2048_bf16", "residual_norm_bwd", 2048, 8, 2048, "bf16", wide=True, post=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("delta", "delta", "delta_bwd", "delta_bwd", "delta_step", "gated_norm", "gated_norm_bwd",
                     "residual_norm", "residual_norm_bwd"))
    dtype = rng.choice(("bf16", "bf16", "fp16"))
    if op.startswith("residual"):
        # a width as models have them, or any number
        H = rng.choice((384, 768, 1024, 1536, 2048, 2560, 4096)) if rng.random() < 0.7 else _log_int(rng, 50, 6000)
        S, B = _log_int(rng, 1, 8192), _log_int(rng, 1, 16)
        while S * B * H > 1 << 27:
            S = S // 2 + 1
        return _case("", op, S, B, H, dtype, wide=rng.random() < 0.5, post=rng.random() < 0.5)
    if op.startswith("gated"):
        H, V = rng.choice((4, 6, 8, 16, 32)), rng.choice((64, 128, 256)) if rng.random() < 0.7 else _log_int(rng, 16, 512)
        S, B = _log_int(rng, 1, 8192), _log_int(rng, 1, 16)
        while S * B * H * V > 1 << 26:
            S = S // 2 + 1
        return _case("", op, S, B, H, dtype, V=V)
    K, V = rng.choice(((64, 64), (128, 128), (128, 128), (64, 128), (96, 128), (40, 72)))
    G = rng.choice((1, 2, 3, 4, 6, 8, 16))
    H = G * rng.choice((1, 1, 2, 3))
    if op == "delta_step":
        B = _log_int(rng, 1, 256)
        while B * H > 4096:
            B = B // 2 + 1
        return _case("", op, 1, B, H, dtype, G, K, V, slots=rng.random() < 0.7)
    S, B = _log_int(rng, 1, 16384), _log_int(rng, 1, 16)
    most = {"delta": 1 << 19, "delta_bwd": 1 << 18}[op]      # tokens times heads
    while S * B * H > most:
        S, B = (S // 2 + 1, B) if rng.random() < 0.7 or B == 1 else (S, B // 2)
    return _case("", op, S, B, H, dtype, G, K, V, lengths=rng.random() < 0.4, carry=rng.random() < 0.5)


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)
    S, B, H, G, K, V = (case[k] for k in ("S", "B", "H", "G", "K", "V"))
    op, dt = case["op"], DTYPES[case["dtype"]]

    def normal(*shape, scale=1.0, dtype=dt):
        return (scale * torch.randn(shape, generator=g, device=DEVICE, dtype=torch.float32)).to(dtype)

    def uniform(*shape):
        return torch.rand(shape, generator=g, device=DEVICE, dtype=torch.float32)

    s = {"op": op}
    if op.startswith("gated"):
        s["x"], s["weight"] = normal(S, B, H, V), 1 + normal(V, scale=0.1)
        s["z"] = normal(S, B, 2 * H * V)[:, :, H * V:].view(S, B, H, V)      # half of a projection's output
        if op.endswith("bwd"):
            s["grad_y"] = normal(S, B, H, V)
        return s
    if op.startswith("residual"):
        stream = torch.float32 if case["wide"] else dt
        s["x"], s["residual"], s["weight"] = normal(S, B, H), normal(S, B, H, scale=2.0, dtype=stream), 1 + normal(H, scale=0.1)
        s["post_weight"] = 1 + normal(H, scale=0.1) if case["post"] else None
        s["scale"] = 0.5 + normal(H, scale=0.1, dtype=torch.float32) if case["post"] else None
        if op.endswith("bwd"):
            s["grad_y"], s["grad_h"] = normal(S, B, H), normal(S, B, H, dtype=stream)
        return s
    s.update(lengths=None, slots=None, state=None, grad_final_state=None, carry=case["carry"])
    # q, k, v leave the short convolution side by side, behind its silu
    n = 2 * G * K + H * V
    qkv = normal(S, B, n)
    qkv = torch.nn.functional.silu(qkv.float()).to(dt)
    s["q"], s["k"], s["v"] = (qkv[..., :G * K].view(S, B, G, K), qkv[..., G * K:2 * G * K].view(S, B, G, K),
                              qkv[..., 2 * G * K:].view(S, B, H, V))
    s["delta"], s["beta"] = normal(S, B, H, scale=0.5), normal(S, B, H)
    # the usual start: A from -1 to -16, steps from 0.001 to 0.1
    s["A"] = -(1 + 15 * uniform(H))
    step = torch.exp(uniform(H) * math.log(100.0) + math.log(1e-3))
    s["delta_bias"] = step + torch.log(-torch.expm1(-step))
    if op == "delta_step":
        rows = B
        if case["slots"]:
            rows = B + B // 4 + 1
            slots = torch.argsort(uniform(rows))[:B].to(torch.int32)
            if B > 3:
                slots[B // 2] = -1   # a padding row of the batch
            s["slots"] = slots
        for k in ("q", "k", "v", "delta", "beta"):
            s[k] = s[k][0]
        s["state"] = normal(rows, H, V, K, scale=0.1, dtype=torch.float32)
        return s
    if case["lengths"]:
        n = (S // 2 + (uniform(B) * (S - S // 2 + 1)).to(torch.int32)).clamp(max=S)
        if B > 2:
            n[1] = 0    # a row that is padding throughout
        s["lengths"] = n.to(torch.int32)
    if case["carry"]:
        s["state"] = normal(B, H, V, K, scale=0.1, dtype=torch.float32)
    if op == "delta_bwd":
        s["grad_y"] = normal(S, B, H, V)
        if case["carry"]:
            s["grad_final_state"] = normal(B, H, V, K, scale=0.1, dtype=torch.float32)
    return s


# ------------------------------------------------------------------ the plain forms
def _rms(x):
    return torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)


def _rms_grad(g, x, r):
    """The gradient of x r(x), r = _rms(x), for g."""
    return r * (g - x * r.square() * (g * x).mean(-1, keepdim=True))


def _plain_gated_norm(s):
    x, z = s["x"].float(), s["z"].float()
    return {"y": (x * _rms(x) * s["weight"].float() * z * torch.sigmoid(z)).to(s["x"].dtype)}


def _plain_gated_norm_bwd(s):
    dt = s["x"].dtype
    x, z, w, gy = s["x"].float(), s["z"].float(), s["weight"].float(), s["grad_y"].float()
    r, sig = _rms(x), torch.sigmoid(z)
    n, gn = x * r, gy * z * sig
    return {"x": _rms_grad(gn * w, x, r).to(dt), "z": (gy * n * w * sig * (1 + z * (1 - sig))).to(dt),
            "weight": (gn * n).sum((0, 1, 2)).to(dt)}


def _branch(s):
    """The branch's norm, what the residual stream gets of it, and that stream, in 32 bits."""
    x = s["x"].float()
    r = _rms(x)
    n = x * r if s["post_weight"] is not None else x
    m = n * s["post_weight"].float() if s["post_weight"] is not None else n
    h = s["residual"].float() + (m * s["scale"] if s["scale"] is not None else m)
    return x, r, n, m, h


def _plain_residual_norm(s):
    h = _branch(s)[-1]
    return {"y": (h * _rms(h) * s["weight"].float()).to(s["x"].dtype), "h": h.to(s["residual"].dtype)}


def _plain_residual_norm_bwd(s):
    x, r, n, m, h = _branch(s)
    dt, gy, rh = s["x"].dtype, s["grad_y"].float(), _rms(h)
    gh = s["grad_h"].float() + _rms_grad(gy * s["weight"].float(), h, rh)
    gm = gh * s["scale"] if s["scale"] is not None else gh
    gx = _rms_grad(gm * s["post_weight"].float(), x, r) if s["post_weight"] is not None else gm
    out = {"x": gx.to(dt), "residual": gh.to(s["residual"].dtype), "weight": (gy * h * rh).sum((0, 1)).to(dt)}
    if s["scale"] is not None:
        out["scale"] = (gh * m).sum((0, 1))
    if s["post_weight"] is not None:
        out["post_weight"] = (gm * n).sum((0, 1)).to(dt)
    return out


CHUNK = 64


def _inverse(L):
    """The inverse of unit lower triangular matrices: of the halves, then of the corner between them."""
    n = L.shape[-1]
    if n == 1:
        return L
    h = n // 2
    both = _inverse(torch.stack([L[..., :h, :h], L[..., h:, h:]]))
    out = torch.zeros_like(L)
    out[..., :h, :h], out[..., h:, h:] = both[0], both[1]
    out[..., h:, :h] = -both[1] @ (L[..., h:, :h] @ both[0])
    return out


def _gates(s):
    """raw and dt, the decays' logarithms and b, [S,B,H], and which tokens are there."""
    raw = s["delta"].float() + s["delta_bias"]
    dt = torch.where(raw > 20, raw, torch.log1p(torch.exp(torch.clamp(raw, max=20.0))))
    b = torch.sigmoid(s["beta"].float())
    return raw, dt, dt * s["A"], b


def _unit(t):
    """Vectors divided by their lengths, and what they were divided by."""
    n = torch.sqrt(t.square().sum(-1, keepdim=True) + EPS)
    return t / n, n


def _chunks(t):
    """[S,B,H,..] as [B,H,chunks,CHUNK,..], zeros behind the end."""
    S = t.shape[0]
    t = torch.cat([t, t.new_zeros(-S % CHUNK, *t.shape[1:])])
    return t.view(-1, CHUNK, *t.shape[1:]).permute(2, 3, 0, 1, *range(4, t.dim() + 1))


def _tokens(t, S):
    """_chunks the other way round."""
    return t.permute(2, 3, 0, 1, *range(4, t.dim())).flatten(0, 1)[:S]


def _delta_terms(s):
    H, K = s["v"].shape[2], s["q"].shape[3]
    raw, dt, la, b = _gates(s)
    q, k = (t.float().repeat_interleave(H // t.shape[2], dim=2) for t in (s["q"], s["k"]))
    (q, qn), (k, kn) = _unit(q), _unit(k)
    q, v = q * K ** -0.5, s["v"].float()
    live = None
    if s["lengths"] is not None:
        live = (torch.arange(q.shape[0], device=q.device)[:, None] < s["lengths"][None, :])[:, :, None]
        la, b = torch.where(live, la, 0.0), torch.where(live, b, 0.0)
        q, k, v = (torch.where(live[..., None], t, 0.0) for t in (q, k, v))
    qc, kc, vc, lc, bc = (_chunks(t) for t in (q, k, v, la, b))
    c = lc.cumsum(-1)
    at = torch.arange(CHUNK, device=q.device)
    D = torch.exp(torch.where(at[:, None] >= at, c[..., :, None] - c[..., None, :], -math.inf))
    kk, qk = kc @ kc.mT, qc @ kc.mT
    L = torch.where(at[:, None] > at, bc[..., None] * D * kk, 0.0)
    T = _inverse(L + torch.eye(CHUNK, device=q.device))
    e = torch.exp(c)[..., None]
    last = torch.exp(c[..., -1:] - c)[..., None]
    W = T @ (bc[..., None] * e * kc)
    U0 = T @ (bc[..., None] * vc)
    # the recurrence itself: one chunk after the other
    first = s["state"].mT if s["state"] is not None else q.new_zeros(*kc.shape[:2], K, v.shape[3])
    states, U, end, kl = [first], [], e[..., -1:, :], last * kc
    for i in range(kc.shape[2]):
        u = U0[:, :, i] - W[:, :, i] @ states[-1]
        U.append(u)
        states.append(end[:, :, i] * states[-1] + kl[:, :, i].mT @ u)
    final = states.pop()
    return dict(raw=raw, dt=dt, qn=qn, kn=kn, live=live, q=qc, k=kc, v=vc, c=c, b=bc, D=D, kk=kk, qk=qk, T=T, e=e, end=end,
                kl=kl, W=W, S=torch.stack(states, 2), U=torch.stack(U, 2), final=final, la=la)


def _plain_delta(s):
    t = _delta_terms(s)
    y = (t["e"] * t["q"]) @ t["S"] + (t["qk"] * t["D"]) @ t["U"]
    out = {"y": _tokens(y, s["q"].shape[0]).to(s["v"].dtype)}
    if s["carry"]:
        out["state"] = t["final"].mT.contiguous()
    return out


def _unit_grad(g, unit, n, heads):
    """The gradient of t for g of _unit(t), summed over the value heads that share it."""
    g = (g - unit * (g * unit).sum(-1, keepdim=True)) / n
    return g.view(*g.shape[:2], heads, -1, g.shape[3]).sum(3)


def _plain_delta_bwd(s):
    t = _delta_terms(s)
    S, B, H = s["beta"].shape
    G, K, out_t = s["q"].shape[2], s["q"].shape[3], s["v"].dtype
    q, k, D, U, S0, e, b, kl, end, T = (t[x] for x in ("q", "k", "D", "U", "S", "e", "b", "kl", "end", "T"))
    gy = s["grad_y"].float()
    if t["live"] is not None:
        gy = torch.where(t["live"][..., None], gy, 0.0)
    gy = _chunks(gy)
    P = t["qk"] * D
    # the states' gradients run backwards, one chunk after the other
    gU0 = P.mT @ gy
    add = (e * q).mT @ gy - t["W"].mT @ gU0
    last = s["grad_final_state"].mT if s["grad_final_state"] is not None else torch.zeros_like(S0[:, :, 0])
    grads = [last]
    for i in reversed(range(q.shape[2])):
        grads.append(end[:, :, i] * grads[-1] + add[:, :, i] - t["W"][:, :, i].mT @ (kl[:, :, i] @ grads[-1]))
    first = grads.pop()
    GS = torch.stack(grads[::-1], 2)
    gU = gU0 + kl @ GS
    gR = T.mT @ gU
    gP = gy @ U.mT
    at = torch.arange(CHUNK, device=q.device)
    gL = torch.where(at[:, None] > at, -(gR @ U.mT), 0.0)
    gPD, gLD = gP * D, gL * D
    gq_state = (gy @ S0.mT) * e
    gk_state, gk_end = -(gR @ S0.mT) * b[..., None] * e, (U @ GS.mT) * torch.exp(t["c"][..., -1:] - t["c"])[..., None]
    gLb = gLD * b[..., None]
    gq = gq_state + gPD @ k
    gk = gPD.mT @ q + gLb @ k + gLb.mT @ k + gk_state + gk_end
    gv = b[..., None] * gR
    state_k = (gk_state * k).sum(-1)                     # b times the gradient of b in front of the state's part
    gb = (gR * (t["v"] - e * (k @ S0))).sum(-1) + (gLD * t["kk"]).sum(-1)
    E = gPD * t["qk"] + gLb * t["kk"]
    ends = (gk_end * k).sum(-1)
    gc = E.sum(-1) - E.sum(-2) + (gq_state * q).sum(-1) + state_k - ends
    gc[..., -1] += ends.sum(-1) + (GS * S0).sum((-1, -2)) * end[..., 0, 0]
    gla = gc.flip(-1).cumsum(-1).flip(-1)
    gq, gk, gv, gb, gla, q, k = (_tokens(x, S) for x in (gq, gk, gv, gb, gla, q, k))
    scale = K ** -0.5
    sig = torch.sigmoid(s["beta"].float())
    graw = gla * s["A"] * torch.sigmoid(t["raw"])
    gbeta = gb * sig * (1 - sig)
    gA = gla * t["dt"]
    if t["live"] is not None:
        graw, gbeta, gA = (torch.where(t["live"], x, 0.0) for x in (graw, gbeta, gA))
    out = {"q": _unit_grad(gq * scale, q / scale, t["qn"], G).to(out_t), "k": _unit_grad(gk, k, t["kn"], G).to(out_t),
           "v": gv.to(out_t), "delta": graw.to(out_t), "beta": gbeta.to(out_t), "A": gA.sum((0, 1)),
           "delta_bias": graw.sum((0, 1))}
    if s["carry"]:
        out["state"] = first.mT.contiguous()
    return out


def _to_slots(cache, slots, new):
    """Writes row b of `new` to cache[slots[b]], negative slots to nowhere."""
    rows, B = cache.shape[0], new.shape[0]
    row_of = torch.full((rows + 1,), -1, device=slots.device, dtype=torch.long)
    row_of[torch.where(slots >= 0, slots, rows).long()] = torch.arange(B, device=slots.device)
    row_of = row_of[:rows].view(rows, *[1] * (new.dim() - 1))
    cache.copy_(torch.where(row_of >= 0, new[row_of.flatten().clamp(min=0)], cache))


def _plain_delta_step(s):
    H, K = s["v"].shape[1], s["q"].shape[2]
    _, _, la, b = _gates(s)
    q, k = (_unit(t.float().repeat_interleave(H // t.shape[1], dim=1))[0] for t in (s["q"], s["k"]))
    old = s["state"] if s["slots"] is None else s["state"][s["slots"].clamp(min=0).long()]
    new = old * torch.exp(la)[..., None, None]
    u = b[..., None] * (s["v"].float() - (new * k[..., None, :]).sum(-1))
    new = new + u[..., None] * k[..., None, :]
    y = (new * (q * K ** -0.5)[..., None, :]).sum(-1)
    if s["slots"] is None:
        s["state"].copy_(new)
    else:
        y = torch.where((s["slots"] >= 0)[:, None, None], y, 0.0)
        _to_slots(s["state"], s["slots"], new)
    return {"y": y.to(s["v"].dtype), "state": s["state"]}


PLAIN = {"delta": _plain_delta, "delta_bwd": _plain_delta_bwd, "delta_step": _plain_delta_step,
         "gated_norm": _plain_gated_norm, "gated_norm_bwd": _plain_gated_norm_bwd,
         "residual_norm": _plain_residual_norm, "residual_norm_bwd": _plain_residual_norm_bwd}


# ------------------------------------------------------------------ the library
def _own(s):
    import causal_conv_backward_gb300 as mcc
    op = s["op"]
    if op == "gated_norm":
        return {"y": mcc.gated_norm(s["x"], s["z"], s["weight"], eps=EPS)}
    if op == "gated_norm_bwd":
        return mcc.gated_norm_backward(s["grad_y"], s["x"], s["z"], s["weight"], eps=EPS)._asdict()
    if op == "residual_norm":
        y, h = mcc.residual_norm(s["x"], s["residual"], s["weight"], post_weight=s["post_weight"], scale=s["scale"], eps=EPS)
        return {"y": y, "h": h}
    if op == "residual_norm_bwd":
        r = mcc.residual_norm_backward(s["grad_y"], s["grad_h"], s["x"], s["residual"], s["weight"],
                                       post_weight=s["post_weight"], scale=s["scale"], eps=EPS)
        return {k: v for k, v in r._asdict().items() if v is not None}
    forms = dict(delta_softplus=True, beta_sigmoid=True, qk_norm=True)
    if op == "delta_step":
        y = mcc.gated_delta_step(s["q"], s["k"], s["v"], s["delta"], s["beta"], s["state"], s["A"], s["delta_bias"],
                                 slots=s["slots"], **forms)
        return {"y": y, "state": s["state"]}
    if op == "delta":
        r = mcc.gated_delta(s["q"], s["k"], s["v"], s["delta"], s["beta"], s["A"], s["delta_bias"], lengths=s["lengths"],
                            state=s["state"], return_state=s["carry"], **forms)
        return {"y": r[0], "state": r[1]} if s["carry"] else {"y": r}
    r = mcc.gated_delta_backward(s["grad_y"], s["q"], s["k"], s["v"], s["delta"], s["beta"], s["A"], s["delta_bias"],
                                 lengths=s["lengths"], state=s["state"], grad_final_state=s["grad_final_state"], **forms)
    return {k: v for k, v in r._asdict().items() if v is not None}


def run(state):
    return _own(state) if own else PLAIN[state["op"]](state)


# ------------------------------------------------------------------ work
def work(case):
    S, B, H, G, K, V = (case[k] for k in ("S", "B", "H", "G", "K", "V"))
    op, t = case["op"], S * B
    if op.startswith("gated"):
        e = t * H * V
        if op == "gated_norm":                  # x, z in, y out
            return {"bytes": 2 * 3 * e + 2 * V, "flops": 10 * e}
        return {"bytes": 2 * 5 * e + 4 * V, "flops": 25 * e}
    if op.startswith("residual"):
        e, r, w = t * H, 4 if case["wide"] else 2, H * (8 if case["post"] else 2)
        if op == "residual_norm":               # x, residual in, h, y out
            return {"bytes": e * (4 + 2 * r) + w, "flops": 10 * e}
        return {"bytes": e * (6 + 3 * r) + 2 * w, "flops": 30 * e}
    state, qkv, gates = B * H * V * K * 4, 2 * G * K + H * V, 2 * H
    if op == "delta_step":                      # the state in and out
        return {"bytes": 2 * state + 2 * B * (qkv + gates + H * V) + 8 * H, "flops": 8 * B * H * V * K}
    # per token and head, in chunks of C: k.k and q.k (half of C each), the state's three products, two triangular ones
    live = 1.0
    if case["lengths"]:                         # between half and all of S each, one of more than two sequences empty
        live = 0.75 * ((B - 1) / B if B > 2 else 1.0)
    flops = live * t * H * (6 * K * V + 2 * CHUNK * (K + V)) + 0.0
    carried = 2 * state if case["carry"] else 0
    if op == "delta":                           # q, k, v and the gates in, y out
        return {"bytes": 2 * t * (live * (qkv + gates) + H * V) + carried + 8 * H, "flops": flops}
    # grad_y too, and the gradients out
    return {"bytes": 2 * t * (live * (qkv + gates + H * V) + qkv + gates) + 1.5 * carried + 16 * H, "flops": 3.5 * flops}


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    d = {k: v.double() if isinstance(v, torch.Tensor) and v.is_floating_point() else v for k, v in s.items()}
    op = case["op"]
    if op.startswith(("gated", "residual")):
        return _exact_norm(op, d)
    if op == "delta_step":
        return _exact_step(d)
    return _exact_delta(case, d)


def _exact_norm(op, d):
    """Values from the definition, gradients by differentiating it."""
    leaves = {k: v.requires_grad_() for k, v in d.items() if isinstance(v, torch.Tensor) and not k.startswith("grad")}
    x = d["x"]

    def norm(t, w):
        return t / torch.sqrt((t * t).sum(-1, keepdim=True) / t.shape[-1] + EPS) * w

    if op.startswith("gated"):
        out = {"y": norm(x, d["weight"]) * d["z"] / (1 + torch.exp(-d["z"]))}
    else:
        m = norm(x, d["post_weight"]) if d["post_weight"] is not None else x
        h = d["residual"] + (d["scale"] * m if d["scale"] is not None else m)
        out = {"y": norm(h, d["weight"]), "h": h}
    if not op.endswith("bwd"):
        return {k: v.detach() for k, v in out.items()}
    loss = sum((v * d["grad_" + k]).sum() for k, v in out.items())
    return dict(zip(leaves, torch.autograd.grad(loss, list(leaves.values()))))


def _exact_gates(d):
    """raw, dt, a, b and the divided q and k, for every value head."""
    raw = d["delta"] + d["delta_bias"]
    dt = torch.logaddexp(raw, torch.zeros_like(raw))
    H = d["v"].shape[-2]
    lengths = [torch.sqrt((d[x] ** 2).sum(-1, keepdim=True) + EPS) for x in ("q", "k")]
    q, k = (torch.repeat_interleave(d[x] / n, H // d[x].shape[-2], dim=-2) for x, n in zip(("q", "k"), lengths))
    return raw, dt, torch.exp(d["A"] * dt), 1 / (1 + torch.exp(-d["beta"])), q, k, lengths


def _exact_step(d):
    _, _, a, b, q, k, _ = _exact_gates(d)
    cache, y = d["state"].clone(), torch.zeros_like(d["v"])
    rows = range(y.shape[0]) if d["slots"] is None else d["slots"].tolist()
    for n, r in enumerate(rows):
        if r >= 0:
            h = cache[r] * a[n].view(-1, 1, 1)
            u = (d["v"][n] - torch.einsum("hvk,hk->hv", h, k[n])) * b[n].view(-1, 1)
            cache[r] = h + torch.einsum("hv,hk->hvk", u, k[n])
            y[n] = torch.einsum("hvk,hk->hv", cache[r], q[n]) / q.shape[-1] ** 0.5
    return {"y": y, "state": cache}


def _exact_delta(case, d):
    """The recurrence itself, one token after the other; states are kept for every BLOCK tokens and made again in between."""
    S, B, H, G, K, V = (case[x] for x in ("S", "B", "H", "G", "K", "V"))
    raw, dt, a, b, q, k, (qn, kn) = _exact_gates(d)
    dev, scale, bwd, block = q.device, K ** -0.5, case["op"] == "delta_bwd", 64
    n = d["lengths"].long() if d["lengths"] is not None else torch.full((B,), S, device=dev)
    live = (torch.arange(S, device=dev).view(S, 1) < n).double().view(S, B, 1)
    a, b, v = a * live + (1 - live), b * live, d["v"]
    state = d["state"] if d["state"] is not None else torch.zeros(B, H, V, K, dtype=torch.float64, device=dev)
    y, kept = torch.empty(S, B, H, V, dtype=torch.float64, device=dev), []

    def token(state, t):
        h = state * a[t].view(B, H, 1, 1)
        miss = v[t] - (h @ k[t].unsqueeze(-1)).squeeze(-1)
        return h, miss, torch.addcmul(h, (miss * b[t].unsqueeze(-1)).unsqueeze(-1), k[t].unsqueeze(-2))

    for t in range(S):
        if bwd and t % block == 0:
            kept.append(state)
        state = token(state, t)[2]
        if not bwd:
            y[t] = (state @ q[t].unsqueeze(-1)).squeeze(-1)
    if not bwd:
        out = {"y": y * scale * live.unsqueeze(-1)}
        if case["carry"]:
            out["state"] = state
        return out
    g = d["grad_final_state"] if d["grad_final_state"] is not None else torch.zeros_like(state)
    gy = d["grad_y"] * live.unsqueeze(-1) * scale
    gq, gk, gv, gb, gl = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v), torch.empty_like(b), torch.empty_like(b)
    for i in reversed(range(len(kept))):
        steps, state = [], kept[i]
        for t in range(i * block, min(S, (i + 1) * block)):
            h, miss, state = token(state, t)
            steps.append((t, h, miss, state))
        for t, h, miss, after in reversed(steps):
            g = torch.addcmul(g, gy[t].unsqueeze(-1), q[t].unsqueeze(-2))
            gq[t] = (gy[t].unsqueeze(-2) @ after).squeeze(-2)
            gu = (g @ k[t].unsqueeze(-1)).squeeze(-1)
            gm = gu * b[t].unsqueeze(-1)                   # of v - h k
            gb[t], gv[t] = (gu * miss).sum(-1), gm
            gk[t] = ((miss * b[t].unsqueeze(-1)).unsqueeze(-2) @ g - gm.unsqueeze(-2) @ h).squeeze(-2)
            gh = torch.addcmul(g, gm.unsqueeze(-1), k[t].unsqueeze(-2), value=-1)
            gl[t] = (gh * h).sum((-1, -2))
            g = gh * a[t].view(B, H, 1, 1)
    gl, gb = gl * live, gb * live
    sig = 1 / (1 + torch.exp(-d["beta"]))

    def through(gx, unit, length):                          # of x for gx of x / |x|, over the heads that share it
        gx = gx - unit * torch.einsum("sbhk,sbhk->sbh", gx, unit).unsqueeze(-1)
        return gx.reshape(S, B, G, H // G, K).sum(3) / length

    out = {"q": through(gq, q, qn), "k": through(gk * live.unsqueeze(-1), k, kn), "v": gv, "beta": gb * sig * (1 - sig),
           "A": (gl * dt).sum((0, 1)), "delta": gl * d["A"] / (1 + torch.exp(-raw))}
    out["delta_bias"] = out["delta"].sum((0, 1))
    if case["carry"]:
        out["state"] = g
    return out
