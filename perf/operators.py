"""What the short convolution and the selective scan are measured on.

The pair is the sequence mixer of a selective state space block, on the
library's [S,B,H] layout:

  conv       y = silu(bias + causal depthwise conv(x, weight)), with a carried
             window of W-1 rows, over whole prompts; its gradients
  conv_step  the same for one new token of every sequence, the windows kept in
             a cache of slots and updated in place
  scan       h_t = exp(dt_t A) h_{t-1} + dt_t B_t u_t,
             y_t = (C_t . h_t + D u_t) silu(z_t),  dt_t = softplus(delta_t + delta_bias),
             over whole prompts; its gradients
  scan_step  the same for one new token of every sequence, states kept in a
             cache of slots and updated in place

listed() and draw() give the cases, prepare() their inputs, run() one pass in
the plain form (own false) or through the library (own true), exact() the same
values from the definitions in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
DEVICE = "cuda"


# ------------------------------------------------------------------ cases
def _case(name, op, S, B, H, dtype, W=0, N=0, G=1, lengths=False, slots=False, carry=False):
    """One case. `carry`: prompts continue from a state and hand one on (the
    backward then also takes the gradient of the state that was handed on).
    `lengths`: right-padded sequences of their own lengths. `slots`: the rows
    of a step are spread over a larger cache, one of them a padding row."""
    c = {"op": op, "S": S, "B": B, "H": H, "dtype": dtype, "W": W, "N": N, "G": G, "lengths": lengths,
         "slots": slots, "carry": carry}
    return dict(c, name=name) if name else c


def listed():
    return [
        # a short prompt of two sequences: a few microseconds, latency counts
        _case("conv_s61_b2_h384_bf16", "conv", 61, 2, 384, "bf16", W=4),
        # the prompt of a serving batch: sequences of unequal lengths, x the first
        # half of a projection's output, the window handed on to decoding
        _case("conv_s4096_b8_h2048_fp16", "conv", 4096, 8, 2048, "fp16", W=4, lengths=True, carry=True),
        # a training step's backward over 64 K tokens
        _case("conv_bwd_s8192_b8_h4096_bf16", "conv_bwd", 8192, 8, 4096, "bf16", W=4),
        # decoding one sequence
        _case("conv_step_b1_h2048_bf16", "conv_step", 1, 1, 2048, "bf16", W=4),
        # decoding a large batch out of a larger cache
        _case("conv_step_b512_h4096_bf16", "conv_step", 1, 512, 4096, "bf16", W=4, slots=True),
        # a short odd prompt of two sequences: latency counts
        _case("scan_s61_b2_h384_bf16", "scan", 61, 2, 384, "bf16", N=16),
        # the prompt of a serving batch, unequal lengths, from and to a state
        _case("scan_s4096_b8_h2048_bf16", "scan", 4096, 8, 2048, "bf16", N=16, lengths=True, carry=True),
        # one long document with few channels: the long axis is all there is to share out
        _case("scan_s131072_b1_h384_bf16", "scan", 131072, 1, 384, "bf16", N=16, carry=True),
        # the backward of a small training step, odd length, two groups sharing B and C
        _case("scan_bwd_s509_b2_h768_fp16", "scan_bwd", 509, 2, 768, "fp16", N=16, G=2),
        # a training step's backward over 16 K tokens
        _case("scan_bwd_s2048_b8_h2048_bf16", "scan_bwd", 2048, 8, 2048, "bf16", N=16),
        # decoding one sequence
        _case("scan_step_b1_h2048_bf16", "scan_step", 1, 1, 2048, "bf16", N=16),
        # decoding a large batch out of a larger cache
        _case("scan_step_b256_h4096_bf16", "scan_step", 1, 256, 4096, "bf16", N=16, slots=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("conv", "conv_bwd", "conv_step", "scan", "scan", "scan_bwd", "scan_bwd", "scan_step"))
    dtype = rng.choice(("bf16", "bf16", "fp16"))
    # channels: a width as models have them, or any number (one rank's odd share, a pruned layer)
    H = rng.choice((384, 512, 640, 768, 1024, 1280, 1536, 2048, 2560, 4096)) if rng.random() < 0.7 else _log_int(rng, 100, 2900)
    W = rng.choice((2, 3, 4, 4, 5, 8)) if op.startswith("conv") else 0
    N = rng.choice((16, 16, 16, 8, 32, 12)) if op.startswith("scan") else 0
    G = rng.choice((1, 1, 2, 4)) if op.startswith("scan") else 1
    H -= H % G
    if op.endswith("step"):
        return _case("", op, 1, _log_int(rng, 1, 256), H, dtype, W, N, G, slots=rng.random() < 0.7)
    S, B = _log_int(rng, 1, 32768), _log_int(rng, 1, 16)
    most = {"conv": 1 << 27, "conv_bwd": 1 << 27, "scan": 1 << 25, "scan_bwd": 1 << 24}[op]
    while S * B * H * max(N, 16) > 16 * most:
        S, B = (S // 2 + 1, B) if rng.random() < 0.7 or B == 1 else (S, B // 2)
    return _case("", op, S, B, H, dtype, W, N, G, lengths=rng.random() < 0.4, carry=rng.random() < 0.5)


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)
    S, B, H, W, N, G = (case[k] for k in ("S", "B", "H", "W", "N", "G"))
    op, dt = case["op"], DTYPES[case["dtype"]]

    def normal(*shape, scale=1.0, dtype=dt):
        return (scale * torch.randn(shape, generator=g, device=DEVICE, dtype=torch.float32)).to(dtype)

    def uniform(*shape):
        return torch.rand(shape, generator=g, device=DEVICE, dtype=torch.float32)

    s = {"op": op, "lengths": None, "slots": None, "state": None, "grad_final_state": None}
    if case["lengths"]:
        n = S // 2 + (uniform(B) * (S - S // 2 + 1)).to(torch.int32)
        n = n.clamp(max=S)
        if B > 2:
            n[1] = 0    # a row that is padding throughout
        s["lengths"] = n.to(torch.int32)
    rows = B
    if case["slots"]:
        rows = B + B // 4 + 1
        slots = torch.argsort(uniform(rows))[:B].to(torch.int32)
        if B > 3:
            slots[B // 2] = -1   # a padding row of the batch
        s["slots"] = slots
    if op.startswith("conv"):
        s["weight"] = ((2 * uniform(W, H) - 1) / math.sqrt(W)).to(dt)
        s["bias"] = normal(H, scale=0.2)
        if op == "conv_step":
            s["x"] = normal(B, H)
            s["state"] = normal(rows, W - 1, H)
            return s
        # x is the first half of the input projection's output
        s["x"] = normal(S, B, 2 * H)[:, :, :H]
        if case["carry"]:
            s["state"] = normal(B, W - 1, H)
        s["carry"] = case["carry"]
        if op == "conv_bwd":
            s["grad_y"] = normal(S, B, H)
            if case["carry"]:
                s["grad_final_state"] = normal(B, W - 1, H)
        return s
    # the usual start of such a layer: A near -1..-N, steps from 0.001 to 0.1
    s["A"] = -torch.arange(1, N + 1, device=DEVICE, dtype=torch.float32) * torch.exp(normal(H, N, scale=0.1, dtype=torch.float32))
    s["D"] = 1 + normal(H, scale=0.1, dtype=torch.float32)
    step = torch.exp(uniform(H) * math.log(100.0) + math.log(1e-3))
    s["delta_bias"] = step + torch.log(-torch.expm1(-step))
    if op == "scan_step":
        s["u"], s["delta"] = normal(B, H), normal(B, H, scale=0.5)
        s["z"] = normal(B, 2 * H)[:, H:]
        bc = normal(B, 2 * G * N)
        s["B"], s["C"] = bc[:, :G * N].view(B, G, N), bc[:, G * N:].view(B, G, N)
        s["state"] = normal(rows, H, N, scale=0.3, dtype=torch.float32)
        return s
    s["u"], s["delta"] = normal(S, B, H), normal(S, B, H, scale=0.5)
    s["z"] = normal(S, B, 2 * H)[:, :, H:]           # the other half of the input projection's output
    bc = normal(S, B, 2 * G * N)                     # B and C come out of one projection
    s["B"], s["C"] = bc[:, :, :G * N].view(S, B, G, N), bc[:, :, G * N:].view(S, B, G, N)
    if case["carry"]:
        s["state"] = normal(B, H, N, scale=0.3, dtype=torch.float32)
    s["carry"] = case["carry"]
    if op == "scan_bwd":
        s["grad_y"] = normal(S, B, H)
        if case["carry"]:
            s["grad_final_state"] = normal(B, H, N, scale=0.3, dtype=torch.float32)
    return s


# ------------------------------------------------------------------ the plain forms
def _valid(s, S):
    """[S,B,1] bool, true before a sequence's length; None where all are."""
    if s["lengths"] is None:
        return None
    return (torch.arange(S, device=s["lengths"].device)[:, None] < s["lengths"][None, :])[:, :, None]


def _padded(s):
    """x in 32 bits behind its W-1 rows of state (zeros without one)."""
    x, W = s["x"].float(), s["weight"].shape[0]
    front = s["state"].float().transpose(0, 1) if s["state"] is not None else x.new_zeros(W - 1, *x.shape[1:])
    return torch.cat([front, x])


def _final_rows(s, S, W):
    """Row numbers [W-1,B] of the padded x that are the final window."""
    B = s["x"].shape[1]
    n = s["lengths"].long() if s["lengths"] is not None else torch.full((B,), S, device=s["x"].device)
    return n[None, :] + torch.arange(W - 1, device=n.device)[:, None]


def _plain_conv(s):
    xp, w, valid = _padded(s), s["weight"].float(), _valid(s, s["x"].shape[0])
    S, W = s["x"].shape[0], w.shape[0]
    pre = sum(xp[k:k + S] * w[k] for k in range(W)) + s["bias"].float()
    y = pre * torch.sigmoid(pre)
    if valid is not None:
        y = torch.where(valid, y, 0.0)
    out = {"y": y.to(s["x"].dtype)}
    if s["carry"]:
        rows = _final_rows(s, S, W)
        out["state"] = torch.gather(xp, 0, rows[:, :, None].expand(-1, -1, xp.shape[2])).transpose(0, 1).to(s["x"].dtype)
    return out


def _plain_conv_bwd(s):
    xp, w, valid = _padded(s), s["weight"].float(), _valid(s, s["x"].shape[0])
    S, W, dt = s["x"].shape[0], w.shape[0], s["x"].dtype
    pre = sum(xp[k:k + S] * w[k] for k in range(W)) + s["bias"].float()
    sig = torch.sigmoid(pre)
    dpre = s["grad_y"].float() * sig * (1 + pre * (1 - sig))
    if valid is not None:
        dpre = torch.where(valid, dpre, 0.0)
    dxp = torch.zeros_like(xp)
    for k in range(W):
        dxp[k:k + S] += dpre * w[k]
    if s["grad_final_state"] is not None:
        rows = _final_rows(s, S, W)
        dxp.scatter_add_(0, rows[:, :, None].expand(-1, -1, xp.shape[2]), s["grad_final_state"].float().transpose(0, 1))
    out = {"x": dxp[W - 1:].to(dt), "weight": torch.stack([(dpre * xp[k:k + S]).sum((0, 1)) for k in range(W)]).to(dt),
           "bias": dpre.sum((0, 1)).to(dt)}
    if s["carry"]:
        out["state"] = dxp[:W - 1].transpose(0, 1).to(dt)
    return out


def _to_slots(cache, slots, new):
    """Writes row b of `new` to cache[slots[b]], negative slots to nowhere."""
    rows, B = cache.shape[0], new.shape[0]
    row_of = torch.full((rows + 1,), -1, device=slots.device, dtype=torch.long)
    row_of[torch.where(slots >= 0, slots, rows).long()] = torch.arange(B, device=slots.device)
    row_of = row_of[:rows].view(rows, *[1] * (new.dim() - 1))
    cache.copy_(torch.where(row_of >= 0, new[row_of.flatten().clamp(min=0)], cache))


def _plain_conv_step(s):
    w, dt = s["weight"].float(), s["x"].dtype
    old = s["state"] if s["slots"] is None else s["state"][s["slots"].clamp(min=0).long()]
    window = torch.cat([old, s["x"][:, None, :]], 1)
    pre = (window.float() * w).sum(1) + s["bias"].float()
    y = (pre * torch.sigmoid(pre)).to(dt)
    if s["slots"] is None:
        s["state"].copy_(window[:, 1:])
    else:
        y = torch.where((s["slots"] >= 0)[:, None], y, 0.0)
        _to_slots(s["state"], s["slots"], window[:, 1:])
    return {"y": y, "state": s["state"]}


BLOCK = 16


def _scan(a, b):
    """h_t = a_t h_{t-1} + b_t along the first axis from h = 0, and the running
    products of a: doubling steps inside blocks, then the blocks' ends likewise."""
    S = a.shape[0]
    T = min(BLOCK, 1 << (S - 1).bit_length())
    pad = -S % T
    if pad:
        a = torch.cat([a, a.new_ones(pad, *a.shape[1:])])
        b = torch.cat([b, b.new_zeros(pad, *b.shape[1:])])
    a, b = a.view(-1, T, *a.shape[1:]), b.view(-1, T, *b.shape[1:])
    step = 1
    while step < T:
        b = torch.cat([b[:, :step], torch.addcmul(b[:, step:], a[:, step:], b[:, :-step])], 1)
        a = torch.cat([a[:, :step], a[:, step:] * a[:, :-step]], 1)
        step *= 2
    if a.shape[0] > 1:
        pa, pb = _scan(a[:, -1], b[:, -1])
        pa, pb = (torch.cat([p.new_full((1, *p.shape[1:]), v), p[:-1]])[:, None] for p, v in ((pa, 1.0), (pb, 0.0)))
        b, a = torch.addcmul(b, a, pb), a * pa
    return a.reshape(-1, *a.shape[2:])[:S], b.reshape(-1, *b.shape[2:])[:S]


def _heads(t, H):
    """[S,B,G,N] seen by each of the H channels: [S,B,H,N] in 32 bits."""
    return t.float().repeat_interleave(H // t.shape[-2], dim=-2)


def _scan_terms(s):
    S, H = s["u"].shape[0], s["u"].shape[2]
    raw, u, Bm, Cm, valid = s["delta"].float() + s["delta_bias"], s["u"].float(), _heads(s["B"], H), _heads(s["C"], H), _valid(s, S)
    dt = torch.where(raw > 20, raw, torch.log1p(torch.exp(torch.clamp(raw, max=20.0))))
    if valid is not None:
        dt = torch.where(valid, dt, 0.0)
    return raw, dt, u, Bm, Cm, valid, torch.exp(dt[..., None] * s["A"])


def _plain_scan(s):
    raw, dt, u, Bm, Cm, valid, a = _scan_terms(s)
    pa, h = _scan(a, (dt * u)[..., None] * Bm)
    if s["state"] is not None:
        h = torch.addcmul(h, pa, s["state"])
    z = s["z"].float()
    y = ((h * Cm).sum(-1) + s["D"] * u) * z * torch.sigmoid(z)
    if valid is not None:
        y = torch.where(valid, y, 0.0)
    out = {"y": y.to(s["u"].dtype)}
    if s["carry"]:
        out["state"] = h[-1].clone()
    return out


def _plain_scan_bwd(s):
    raw, dt, u, Bm, Cm, valid, a = _scan_terms(s)
    S, B, H = u.shape
    G, N, out_t = s["B"].shape[2], s["B"].shape[3], s["u"].dtype
    pa, h = _scan(a, (dt * u)[..., None] * Bm)
    if s["state"] is not None:
        h = torch.addcmul(h, pa, s["state"])
    del pa
    first = s["state"] if s["state"] is not None else torch.zeros_like(h[0])
    gy, z = s["grad_y"].float(), s["z"].float()
    if valid is not None:
        gy = torch.where(valid, gy, 0.0)
    sig = torch.sigmoid(z)
    y = (h * Cm).sum(-1) + s["D"] * u
    gz = gy * y * sig * (1 + z * (1 - sig))
    gy = gy * z * sig
    # the states' gradients run backwards: g_t = C_t gy_t + a_{t+1} g_{t+1}
    last = s["grad_final_state"] if s["grad_final_state"] is not None else torch.zeros_like(h[0])
    after = torch.cat([a[1:], torch.ones_like(a[:1])])
    pg, gh = _scan(after.flip(0), (gy[..., None] * Cm).flip(0))
    gh = torch.addcmul(gh, pg, last).flip(0)
    del pg, after
    gC = (h * gy[..., None]).view(S, B, G, H // G, N).sum(3)
    gB = (gh * (dt * u)[..., None]).view(S, B, G, H // G, N).sum(3)
    gb = (gh * Bm).sum(-1)
    prev = torch.cat([first[None], h[:-1]])
    ga = gh * a * prev                                # the gradient of dt A
    del prev, h
    gdt = (ga * s["A"]).sum(-1) + gb * u
    graw = torch.where(raw > 20, gdt, gdt * torch.sigmoid(raw))
    if valid is not None:
        graw = torch.where(valid, graw, 0.0)
    out = {"u": (gb * dt + gy * s["D"]).to(out_t), "delta": graw.to(out_t), "A": (ga * dt[..., None]).sum((0, 1)),
           "B": gB.to(out_t), "C": gC.to(out_t), "D": (gy * u).sum((0, 1)), "z": gz.to(out_t), "delta_bias": graw.sum((0, 1))}
    if s["carry"]:
        out["state"] = gh[0] * a[0]
    return out


def _plain_scan_step(s):
    H = s["u"].shape[1]
    raw, u, z = s["delta"].float() + s["delta_bias"], s["u"].float(), s["z"].float()
    dt = torch.where(raw > 20, raw, torch.log1p(torch.exp(torch.clamp(raw, max=20.0))))
    old = s["state"] if s["slots"] is None else s["state"][s["slots"].clamp(min=0).long()]
    new = old * torch.exp(dt[..., None] * s["A"]) + (dt * u)[..., None] * _heads(s["B"], H)
    y = ((new * _heads(s["C"], H)).sum(-1) + s["D"] * u) * z * torch.sigmoid(z)
    if s["slots"] is None:
        s["state"].copy_(new)
    else:
        y = torch.where((s["slots"] >= 0)[:, None], y, 0.0)
        _to_slots(s["state"], s["slots"], new)
    return {"y": y.to(s["u"].dtype), "state": s["state"]}


PLAIN = {"conv": _plain_conv, "conv_bwd": _plain_conv_bwd, "conv_step": _plain_conv_step,
         "scan": _plain_scan, "scan_bwd": _plain_scan_bwd, "scan_step": _plain_scan_step}


# ------------------------------------------------------------------ the library
def _own(s):
    import causal_conv_backward_gb300 as mcc
    op = s["op"]
    if op == "conv":
        r = mcc.short_conv(s["x"], s["weight"], s["bias"], lengths=s["lengths"], state=s["state"], return_state=s["carry"])
        return {"y": r[0], "state": r[1]} if s["carry"] else {"y": r}
    if op == "conv_bwd":
        r = mcc.short_conv_backward(s["grad_y"], s["x"], s["weight"], s["bias"], lengths=s["lengths"], state=s["state"],
                                    grad_final_state=s["grad_final_state"])
        return {k: v for k, v in r._asdict().items() if v is not None}
    if op == "conv_step":
        y = mcc.short_conv_step(s["x"], s["state"], s["weight"], s["bias"], slots=s["slots"])
        return {"y": y, "state": s["state"]}
    if op == "scan":
        r = mcc.selective_scan(s["u"], s["delta"], s["A"], s["B"], s["C"], s["D"], s["z"], s["delta_bias"],
                               delta_softplus=True, lengths=s["lengths"], state=s["state"], return_state=s["carry"])
        return {"y": r[0], "state": r[1]} if s["carry"] else {"y": r}
    if op == "scan_bwd":
        r = mcc.selective_scan_backward(s["grad_y"], s["u"], s["delta"], s["A"], s["B"], s["C"], s["D"], s["z"], s["delta_bias"],
                                        delta_softplus=True, lengths=s["lengths"], state=s["state"],
                                        grad_final_state=s["grad_final_state"])
        return {k: v for k, v in r._asdict().items() if v is not None}
    y = mcc.selective_scan_step(s["u"], s["delta"], s["state"], s["A"], s["B"], s["C"], s["D"], s["z"], s["delta_bias"],
                                delta_softplus=True, slots=s["slots"])
    return {"y": y, "state": s["state"]}


def run(state):
    return _own(state) if own else PLAIN[state["op"]](state)


# ------------------------------------------------------------------ work
def work(case):
    S, B, H, W, N, G = (case[k] for k in ("S", "B", "H", "W", "N", "G"))
    e = S * B * H
    live = 0.75 if case["lengths"] else 1.0     # tokens before their sequence's length, on average
    if case["op"].startswith("conv"):
        window = B * (W - 1) * H * 2
        if case["op"] == "conv_step":           # x and the window in, y and the window out
            return {"bytes": 2 * e * 2 + 2 * window + (W + 1) * H * 2, "flops": e * (2 * W + 5)}
        carried = 2 * window if case["carry"] else 0
        if case["op"] == "conv":                # x in, y out
            return {"bytes": 2 * e * (live + 1) + (W + 1) * H * 2 + carried, "flops": e * live * (2 * W + 5)}
        return {"bytes": 2 * e * (2 * live + 1) + 2 * (W + 1) * H * 2 + 1.5 * carried,   # x, grad_y in, grad_x out
                "flops": e * live * (6 * W + 12)}
    weights = H * (N + 2) * 4
    states = B * H * N * 4
    bc = S * B * G * N * 2 * 2
    if case["op"] == "scan_step":               # u, delta, z and the state in, y and the state out
        return {"bytes": 4 * e * 2 + bc + weights + 2 * states, "flops": e * (7 * N + 25)}
    carried = 2 * states if case["carry"] else 0
    if case["op"] == "scan":                    # u, delta, z in, y out
        return {"bytes": 2 * e * (3 * live + 1) + live * bc + weights + carried, "flops": e * live * (7 * N + 25)}
    # u, delta, z, grad_y in, three gradients out, and those of B, C and the weights
    return {"bytes": 2 * e * (4 * live + 3) + (live + 1) * bc + 2 * weights + 1.5 * carried, "flops": e * live * (21 * N + 60)}


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    s = {k: v.to("cpu" if case["op"].endswith("step") else v.device) if isinstance(v, torch.Tensor) else v
         for k, v in prepare(case, seed).items()}
    d = {k: v.double() if isinstance(v, torch.Tensor) and v.is_floating_point() else v for k, v in s.items()}
    B, H, W, N = (case[k] for k in ("B", "H", "W", "N"))
    op = case["op"]
    if op.endswith("step"):
        return _exact_step(op, d, B, H, W)
    S = case["S"]
    dev = d["x"].device if "x" in d else d["u"].device
    n = s["lengths"].long() if s["lengths"] is not None else torch.full((B,), S, device=dev)
    live = (torch.arange(S, device=dev).view(S, 1) < n.view(1, B)).view(S, B, 1)
    if op.startswith("conv"):
        return _exact_conv(op, case, d, n, live, dev)
    return _exact_scan(op, case, d, n, live, dev)


def _exact_step(op, d, B, H, W):
    """Token by token, sequence by sequence."""
    rows = range(B) if d["slots"] is None else [int(v) for v in d["slots"]]
    state = d["state"].clone()
    y = torch.zeros(B, H, dtype=torch.float64)
    for b, r in enumerate(rows):
        if r < 0:
            continue
        if op == "conv_step":
            window = torch.cat([state[r], d["x"][b].view(1, H)])
            p = torch.einsum("kh,kh->h", window, d["weight"]) + d["bias"]
            y[b] = p / (1 + torch.exp(-p))
            state[r] = window[1:]
        else:
            per = H // d["B"].shape[1]
            Bm, Cm = (d[k][b].unsqueeze(1).expand(-1, per, -1).reshape(H, -1) for k in ("B", "C"))
            raw = d["delta"][b] + d["delta_bias"]
            dt = torch.logaddexp(raw, torch.zeros_like(raw)).view(H, 1)
            state[r] = torch.exp(dt * d["A"]) * state[r] + dt * Bm * d["u"][b].view(H, 1)
            z = d["z"][b]
            y[b] = (torch.einsum("hn,hn->h", state[r], Cm) + d["D"] * d["u"][b]) * z / (1 + torch.exp(-z))
    return {"y": y, "state": state}


def _exact_conv(op, case, d, n, live, dev):
    S, B, H, W = (case[k] for k in ("S", "B", "H", "W"))
    past = d["state"].permute(1, 0, 2) if d["state"] is not None else torch.zeros(W - 1, B, H, dtype=torch.float64, device=dev)
    xs = torch.cat((past, d["x"]), 0)
    taps = xs.unfold(0, W, 1)                                         # [S,B,H,W]
    pre = torch.einsum("sbhk,kh->sbh", taps, d["weight"]) + d["bias"]
    gate = 1 / (1 + torch.exp(-pre))
    at = n.view(1, B) + torch.arange(W - 1, device=dev).view(W - 1, 1)
    col = torch.arange(B, device=dev).view(1, B).expand(W - 1, B)
    if op == "conv":
        out = {"y": pre * gate * live}
        if case["carry"]:
            out["state"] = xs[at, col].permute(1, 0, 2)
        return out
    g = d["grad_y"] * live * (gate + pre * gate * (1 - gate))
    gxs = torch.zeros_like(xs)
    for k in range(W):
        gxs[k:S + k] += g * d["weight"][k]
    if d["grad_final_state"] is not None:
        gxs.index_put_((at, col), d["grad_final_state"].permute(1, 0, 2), accumulate=True)
    out = {"x": gxs[W - 1:], "weight": torch.einsum("sbh,sbhk->kh", g, taps), "bias": g.sum((0, 1))}
    if case["carry"]:
        out["state"] = gxs[:W - 1].permute(1, 0, 2)
    return out


def _exact_scan(op, case, d, n, live, dev):
    """The recurrence itself, one token after the other."""
    S, B, H, N, G = (case[k] for k in ("S", "B", "H", "N", "G"))
    if op == "scan" and S * B * H * N > 3e9 or op == "scan_bwd" and S * B * H * N > 1e9:
        return None
    zero = torch.zeros(B, H, N, dtype=torch.float64, device=dev)
    first = d["state"] if d["state"] is not None else zero
    raw = d["delta"] + d["delta_bias"]
    dt = torch.logaddexp(raw, torch.zeros_like(raw)) * live
    per = H // G

    def wide(t, i, j):                                                # B or C of steps i..j for each channel
        return t[i:j].unsqueeze(3).expand(-1, -1, -1, per, -1).reshape(j - i, B, H, N)

    part = max(1, min(S, int(2e8 // (B * H * N))))
    h, hs, y = first, [], torch.empty(S, B, H, dtype=torch.float64, device=dev)
    for i in range(0, S, part):
        j = min(S, i + part)
        a = torch.exp(dt[i:j].unsqueeze(3) * d["A"])
        b = wide(d["B"], i, j) * (dt[i:j] * d["u"][i:j]).unsqueeze(3)
        for t in range(j - i):
            h = torch.addcmul(b[t], a[t], h, out=b[t])
        h = h.clone()
        y[i:j] = torch.einsum("sbhn,sbhn->sbh", b, wide(d["C"], i, j))
        if op == "scan_bwd":
            hs.append(b)
    y += d["D"] * d["u"]
    gate = 1 / (1 + torch.exp(-d["z"]))
    if op == "scan":
        out = {"y": y * d["z"] * gate * live}
        if case["carry"]:
            out["state"] = h
        return out
    out = {"z": d["grad_y"] * live * y * gate * (1 + d["z"] * (1 - gate))}
    gy = d["grad_y"] * live * d["z"] * gate
    out["D"] = (gy * d["u"]).sum((0, 1))
    out["C"], out["B"] = (torch.empty(S, B, G, N, dtype=torch.float64, device=dev) for _ in range(2))
    gdt, gu = torch.empty_like(y), torch.empty_like(y)
    gA = torch.zeros(H, N, dtype=torch.float64, device=dev)
    g = d["grad_final_state"] if d["grad_final_state"] is not None else zero   # of the state, from later tokens
    starts = list(range(0, S, part))
    for q in reversed(range(len(starts))):
        i, j = starts[q], min(S, starts[q] + part)
        a = torch.exp(dt[i:j].unsqueeze(3) * d["A"])
        gh = wide(d["C"], i, j) * gy[i:j].unsqueeze(3)
        for t in reversed(range(j - i)):
            gh[t] += g
            g = gh[t] * a[t]
        before = torch.cat([(hs[q - 1][-1] if q else first).unsqueeze(0), hs[q][:-1]])
        out["C"][i:j] = (hs[q] * gy[i:j].unsqueeze(3)).reshape(j - i, B, G, per, N).sum(3)
        out["B"][i:j] = (gh * (dt[i:j] * d["u"][i:j]).unsqueeze(3)).reshape(j - i, B, G, per, N).sum(3)
        inner = torch.einsum("sbhn,sbhn->sbh", gh, wide(d["B"], i, j))
        through = gh * a * before
        gA += torch.einsum("sbhn,sbh->hn", through, dt[i:j])
        gdt[i:j] = torch.einsum("sbhn,hn->sbh", through, d["A"]) + inner * d["u"][i:j]
        gu[i:j] = inner * dt[i:j] + gy[i:j] * d["D"]
    out["u"], out["A"] = gu, gA
    out["delta"] = gdt * live / (1 + torch.exp(-raw))
    out["delta_bias"] = out["delta"].sum((0, 1))
    if case["carry"]:
        out["state"] = g
    return out
