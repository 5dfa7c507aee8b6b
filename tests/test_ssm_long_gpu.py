"""The short convolution and the selective scan at sizes where runs of rows are
long and chunks hold several tiles: many sequences of few channels, against the
definitions in float64 on the GPU. Each test first asserts from the workspace's
size that the plan has the form it is there for."""
import ctypes

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import causal_conv_backward_gb300 as m  # noqa: E402
import ssm_reference as ref  # noqa: E402
from causal_conv_backward_gb300 import _ssm  # noqa: E402
from test_ssm_gpu import BF16, F32, FP16, as_strided, cuda_ready, guards, lens, poison, rand  # noqa: E402,F401


def some_lengths(S, B):
    """Every third sequence whole, the others ending anywhere, one empty and one of one token."""
    return [S if b % 3 == 0 else 0 if b == 1 else 1 if b == 2 else (b * 7919) % (S + 1) for b in range(B)]


def live_rows(lengths, S, B):
    """[S,B,1] bool."""
    n = torch.full((B,), S, device="cuda") if lengths is None else torch.tensor(lengths, device="cuda")
    return (torch.arange(S, device="cuda")[:, None] < n)[:, :, None]


def leaf(t):
    return None if t is None else t.detach().double().requires_grad_(True)


def workspace(name, args):
    n = ctypes.c_uint64()
    assert getattr(_ssm._load(), f"mcc1d_{name}_workspace_size")(ctypes.byref(args), n) == 0
    return n.value


# ------------------------------------------------------------------ short convolution
def conv64(x, w, b, silu, lengths, state):
    """The convolution and its final window, all sequences at once."""
    (S, B, H), W = x.shape, w.shape[0]
    live = live_rows(lengths, S, B)
    past = torch.zeros(W - 1, B, H, dtype=x.dtype, device=x.device) if state is None else state.transpose(0, 1)
    rows = torch.cat([past, torch.where(live, x, 0.0)])
    pre = sum(rows[k:k + S] * w[k] for k in range(W))
    if b is not None:
        pre = pre + b
    y = torch.where(live, pre * torch.sigmoid(pre) if silu else pre, 0.0)
    at = live.sum(0).view(1, B, 1) + torch.arange(W - 1, device=x.device).view(-1, 1, 1)
    return y, torch.gather(rows, 0, at.expand(-1, -1, H)).transpose(0, 1)


CONV = [  # S, B, H, W, dtype, lengths, silu, layout, channels per thread
    (530, 152, 256, 4, BF16, True, True, "dense", 4),
    (517, 160, 256, 3, FP16, False, False, "slice", 4),
    (530, 152, 130, 2, FP16, True, True, "batch first", 2),
    (530, 152, 258, 6, BF16, True, True, "dense", 2),
    (523, 152, 128, 8, FP16, True, True, "slice", 2),
    (530, 152, 101, 4, BF16, True, True, "odd", 1),
    (519, 152, 101, 7, FP16, True, False, "odd", 1),
]


@pytest.mark.parametrize("S,B,H,W,dtype,ends,silu,layout,vec", CONV)
def test_conv_long_runs(S, B, H, W, dtype, ends, silu, layout, vec):
    lengths = some_lengths(S, B) if ends else None
    ln = lens(lengths)
    x0, w, b = rand(S, B, H, dtype=dtype, seed=1), rand(W, H, dtype=dtype, scale=W ** -0.5, seed=2), rand(H, dtype=dtype, seed=3)
    s0, gy0, gf = rand(B, W - 1, H, dtype=dtype, seed=4), rand(S, B, H, dtype=dtype, seed=5), rand(B, W - 1, H, dtype=dtype, seed=6)
    x, gy = (poison(as_strided(t.clone(), layout), ln) for t in (x0, gy0))
    # the backward: a run of L rows per warp, eight warps to a block of partial sums [W+1,H]
    a = m.ShortConvBwdArgs(grad_y=256, grad_y_strides=(B * H, H), x=256, x_strides=(B * H, H), weight=256, grad_x=256,
                           grad_weight=256, S=S, B=B, H=H, W=W)
    blocks = workspace("short_conv_bwd", a) // (4 * (W + 1) * H * B)
    assert blocks <= (S + 8 * 64 - 1) // (8 * 64)       # L >= 64: sixteen batches of rows
    # the forward: runs get shorter until 1216 blocks of 128 threads
    threads = B * (H // vec)
    assert (threads + 127) // 128 * ((S + 31) // 32) >= 1216    # L >= 32
    leaves = [leaf(t) for t in (x0, w, b, s0)]
    ry, rf = conv64(*leaves[:3], silu, lengths, leaves[3])
    kw = dict(activation="silu" if silu else None, lengths=ln, state=s0)
    y, final = m.short_conv(x, w, b, return_state=True, **kw)
    ref.check(y, ry, W, "y")
    assert torch.equal(final.double(), rf)
    loss = (ry * gy0.double()).sum() + (rf * gf.double()).sum()
    got = m.short_conv_backward(gy, x, w, b, grad_final_state=gf, **kw)
    for name, want in zip(("x", "weight", "bias", "state"), torch.autograd.grad(loss, leaves)):
        ref.check(getattr(got, name), want, W if name in ("x", "state") else S * B, name)


@pytest.mark.parametrize("dtype,silu", [(BF16, True), (FP16, False)])
def test_conv_forward_longest_runs(dtype, silu):
    """Runs of 128 rows, four channels per thread."""
    S, B, H, W = 1030, 2, 69632, 4
    assert B * H // 4 // 128 * ((S + 127) // 128) >= 1216
    lengths = [S, 777]
    x, w, b = rand(S, B, H, dtype=dtype, seed=1), rand(W, H, dtype=dtype, scale=0.5, seed=2), rand(H, dtype=dtype, seed=3)
    y = m.short_conv(x, w, b, activation="silu" if silu else None, lengths=lens(lengths))
    for h in range(0, H, H // 4):       # a quarter of the channels at a time
        c = slice(h, h + H // 4)
        ref.check(y[:, :, c], conv64(x[:, :, c].double(), w[:, c].double(), b[c].double(), silu, lengths, None)[0], W, "y")


# ------------------------------------------------------------------ selective scan
def scan64(t, lengths):
    """The scan and its final state, token by token, all sequences at once."""
    S, B, H = t["u"].shape
    live, per = live_rows(lengths, S, B), H // t["B"].shape[2]
    dt = t["delta"] if t["delta_bias"] is None else t["delta"] + t["delta_bias"]
    dt = torch.where(live, torch.logaddexp(dt, torch.zeros_like(dt)), 0.0)[..., None]
    a, b = torch.exp(dt * t["A"]), dt * t["u"][..., None] * t["B"].repeat_interleave(per, 2)
    h, hs = t["state"], []
    for s in range(S):
        h = a[s] * h + b[s]
        hs.append(h)
    y = (torch.stack(hs) * t["C"].repeat_interleave(per, 2)).sum(-1) + t["D"] * t["u"]
    return torch.where(live, y * t["z"] * torch.sigmoid(t["z"]), 0.0), h


def scan_bwd_chunks(S, B, H, N, G):
    """Tiles and chunks of the backward's plan, from its workspace: per chunk two states, the sum of dt, grad_A,
    grad_D and grad_delta_bias; per tile a state and a sum of dt; per token, sequence and block a row of grad_B, grad_C."""
    lanes = 1
    while 4 * lanes < N:
        lanes *= 2
    tile, np = (4 * lanes if lanes < 4 else 16), 4 * lanes
    a = m.ScanBwdArgs(fwd=m.ScanArgs(u=256, u_strides=(B * H, H), delta=256, delta_strides=(B * H, H), B_=256,
                                     B_strides=(B * G * N, G * N, N), C=256, C_strides=(B * G * N, G * N, N), A=256,
                                     S=S, B=B, H=H, N=N, G=G, flags=2),
                      grad_y=256, grad_y_strides=(B * H, H), grad_u=256, grad_delta=256, grad_B=256, grad_C=256, grad_A=256)
    have, tiles = workspace("scan_bwd", a), (S + tile - 1) // tile
    blocks = G * ((H // G + 256 // lanes - 1) // (256 // lanes))

    def need(chunks):
        parts = [chunks * np * 4] * 3 + [chunks * 4, chunks * 8, tiles * np * 4, tiles * 4]
        return sum((B * H * p + 255) // 256 * 256 for p in parts) + (S * B * blocks * 2 * np * 4 + 255) // 256 * 256

    chunks = [c for c in range(1, tiles + 1) if need(c) == have]
    assert len(chunks) == 1
    return tiles, chunks[0]


SCAN_BWD = [  # S, B, H, N, G, dtype, lengths, layout
    (163, 128, 10, 3, 2, BF16, True, "dense"),
    (330, 128, 10, 8, 2, FP16, True, "slice"),
    (329, 256, 10, 16, 1, BF16, True, "dense"),
    (330, 128, 12, 16, 2, FP16, True, "batch first"),
    (450, 128, 7, 16, 1, BF16, False, "odd"),
    (330, 128, 6, 29, 2, BF16, True, "odd"),
    (330, 128, 4, 64, 2, FP16, True, "dense"),
    (420, 3, 100, 16, 50, BF16, True, "dense"),
    (330, 5, 1600, 32, 1, BF16, False, "dense"),
]


@pytest.mark.parametrize("S,B,H,N,G,dtype,ends,layout", SCAN_BWD)
def test_scan_backward_over_chunks_of_several_tiles(S, B, H, N, G, dtype, ends, layout):
    tiles, chunks = scan_bwd_chunks(S, B, H, N, G)
    assert chunks > 1 and tiles >= 2 * chunks
    lengths = some_lengths(S, B) if ends else None
    ln = lens(lengths)
    clean = {"u": rand(S, B, H, dtype=dtype, seed=1), "delta": rand(S, B, H, dtype=dtype, scale=0.5, seed=2),
             # long and short memories: states of the chunks before still count
             "A": -torch.exp(2 * rand(H, N, dtype=F32, seed=3) - 2), "B": rand(S, B, G, N, dtype=dtype, seed=4),
             "C": rand(S, B, G, N, dtype=dtype, seed=5), "D": rand(H, dtype=F32, seed=6), "z": rand(S, B, H, dtype=dtype, seed=7),
             "delta_bias": rand(H, dtype=F32, seed=8) - 3, "state": rand(B, H, N, dtype=F32, seed=9)}
    t = {k: poison(as_strided(v.clone(), layout), ln) if k in ("u", "delta", "B", "C", "z") else v for k, v in clean.items()}
    args = [t[k] for k in ("u", "delta", "A", "B", "C", "D", "z", "delta_bias")]
    gy0, gf = rand(S, B, H, dtype=dtype, seed=20), rand(B, H, N, dtype=F32, seed=21)
    leaves = {k: leaf(v) for k, v in clean.items()}
    ry, rf = scan64(leaves, lengths)
    y, final = m.selective_scan(*args, delta_softplus=True, lengths=ln, state=t["state"], return_state=True)
    ref.check(y, ry, N + S, "y")
    ref.check(final, rf, N + S, "final state")
    loss = (ry * gy0.double()).sum() + (rf * gf.double()).sum()
    got = m.selective_scan_backward(poison(as_strided(gy0.clone(), layout), ln), *args, delta_softplus=True, lengths=ln,
                                    state=t["state"], grad_final_state=gf)
    for k, want in zip(got._fields, torch.autograd.grad(loss, [leaves[k] for k in got._fields])):
        terms = {"B": H // G + S, "C": H // G + S, "A": S * B, "D": S * B, "delta_bias": S * B}.get(k, 4 * N + S)
        ref.check(getattr(got, k), want, terms, k)


@pytest.mark.parametrize("S,B,H,N,G,dtype,layout", [
    (230, 2, 20, 3, 1, BF16, "dense"), (230, 2, 21, 4, 1, FP16, "odd"), (300, 2, 36, 8, 3, BF16, "slice"),
    (300, 2, 33, 16, 1, BF16, "odd"), (300, 1, 40, 32, 2, FP16, "dense"), (260, 2, 21, 64, 1, BF16, "odd"),
])
def test_scan_forward_in_chunks(S, B, H, N, G, dtype, layout):
    a = m.ScanArgs(u=256, u_strides=(B * H, H), delta=256, delta_strides=(B * H, H), B_=256, B_strides=(B * G * N, G * N, N),
                   C=256, C_strides=(B * G * N, G * N, N), A=256, y=256, S=S, B=B, H=H, N=N, G=G, flags=2)
    assert workspace("scan", a) > 0     # a plan of one chunk needs none
    lengths = [S, S - 67][:B]
    ln = lens(lengths)
    clean = {"u": rand(S, B, H, dtype=dtype, seed=1), "delta": rand(S, B, H, dtype=dtype, scale=0.5, seed=2),
             "A": -torch.exp(2 * rand(H, N, dtype=F32, seed=3) - 2), "B": rand(S, B, G, N, dtype=dtype, seed=4),
             "C": rand(S, B, G, N, dtype=dtype, seed=5), "D": rand(H, dtype=F32, seed=6), "z": rand(S, B, H, dtype=dtype, seed=7),
             "delta_bias": rand(H, dtype=F32, seed=8) - 3, "state": rand(B, H, N, dtype=F32, seed=9)}
    t = {k: poison(as_strided(v.clone(), layout), ln) if k in ("u", "delta", "B", "C", "z") else v for k, v in clean.items()}
    ry, rf = scan64({k: v.double() for k, v in clean.items()}, lengths)
    y, final = m.selective_scan(*[t[k] for k in ("u", "delta", "A", "B", "C", "D", "z", "delta_bias")], delta_softplus=True,
                                lengths=ln, state=t["state"], return_state=True)
    ref.check(y, ry, N + S, "y")
    ref.check(final, rf, N + S, "final state")
