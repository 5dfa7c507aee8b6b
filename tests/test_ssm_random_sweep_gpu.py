"""Seeded random cases of the short convolution and the selective scan against
their definitions in 64 bits: shapes, groups, states, options, lengths and a
memory order drawn for every tensor."""
import random

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import causal_conv_backward_gb300 as m  # noqa: E402
import ssm_reference as ref  # noqa: E402
from test_ssm_gpu import as_strided, cuda_ready, guards, lens, poison, rand, reference_scan  # noqa: E402,F401

LAYOUTS = ("dense", "slice", "odd", "batch first")


@pytest.mark.parametrize("seed", range(30))
def test_scan(seed):
    r = random.Random(seed)
    G = r.choice((1, 1, 2, 3))
    S, B, H, N = r.randint(1, 90), r.randint(1, 4), G * r.choice((r.randint(1, 40), 32, 64)), r.choice((16, r.randint(1, 64)))
    dtype = r.choice((torch.bfloat16, torch.float16))
    opts = "p" + "".join(o for o in "Dzbs" if r.random() < 0.6)
    lengths = [r.randint(0, S) for _ in range(B)] if r.random() < 0.5 else None
    ln = lens(lengths)
    clean = {"u": rand(S, B, H, dtype=dtype, seed=1), "delta": rand(S, B, H, dtype=dtype, scale=0.5, seed=2),
             "A": -torch.exp(rand(H, N, dtype=torch.float32, seed=3)), "B": rand(S, B, G, N, dtype=dtype, seed=4),
             "C": rand(S, B, G, N, dtype=dtype, seed=5), "D": rand(H, dtype=torch.float32, seed=6) if "D" in opts else None,
             "z": rand(S, B, H, dtype=dtype, seed=7) if "z" in opts else None,
             "delta_bias": rand(H, dtype=torch.float32, seed=8) - 2 if "b" in opts else None,
             "state": rand(B, H, N, dtype=torch.float32, seed=9) if "s" in opts else None}
    t = {k: poison(as_strided(v.clone(), r.choice(LAYOUTS)), ln) if v is not None and k in ("u", "delta", "B", "C", "z") else v
         for k, v in clean.items()}
    args = [t[k] for k in ("u", "delta", "A", "B", "C", "D", "z", "delta_bias")]
    leaves, ry, rf = reference_scan(clean, opts, lengths)
    y, f = m.selective_scan(*args, delta_softplus=True, lengths=ln, state=t["state"], return_state=True)
    ref.check(y, ry, N + 64, "y")
    ref.check(f, rf, N + 64, "final state")
    gy = rand(S, B, H, dtype=dtype, seed=20)
    gf = rand(B, H, N, dtype=torch.float32, seed=21) if r.random() < 0.5 else None
    loss = (ry * ref.to64(gy)).sum() + ((rf * ref.to64(gf)).sum() if gf is not None else 0)
    loss = loss + sum(0 * v.sum() for v in leaves.values() if v is not None)     # a graph even where no token is left
    got = m.selective_scan_backward(poison(as_strided(gy.clone(), r.choice(LAYOUTS)), ln), *args, delta_softplus=True,
                                    lengths=ln, state=t["state"], grad_final_state=gf)
    names = [k for k in got._fields if leaves[k] is not None]
    for k, v in zip(names, torch.autograd.grad(loss, [leaves[k] for k in names], allow_unused=True)):
        terms = {"B": H // G + 64, "C": H // G + 64, "A": S * B, "D": S * B, "delta_bias": S * B}.get(k, 4 * N + 64)
        ref.check(getattr(got, k), torch.zeros_like(leaves[k]) if v is None else v, terms, k)


@pytest.mark.parametrize("seed", range(30))
def test_conv(seed):
    r = random.Random(1000 + seed)
    S, B, H, W = r.randint(1, 300), r.randint(1, 4), r.choice((r.randint(1, 140), 64, 256)), r.randint(1, 8)
    dtype = r.choice((torch.bfloat16, torch.float16))
    silu, has_bias, has_state = r.random() < 0.7, r.random() < 0.7, r.random() < 0.6
    lengths = [r.randint(0, S) for _ in range(B)] if r.random() < 0.5 else None
    ln = lens(lengths)
    x, w = rand(S, B, H, dtype=dtype, seed=1), rand(W, H, dtype=dtype, scale=W ** -0.5, seed=2)
    b = rand(H, dtype=dtype, seed=3) if has_bias else None
    st = rand(B, W - 1, H, dtype=dtype, seed=4) if has_state else None
    xs = poison(as_strided(x.clone(), r.choice(LAYOUTS)), ln)
    kw = dict(activation="silu" if silu else None, lengths=ln, state=st)
    leaves = [ref.to64(t, grad=True) for t in (x, w, b, st)]
    ry, rf = ref.conv(leaves[0], leaves[1], leaves[2], silu, lengths, leaves[3])
    y, f = m.short_conv(xs, w, b, return_state=True, **kw)
    ref.check(y, ry, W, "y")
    assert torch.equal(f.cpu().double(), rf.detach())
    gy = rand(S, B, H, dtype=dtype, seed=5)
    gf = rand(B, W - 1, H, dtype=dtype, seed=6) if r.random() < 0.5 else None
    loss = (ry * ref.to64(gy)).sum() + ((rf * ref.to64(gf)).sum() if gf is not None else 0)
    loss = loss + sum(0 * v.sum() for v in leaves if v is not None)
    got = m.short_conv_backward(poison(as_strided(gy.clone(), r.choice(LAYOUTS)), ln), xs, w, b, grad_final_state=gf, **kw)
    names = [(k, leaf) for k, leaf in zip(("x", "weight", "bias", "state"), leaves) if leaf is not None]
    for (k, leaf), v in zip(names, torch.autograd.grad(loss, [leaf for _, leaf in names], allow_unused=True)):
        ref.check(getattr(got, k), torch.zeros_like(leaf) if v is None else v, W if k in ("x", "state") else S * B, k)
