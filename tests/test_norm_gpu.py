"""The gated norm and the residual norm against float64: row lengths on both
sides of every choice of threads, odd ones, strides, single tokens, types."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import causal_conv_backward_gb300 as m  # noqa: E402
import norm_reference as ref  # noqa: E402

BF16, FP16, F32 = torch.bfloat16, torch.float16, torch.float32
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def cuda_ready():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from causal_conv_backward_gb300 import build
    build.build()


def rand(*shape, dtype=BF16, scale=1.0, seed=0, add=0.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (add + scale * torch.randn(shape, generator=g, device="cuda")).to(dtype)


def d64(t):
    return None if t is None else t.detach().double().cpu().requires_grad_()


def strided(t, how):
    """The same values in another layout, the last axis adjacent."""
    if how == "dense":
        return t
    if how == "half":          # the second half of a projection's rows
        wide = torch.full((*t.shape[:-1], 2 * t.shape[-1]), float("nan"), dtype=t.dtype, device=t.device)
        wide[..., t.shape[-1]:] = t
        return wide[..., t.shape[-1]:]
    if how == "odd":           # rows at odd addresses
        wide = torch.full((*t.shape[:-1], t.shape[-1] + 3), float("nan"), dtype=t.dtype, device=t.device)
        wide[..., 1:-2] = t
        return wide[..., 1:-2]
    return t.transpose(0, 1).contiguous().transpose(0, 1)      # "swapped"


# D on both sides of 64, 128, 256, 1024, 2048, 4096 (vectors) and 128, 512, 2048 (single values)
@pytest.mark.parametrize("D", [1, 3, 8, 64, 72, 100, 128, 136, 129, 256, 264, 511, 513, 1024, 1032, 2047, 2048, 2056, 2051, 4104, 16384, 16383])
@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_gated_norm(D, dtype):
    S, B, H = (5, 3, 7) if D <= 512 else (3, 2, 2)
    x, z, w, gy = rand(S, B, H, D, dtype=dtype, seed=1), rand(S, B, H, D, dtype=dtype, seed=2), rand(D, dtype=dtype, seed=3, add=1), rand(S, B, H, D, dtype=dtype, seed=4)
    check_gated(x, z, w, gy, EPS)


@pytest.mark.parametrize("how", ["half", "odd", "swapped"])
@pytest.mark.parametrize("D", [64, 100, 128, 2048])
def test_gated_norm_strides(how, D):
    S, B, H = 4, 3, 2
    x, z, w, gy = rand(S, B, H, D, seed=1), rand(S, B, H, D, seed=2), rand(D, seed=3, add=1), rand(S, B, H, D, seed=4)
    check_gated(strided(x, how), strided(z, how), w, strided(gy, how), 1e-3)
    check_gated(x, None, w, strided(gy, how), 1e-3)


def check_gated(x, z, w, gy, eps):
    x6, z6, w6, g6 = d64(x), d64(z), d64(w), gy.double().cpu()
    want = ref.gated(x6, z6, w6, eps)
    ref.check(m.gated_norm(x, z, w, eps=eps), want, want.abs(), what="y")
    got = m.gated_norm_backward(gy, x, z, w, eps=eps)
    leaves = [t for t in (x6, z6, w6) if t is not None]
    grads = torch.autograd.grad((want * g6).sum(), leaves)
    with torch.no_grad():
        r = 1 / torch.sqrt(x6.square().mean(-1, keepdim=True) + eps)
        gate = 1 if z6 is None else z6 * torch.sigmoid(z6)
        n, t = x6 * r, (g6 * gate * w6).abs()
        # grad_x is a difference of two terms, the second a mean of products
        size_x = r * (t + n.abs() * (t * n.abs()).mean(-1, keepdim=True))
        size_w = (g6 * gate * n).abs().sum((0, 1, 2))
        ref.check(got.x, grads[0], size_x, what="x")
        if z6 is None:
            assert got.z is None
        else:
            ref.check(got.z, grads[1], (g6 * n * w6).abs() * (1 + z6.abs()), what="z")
        ref.check(got.weight, grads[-1], size_w, what="weight")


@pytest.mark.parametrize("shape", [(5, 33), (3, 5, 64), (1, 1, 1, 128)])
def test_gated_norm_leading_axes(shape):
    x, z, w = rand(*shape, seed=1), rand(*shape, seed=2), rand(shape[-1], seed=3)
    y = m.gated_norm(x, z, w)
    ref.check(y, ref.gated(d64(x), d64(z), d64(w), EPS), y.abs() * 2, what="y")
    assert m.gated_norm_backward(y, x, z, w).x.shape == x.shape


@pytest.mark.parametrize("H", [1, 40, 100, 384, 1000, 1001, 2048, 2500, 4096, 8192, 5001])
@pytest.mark.parametrize("dtype,wide", [(BF16, False), (BF16, True), (FP16, False), (FP16, True)])
@pytest.mark.parametrize("branch", ["", "p", "s", "ps"])
def test_residual_norm(H, dtype, wide, branch):
    S, B = 5, 3
    check_residual(*residual_inputs(S, B, H, dtype, wide, branch), True)


def residual_inputs(S, B, H, dtype, wide, branch, how="dense"):
    rt = F32 if wide else dtype
    x, r = strided(rand(S, B, H, dtype=dtype, seed=1), how), strided(rand(S, B, H, dtype=rt, seed=2, scale=2.0), how)
    w = rand(H, dtype=dtype, seed=3, add=1)
    post = rand(H, dtype=dtype, seed=4, add=1) if "p" in branch else None
    scale = rand(H, dtype=F32, seed=5) if "s" in branch else None
    gy, gh = strided(rand(S, B, H, dtype=dtype, seed=6), how), strided(rand(S, B, H, dtype=rt, seed=7), how)
    return x, r, w, post, scale, gy, gh


@pytest.mark.parametrize("how", ["half", "odd", "swapped"])
@pytest.mark.parametrize("H", [64, 999, 2048])
@pytest.mark.parametrize("wide", [False, True])
def test_residual_norm_strides(how, H, wide):
    check_residual(*residual_inputs(4, 3, H, BF16, wide, "ps", how), False)


def check_residual(x, r, w, post, scale, gy, gh, with_h):
    x6, r6, w6, p6, s6 = (d64(t) for t in (x, r, w, post, scale))
    gy6, gh6 = gy.double().cpu(), gh.double().cpu()
    y6, h6 = ref.residual(x6, r6, w6, p6, s6, EPS)
    y, h = m.residual_norm(x, r, w, post_weight=post, scale=scale, eps=EPS)
    assert h.dtype is r.dtype and y.dtype is x.dtype
    with torch.no_grad():
        m6 = x6 if p6 is None else ref.rms(x6, EPS) * p6
        sm = m6 if s6 is None else s6 * m6
        size_h = r6.abs() + sm.abs()           # what cancels in the sum
        rh = 1 / torch.sqrt(h6.square().mean(-1, keepdim=True) + EPS)
        ref.check(h, h6, size_h, what="h")
        ref.check(y, y6, (size_h + h6.abs()) * rh * w6.abs(), what="y")
    got = m.residual_norm_backward(gy, gh if with_h else None, x, r, w, post_weight=post, scale=scale, eps=EPS)
    loss = (y6 * gy6).sum() + ((h6 * gh6).sum() if with_h else 0)
    names = [k for k, t in zip(got._fields, (x6, r6, w6, p6, s6)) if t is not None]
    want = dict(zip(names, torch.autograd.grad(loss, [t for t in (x6, r6, w6, p6, s6) if t is not None])))
    with torch.no_grad():
        n, nh = (size_h + h6.abs()) * rh, (gy6 * w6).abs()
        size_g = (gh6.abs() if with_h else 0) + rh * (nh + n * (nh * n).mean(-1, keepdim=True))
        gm = size_g * (1 if s6 is None else s6.abs())
        size_x = gm
        if p6 is not None:
            r1 = 1 / torch.sqrt(x6.square().mean(-1, keepdim=True) + EPS)
            n1, t = (x6 * r1).abs(), gm * p6.abs()
            size_x = r1 * (t + n1 * (t * n1).mean(-1, keepdim=True))
            ref.check(got.post_weight, want["post_weight"], (gm * n1).sum((0, 1)), what="post_weight")
        ref.check(got.x, want["x"], size_x, what="x")
        ref.check(got.residual, want["residual"], size_g, what="residual")
        ref.check(got.weight, want["weight"], (gy6.abs() * n).sum((0, 1)), what="weight")
        if s6 is not None:
            ref.check(got.scale, want["scale"], (size_g * m6.abs()).sum((0, 1)), what="scale")
    for k, t in (("post_weight", post), ("scale", scale)):
        assert (getattr(got, k) is None) == (t is None)


def test_single_token_and_leading_axes():
    x, r, w = rand(3, 512, seed=1), rand(3, 512, dtype=F32, seed=2), rand(512, seed=3)
    y, h = m.residual_norm(x, r, w)
    y3, h3 = m.residual_norm(x[None], r[None], w)
    assert y.shape == x.shape and torch.equal(y, y3[0]) and torch.equal(h, h3[0])


def test_many_rows_sum_their_weights():
    """More rows than one pass of the blocks: the partial sums of all of them."""
    S, B, H, D = 3001, 2, 4, 128
    x, z, w, gy = rand(S, B, H, D, seed=1), rand(S, B, H, D, seed=2), rand(D, seed=3, add=1), rand(S, B, H, D, seed=4)
    check_gated(x, z, w, gy, EPS)
    check_residual(*residual_inputs(2100, 2, 2048, BF16, True, "ps"), True)


def test_zero_rows_and_large_values():
    """A row of zeros is zero (eps holds the root), values near fp32's root of its largest are not lost."""
    x, z, w = rand(4, 2, 1, 96, seed=1), rand(4, 2, 1, 96, seed=2), rand(96, seed=3)
    x[1] = 0
    x[2] *= 1e17                                    # squares near 1e34
    x[3] *= 1e-17
    y = m.gated_norm(x, z, w)
    assert not y[1].any()
    want = ref.gated(d64(x), d64(z), d64(w), EPS)
    ref.check(y, want, want.abs(), what="y")
    g = m.gated_norm_backward(rand(4, 2, 1, 96, seed=4), x, z, w)
    assert all(torch.isfinite(t).all() for t in g)


def test_same_bits_every_time_and_in_a_graph():
    args = residual_inputs(300, 3, 1536, BF16, True, "ps")
    x, r, w, post, scale, gy, gh = args
    kw = dict(post_weight=post, scale=scale)
    first = (*m.residual_norm(x, r, w, **kw), *m.residual_norm_backward(gy, gh, x, r, w, **kw))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        again = (*m.residual_norm(x, r, w, **kw), *m.residual_norm_backward(gy, gh, x, r, w, **kw))
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(first, again))


# both sides of the shapes' widths, with more rows than blocks
@pytest.mark.parametrize("D", [257, 512, 520, 1025, 1536, 1544, 2560, 4097, 4104, 8191, 8192, 8193, 8200, 16383, 16384])
def test_many_rows_of_each_shape(D):
    x, z, w, gy = rand(107, 3, 1, D, seed=1), rand(107, 3, 1, D, seed=2), rand(D, seed=3, add=1), rand(107, 3, 1, D, seed=4)
    check_gated(x, z, w, gy, EPS)
    check_residual(*residual_inputs(107, 3, D, BF16, True, "ps"), True)
    check_residual(*residual_inputs(107, 3, D, FP16, False, ""), False)
