"""The short convolution and the selective scan on a stream of their own while
the current stream is busy: memory that one of the two still uses is not handed
to the other. Waits are kernels that spin for a fixed number of cycles."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import causal_conv_backward_gb300 as m  # noqa: E402

CYCLES = 100_000_000      # some 50 ms


@pytest.fixture(scope="module", autouse=True)
def cuda_ready():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from causal_conv_backward_gb300 import build
    build.build()


def inputs():
    S, B, H, W, N = 300, 2, 96, 4, 16
    g = torch.Generator(device="cuda").manual_seed(0)

    def rand(*shape, dtype=torch.bfloat16):
        return torch.randn(shape, generator=g, device="cuda").to(dtype)

    f32 = torch.float32
    x, w, b, win = rand(S, B, H), rand(W, H), rand(H), rand(B, W - 1, H)
    scan = dict(delta=rand(S, B, H), A=-torch.exp(rand(H, N, dtype=f32)), B=rand(S, B, 1, N), C=rand(S, B, 1, N), D=rand(H, dtype=f32),
                z=rand(S, B, H), delta_bias=rand(H, dtype=f32))
    state, gy = rand(B, H, N, dtype=f32), rand(S, B, H)
    ln = torch.tensor([S, 211], dtype=torch.int32, device="cuda")
    one = dict(scan, **{k: scan[k][0].contiguous() for k in ("delta", "B", "C", "z")})
    return {
        "short_conv": (m.short_conv, dict(x=x, weight=w, bias=b, lengths=ln, state=win, return_state=True)),
        "short_conv_backward": (m.short_conv_backward, dict(grad_y=gy, x=x, weight=w, bias=b, lengths=ln, state=win)),
        "short_conv_step": (m.short_conv_step, dict(x=x[0].contiguous(), state=win, weight=w, bias=b)),
        "selective_scan": (m.selective_scan, dict(scan, u=x, lengths=ln, state=state, return_state=True, delta_softplus=True)),
        "selective_scan_backward": (m.selective_scan_backward, dict(scan, grad_y=gy, u=x, lengths=ln, state=state, delta_softplus=True)),
        "selective_scan_step": (m.selective_scan_step, dict(one, u=x[0].contiguous(), state=state, delta_softplus=True)),
    }


NAMES = ("short_conv", "short_conv_backward", "short_conv_step", "selective_scan", "selective_scan_backward", "selective_scan_step")


def call(name, args, **kw):
    """The outputs, the state that a step moves on among them."""
    out = args[name][0](**args[name][1], **kw)
    out = list(out) if isinstance(out, tuple) else [out]
    return [t for t in out if t is not None] + ([args[name][1]["state"]] if name.endswith("step") else [])


def same(got, want):
    return all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("name", NAMES)
def test_current_stream_still_writes_freed_memory(name):
    want = [t.clone() for t in call(name, inputs())]
    args, side = inputs(), torch.cuda.Stream()
    torch.cuda.synchronize()
    old = [torch.empty_like(t) for t in want for _ in range(4)]
    torch.cuda._sleep(CYCLES)
    for t in old:
        t.fill_(float("nan"))
    del t, old                          # free for the current stream, which has yet to write them
    got = call(name, args, stream=side)
    torch.cuda.synchronize()
    assert same(got, want)


@pytest.mark.parametrize("name", NAMES)
def test_inputs_freed_while_the_stream_works(name):
    want = [t.clone() for t in call(name, inputs())]
    args, side = inputs(), torch.cuda.Stream()
    torch.cuda.synchronize()
    sizes = [(t.shape, t.dtype) for t in args[name][1].values() if isinstance(t, torch.Tensor)]
    with torch.cuda.stream(side):
        torch.cuda._sleep(CYCLES)
    got = call(name, args, stream=side)
    args.clear()
    new = [torch.full(shape, 1, dtype=dtype, device="cuda") for shape, dtype in sizes for _ in range(4)]
    torch.cuda.synchronize()
    assert same(got, want) and len(new) > 0


@pytest.mark.parametrize("name", [n for n in NAMES if not n.endswith("step")])
def test_outputs_freed_while_the_current_stream_reads_them(name):
    want = [t.clone() for t in call(name, inputs())]
    args, side = inputs(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = call(name, args, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(CYCLES)
    copies = [t.clone() for t in got]
    del got
    with torch.cuda.stream(side):
        new = [torch.full_like(t, 1) for t in want for _ in range(4)]
    torch.cuda.synchronize()
    assert same(copies, want) and len(new) > 0
