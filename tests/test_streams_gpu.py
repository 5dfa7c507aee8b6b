"""forward() and backward() on a stream of their own while the current stream
still writes memory that its pool has handed back (a kernel that spins for a
fixed number of cycles keeps it busy)."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import causal_conv_backward_gb300 as m  # noqa: E402
from test_ssm_streams_gpu import CYCLES, cuda_ready, same  # noqa: E402,F401


def inputs(strided):
    S, B, H, W = 256, 2, 384, 3
    g = torch.Generator(device="cuda").manual_seed(0)
    gy, x, w = (torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16) for shape in ((S, B, H), (S, B, H), (W, H)))
    mask = torch.rand(B, S, generator=g, device="cuda") < 0.8
    return (gy, x.repeat(1, 1, 2)[:, :, :H] if strided else x, w, mask)


def call(name, args, **kw):
    out = m.forward(*args[1:], **kw) if name == "forward" else m.backward(*args, **kw)
    return list(out) if isinstance(out, tuple) else [out]


@pytest.mark.parametrize("handle", [False, True])
@pytest.mark.parametrize("strided", [False, True])
@pytest.mark.parametrize("name", ["forward", "backward"])
def test_current_stream_still_writes_freed_memory(name, strided, handle):
    want = [t.clone() for t in call(name, inputs(strided))]
    args, side = inputs(strided), torch.cuda.Stream()
    torch.cuda.synchronize()
    old = [torch.empty_like(t) for t in want for _ in range(4)]
    torch.cuda._sleep(CYCLES)
    for t in old:
        t.fill_(float("nan"))
    del t, old
    got = call(name, args, stream=side.cuda_stream if handle else side)
    torch.cuda.synchronize()
    assert same(got, want)


@pytest.mark.parametrize("strided", [False, True])
@pytest.mark.parametrize("name", ["forward", "backward"])
def test_tensors_freed_while_the_streams_work(name, strided):
    want = [t.clone() for t in call(name, inputs(strided))]
    args, side = inputs(strided), torch.cuda.Stream()
    torch.cuda.synchronize()
    sizes = [(t.shape, t.dtype) for t in args]
    with torch.cuda.stream(side):
        torch.cuda._sleep(CYCLES)
    got = call(name, args, stream=side)
    del args
    new = [torch.full(shape, 1, dtype=dtype, device="cuda") for shape, dtype in sizes for _ in range(4)]
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(CYCLES)
    copies = [t.clone() for t in got]
    del got
    with torch.cuda.stream(side):
        new += [torch.full_like(t, 1) for t in want for _ in range(4)]
    torch.cuda.synchronize()
    assert same(copies, want)
