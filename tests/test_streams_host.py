"""forward() and backward() on a given stream: which stream's memory they take
and what they record, on fake tensors (no GPU needed)."""
import contextlib
import sys
import types

import pytest

from causal_conv_backward_gb300 import _lib
from test_ssm_streams_host import Lib, Stream, Tensor as Base, outputs


class Tensor(Base):
    def stride(self, i=None):
        return tuple(Base.stride(self, k) for k in range(len(self.shape))) if i is None else Base.stride(self, i)


class Strided(Tensor):
    def is_contiguous(self):
        return False


class AnyLib(Lib):
    """As Lib; a size goes to the last argument, which is by reference."""
    def __getattr__(self, name):
        def call(*args):
            if name.endswith("_workspace_size"):
                args[-1]._obj.value = 64
            return 0
        return call


@pytest.fixture
def fake(monkeypatch):
    f = types.SimpleNamespace(main=Stream("main"), made=[])
    f.current = f.main

    def empty(shape, dtype=None, device=None):
        f.made.append(Tensor((shape,) if isinstance(shape, int) else shape, dtype, f.current))
        return f.made[-1]

    @contextlib.contextmanager
    def stream(s):
        before, f.current = f.current, s
        yield
        f.current = before

    f.handles = {}
    cuda = types.SimpleNamespace(stream=stream, current_stream=lambda device=None: f.current, Stream=Stream,
                                 ExternalStream=lambda h, device=None: f.handles[h], default_stream=lambda device=None: f.main)
    torch = types.SimpleNamespace(empty=empty, cuda=cuda, uint8="u8", bool="bool")
    monkeypatch.setitem(sys.modules, "torch", torch)
    monkeypatch.setattr(_lib, "load", AnyLib)
    return f


def call(name, cls):
    S, B, H = 8, 2, 64
    x, w, mask, gy = cls((S, B, H), "bf16"), Tensor((3, H), "bf16"), Tensor((B, S), "u8"), Tensor((S, B, H), "bf16")
    return (_lib.forward, (x, w, mask)) if name == "forward" else (_lib.backward, (gy, x, w, mask))


@pytest.mark.parametrize("cls", [Tensor, Strided])
@pytest.mark.parametrize("name", ["forward", "backward"])
@pytest.mark.parametrize("handle", [False, True])
def test_memory_comes_from_the_stream_that_writes_it(fake, name, cls, handle):
    f, args = call(name, cls)
    side = Stream("side")
    fake.handles[side.cuda_stream] = side
    out = outputs(f(*args, stream=side.cuda_stream if handle else side))
    assert fake.made and all(t.pool is side for t in fake.made)
    assert all(fake.main in t.recorded for t in out)
    assert all(side in t.recorded for t in args)


@pytest.mark.parametrize("name", ["forward", "backward"])
def test_current_stream_needs_no_records(fake, name):
    f, args = call(name, Tensor)
    f(*args)
    assert all(t.pool is fake.main and not t.recorded for t in fake.made)
    assert not any(t.recorded for t in args)
