"""Which stream's memory the binding's calls take and what they record, on fake
tensors (no GPU needed)."""
import contextlib
import types

import pytest

from causal_conv_backward_gb300 import _ssm


class Stream:
    def __init__(self, name, index=0):
        self.name, self.device, self.cuda_stream = name, types.SimpleNamespace(index=index), id(self)


class Tensor:
    is_cuda, device = True, "cuda:0"

    def __init__(self, shape, dtype, pool=None):
        self.shape, self.dtype, self.pool, self.recorded = tuple(shape), dtype, pool, []

    def dim(self):
        return len(self.shape)

    def stride(self, i):
        i, n = i % len(self.shape), 1
        for s in self.shape[i + 1:]:
            n *= s
        return n

    def get_device(self):
        return 0

    def is_contiguous(self):
        return True

    def numel(self):
        return self.shape[0] * self.stride(0)

    def element_size(self):
        return 4 if self.dtype == "f32" else 2

    def data_ptr(self):
        return id(self) << 8        # far apart

    def record_stream(self, stream):
        self.recorded.append(stream)


class Lib:
    """Every call succeeds; sizes are 64 bytes."""
    def __getattr__(self, name):
        def call(args, *rest):
            if name.endswith("_workspace_size"):
                rest[0].value = 64
            return 0
        return call


@pytest.fixture
def fake(monkeypatch):
    main = Stream("main")
    f = types.SimpleNamespace(main=main, current=main, made=[])

    def empty(shape, dtype=None, device=None):
        t = Tensor((shape,) if isinstance(shape, int) else shape, dtype, f.current)
        f.made.append(t)
        return t

    @contextlib.contextmanager
    def stream(s):
        before, f.current = f.current, s
        yield
        f.current = before

    cuda = types.SimpleNamespace(stream=stream, current_stream=lambda index=None: f.current)
    torch = types.SimpleNamespace(bfloat16="bf16", float16="fp16", float32="f32", int32="i32", uint8="u8", empty=empty, cuda=cuda)
    for name, value in (("_lib", Lib()), ("_torch", torch), ("_raw_stream", lambda index: f.current.cuda_stream),
                        ("_current_device", lambda: 0)):
        monkeypatch.setattr(_ssm, name, value)
    return f


def calls():
    S, B, H, W, N, G = 6, 2, 8, 4, 4, 1
    t = lambda *shape, dtype="bf16": Tensor(shape, dtype)
    x, w, b, win = t(S, B, H), t(W, H), t(H), t(B, W - 1, H)
    scan = (t(S, B, H), t(H, N, dtype="f32"), t(S, B, G, N), t(S, B, G, N), t(H, dtype="f32"), t(S, B, H), t(H, dtype="f32"))
    one = (t(B, H), t(B, H), t(B, H, N, dtype="f32"), t(H, N, dtype="f32"), t(B, G, N), t(B, G, N), t(H, dtype="f32"), t(B, H),
           t(H, dtype="f32"))
    ln, st = t(B, dtype="i32"), t(B, H, N, dtype="f32")
    return {
        "short_conv": ((x, w, b), dict(state=win, lengths=ln, return_state=True)),
        "short_conv_backward": ((t(S, B, H), x, w, b), dict(state=win, lengths=ln, grad_final_state=t(B, W - 1, H))),
        "short_conv_step": ((t(B, H), win, w, b), dict(slots=t(B, dtype="i32"))),
        "selective_scan": ((x, *scan), dict(state=st, lengths=ln, return_state=True)),
        "selective_scan_backward": ((t(S, B, H), x, *scan), dict(state=st, lengths=ln, grad_final_state=t(B, H, N, dtype="f32"))),
        "selective_scan_step": (one, dict(slots=t(B, dtype="i32"))),
    }


NAMES = list(calls())


def outputs(result):
    return [t for t in (result if isinstance(result, tuple) else (result,)) if t is not None]


@pytest.mark.parametrize("name", NAMES)
def test_memory_comes_from_the_stream_that_writes_it(fake, name):
    """A block of the current stream's pool may still be in use there, and
    nothing orders the given stream after that."""
    args, kw = calls()[name]
    side = Stream("side")
    out = outputs(getattr(_ssm, name)(*args, stream=side, **kw))
    assert fake.made and all(t.pool is side for t in fake.made)     # outputs and workspace
    assert fake.current is fake.main
    # freed by the caller, an output is not reused on `side` before the caller's stream is done with it
    assert out and all(fake.main in t.recorded for t in out)
    # and an input not before `side` is
    tensors = [t for t in (*args, *kw.values()) if isinstance(t, Tensor)]
    assert all(side in t.recorded for t in tensors)


@pytest.mark.parametrize("name", NAMES)
def test_current_stream_needs_no_records(fake, name):
    args, kw = calls()[name]
    getattr(_ssm, name)(*args, **kw)
    assert all(t.pool is fake.main and not t.recorded for t in fake.made)
    assert not any(t.recorded for t in (*args, *kw.values()) if isinstance(t, Tensor))


@pytest.mark.parametrize("name", ["short_conv", "short_conv_step", "selective_scan", "selective_scan_step"])
def test_a_given_output_is_recorded_on_the_stream(fake, name):
    args, kw = calls()[name]
    y, side = Tensor(args[0].shape, "bf16"), Stream("side")
    assert outputs(getattr(_ssm, name)(*args, y=y, stream=side, **kw))[0] is y
    assert side in y.recorded


@pytest.mark.parametrize("name", NAMES)
def test_a_stream_of_another_device_is_refused(fake, name):
    args, kw = calls()[name]
    with pytest.raises(ValueError, match="stream is on cuda:1"):
        getattr(_ssm, name)(*args, stream=Stream("there", index=1), **kw)
    assert not fake.made and not any(t.recorded for t in args if isinstance(t, Tensor))
