"""Which stream's memory the calls of the gated delta rule and the norms take and
what they record, on fake tensors (no GPU needed)."""
import pytest

import test_ssm_streams_host as base
from causal_conv_backward_gb300 import _delta, _norm
from test_ssm_streams_host import Stream, fake, outputs  # noqa: F401


class Tensor(base.Tensor):
    def stride(self, i=None):
        n = len(self.shape)
        return tuple(super(Tensor, self).stride(j) for j in range(n)) if i is None else super().stride(i)


@pytest.fixture(autouse=True)
def tensors(monkeypatch):
    monkeypatch.setattr(base, "Tensor", Tensor)


def calls():
    S, B, H, G, K, V, D = 40, 2, 4, 2, 8, 16, 8
    t = lambda *shape, dtype="bf16": Tensor(shape, dtype)  # noqa: E731
    delta = (t(S, B, G, K), t(S, B, G, K), t(S, B, H, V), t(S, B, H), t(S, B, H), t(H, dtype="f32"), t(H, dtype="f32"))
    one = (t(B, G, K), t(B, G, K), t(B, H, V), t(B, H), t(B, H), t(B, H, V, K, dtype="f32"), t(H, dtype="f32"), t(H, dtype="f32"))
    kw = dict(state=t(B, H, V, K, dtype="f32"), lengths=t(B, dtype="i32"))
    norm, row = (t(S, B, H, D), t(S, B, H, D), t(D)), (t(S, B, H), t(S, B, H, dtype="f32"), t(H))
    post = dict(post_weight=t(H), scale=t(H, dtype="f32"))
    return {
        "gated_delta": (_delta.gated_delta, delta, dict(kw, return_state=True)),
        "gated_delta_backward": (_delta.gated_delta_backward, (t(S, B, H, V), *delta), dict(kw, grad_final_state=t(B, H, V, K, dtype="f32"))),
        "gated_delta_step": (_delta.gated_delta_step, one, dict(slots=t(B, dtype="i32"))),
        "gated_norm": (_norm.gated_norm, norm, {}),
        "gated_norm_backward": (_norm.gated_norm_backward, (t(S, B, H, D), *norm), {}),
        "residual_norm": (_norm.residual_norm, row, post),
        "residual_norm_backward": (_norm.residual_norm_backward, (t(S, B, H), t(S, B, H, dtype="f32"), *row), post),
    }


NAMES = list(calls())


@pytest.mark.parametrize("name", NAMES)
def test_memory_comes_from_the_stream_that_writes_it(fake, name):
    f, args, kw = calls()[name]
    side = Stream("side")
    out = outputs(f(*args, stream=side, **kw))
    assert fake.made and all(t.pool is side for t in fake.made)     # outputs and workspace
    assert fake.current is fake.main
    assert out and all(fake.main in t.recorded for t in out)
    tensors = [t for t in (*args, *kw.values()) if isinstance(t, base.Tensor)]
    assert all(side in t.recorded for t in tensors)


@pytest.mark.parametrize("name", NAMES)
def test_current_stream_needs_no_records(fake, name):
    f, args, kw = calls()[name]
    f(*args, **kw)
    assert all(t.pool is fake.main and not t.recorded for t in fake.made)
    assert not any(t.recorded for t in (*args, *kw.values()) if isinstance(t, base.Tensor))


@pytest.mark.parametrize("name", ["gated_delta", "gated_delta_step", "gated_norm", "residual_norm"])
def test_a_given_output_is_recorded_on_the_stream(fake, name):
    f, args, kw = calls()[name]
    like = args[2] if name.startswith("gated_delta") else args[0]
    y, side = Tensor(like.shape, "bf16"), Stream("side")
    assert outputs(f(*args, y=y, stream=side, **kw))[0] is y
    assert side in y.recorded


@pytest.mark.parametrize("name", NAMES)
def test_a_stream_of_another_device_is_refused(fake, name):
    f, args, kw = calls()[name]
    with pytest.raises(ValueError, match="stream is on cuda:1"):
        f(*args, stream=Stream("there", index=1), **kw)
    assert not fake.made and not any(t.recorded for t in args if isinstance(t, base.Tensor))


BAD = [("gated_delta", 3, "delta needs A"), ("gated_delta_step", 6, "delta needs A"), ("gated_delta_backward", 6, "delta needs A")]


@pytest.mark.parametrize("name,at,message", BAD)
def test_a_decay_without_A_is_refused(fake, name, at, message):
    f, args, kw = calls()[name]
    args = list(args)
    args[{"gated_delta": 5, "gated_delta_step": 6, "gated_delta_backward": 6}[name]] = None
    with pytest.raises(ValueError, match=message):
        f(*args, **kw)


@pytest.mark.parametrize("name", NAMES)
def test_wrong_shapes_and_types_are_refused(fake, name):
    f, args, kw = calls()[name]
    for i, t in enumerate(args):
        for other in (Tensor((*t.shape[:-1], t.shape[-1] + 1), t.dtype), Tensor(t.shape, "f64")):
            if i == 0 and other.dtype != "f64":
                continue                    # the leading tensor's shape is the others' measure
            with pytest.raises((ValueError, TypeError)):
                f(*[other if j == i else a for j, a in enumerate(args)], **kw)
