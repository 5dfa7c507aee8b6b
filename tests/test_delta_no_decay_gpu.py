"""The gated delta rule without delta: A and delta_bias may be given, change
nothing, and have gradients of zero."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import causal_conv_backward_gb300 as m  # noqa: E402
from test_delta_gpu import FORMS, cuda_ready, inputs  # noqa: E402,F401


@pytest.mark.parametrize("S", [9, 70])
@pytest.mark.parametrize("given", [("A",), ("delta_bias",), ("A", "delta_bias")])
@pytest.mark.parametrize("own_stream", [False, True])
def test_what_no_decay_reads(S, given, own_stream):
    t, _, gy, _ = inputs(S, 2, 4, 2, 16, 16)
    args, more = [t[k] for k in ("q", "k", "v")] + [None, t["beta"]], {k: t[k] for k in given}
    want_y, want = m.gated_delta(*args, **FORMS), m.gated_delta_backward(gy, *args, **FORMS)
    step = [x if x is None else x[0] for x in args]
    state = torch.zeros(2, 4, 16, 16, device="cuda"), torch.zeros(2, 4, 16, 16, device="cuda")
    torch.cuda.synchronize()
    stream = torch.cuda.Stream() if own_stream else None
    y, got = m.gated_delta(*args, **more, **FORMS, stream=stream), m.gated_delta_backward(gy, *args, **more, **FORMS, stream=stream)
    steps = m.gated_delta_step(*step, state[0], **FORMS), m.gated_delta_step(*step, state[1], **more, **FORMS, stream=stream)
    torch.cuda.synchronize()
    assert torch.equal(y, want_y) and torch.equal(*steps) and torch.equal(*state)
    for k in got._fields:
        g = getattr(got, k)
        if k in given:
            assert g.shape == t[k].shape and g.dtype is torch.float32 and not g.any()
        elif getattr(want, k) is None:
            assert g is None
        else:
            assert torch.equal(g, getattr(want, k)), k
