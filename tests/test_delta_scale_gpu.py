"""The gated delta rule's scale of q at both ends of fp32's range."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import causal_conv_backward_gb300 as m  # noqa: E402
from ssm_reference import check, to64  # noqa: E402
from test_delta_gpu import FORMS, cuda_ready, inputs, reference  # noqa: E402,F401

NAMES = ("q", "k", "v", "delta", "beta", "A", "delta_bias", "state")


@pytest.mark.parametrize("S", [9, 70])
@pytest.mark.parametrize("scale", [0.0, 1e-25, 1e-21, 1e-12, 1e12, 1e25])
def test_scales(S, scale):
    B, H, G, K, V = 2, 4, 2, 32, 24
    t, clean, gy, _ = inputs(S, B, H, G, K, V, what="dbs")
    leaves, ry, rf = reference(clean, None, scale=scale)
    args = [t[k] for k in NAMES[:-1]]
    y, final = m.gated_delta(*args, state=t["state"], scale=scale, return_state=True, **FORMS)
    check(y, ry, K + 256, "y")
    check(final, rf, K + 256, "final state")
    got = m.gated_delta_backward(gy, *args, state=t["state"], scale=scale, **FORMS)
    for k, want in zip(NAMES, torch.autograd.grad((ry * to64(gy)).sum(), [leaves[k] for k in NAMES])):
        check(getattr(got, k), want, S * B * 64 if k in ("A", "delta_bias") else K * V + 256, k)


def test_no_keys_are_refused():
    t, _, _, _ = inputs(9, 2, 4, 2, 16, 16)
    q = t["q"][..., :0]
    for call in (lambda: m.gated_delta(q, q, t["v"], t["delta"], t["beta"], t["A"]),
                 lambda: m.gated_delta_backward(t["v"], q, q, t["v"], t["delta"], t["beta"], t["A"]),
                 lambda: m.gated_delta_step(q[0], q[0], t["v"][0], t["delta"][0], t["beta"][0], t["state"][..., :0], t["A"])):
        with pytest.raises(m.Mcc1dError):
            call()
