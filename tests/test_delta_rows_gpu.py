"""Rows of the gated delta rule's states are independent of one another: values of
V that are quieter than others by many powers of two, in v, the state or the
gradients, keep their own bits."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import causal_conv_backward_gb300 as m  # noqa: E402
from ssm_reference import to64  # noqa: E402
from test_delta_gpu import BF16, FORMS, cuda_ready, inputs, reference  # noqa: E402,F401
from test_delta_range_gpu import near  # noqa: E402


def of_row(want):
    """A row's own size: its largest value over the tokens (or keys)."""
    return want.detach().abs().amax(0, keepdim=True)


@pytest.mark.parametrize("S", [20, 64, 200])
@pytest.mark.parametrize("K,V", [(32, 24), (128, 200)])
@pytest.mark.parametrize("step", [-1.0, -3.0])
def test_quiet_rows(S, K, V, step):
    """Row v is 2^(step v) of the first, down to 2^-72, in a shuffled order."""
    B, H, G = 2, 2, 1
    t, clean, gy, gf = inputs(S, B, H, G, K, V)
    by = 2.0 ** (step * torch.arange(V, device="cuda").remainder(24).float())
    by = by[torch.randperm(V, generator=torch.Generator().manual_seed(0)).cuda()]
    for d in (t, clean):
        d["v"], d["state"] = (d["v"].float() * by).to(BF16), d["state"] * by[:, None]
    gy, gf = (gy.float() * by).to(BF16), gf * by[:, None]
    leaves, ry, rf = reference(clean, None)
    args = [t[k] for k in ("q", "k", "v", "delta", "beta", "A", "delta_bias")]
    y, final = m.gated_delta(*args, state=t["state"], return_state=True, **FORMS)
    near(y, ry, K + 256, of_row(ry), "y")
    near(final, rf, K + 256, rf.detach().abs().amax(-1, keepdim=True), "final state")
    got = m.gated_delta_backward(gy, *args, state=t["state"], grad_final_state=gf, **FORMS)
    gv, gs = torch.autograd.grad((ry * to64(gy)).sum() + (rf * to64(gf)).sum(), [leaves["v"], leaves["state"]])
    near(got.v, gv, K + 256, of_row(gv), "grad v")
    near(got.state, gs, K + 256, gs.abs().amax(-1, keepdim=True), "grad state")
