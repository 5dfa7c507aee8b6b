"""States of the gated delta rule that fade over thousands of tokens, one at a
time and in chunks."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import causal_conv_backward_gb300 as m  # noqa: E402
from test_delta_gpu import BF16, F32, cuda_ready, rand  # noqa: E402,F401


@pytest.mark.parametrize("rate", [1e-3, 3e-4])
def test_a_state_that_fades_slowly(rate):
    """Nothing is written: what is left of a state is the product of the decays. A
    step rounds a product once, by 2^-24 at most and with no sign of its own:
    its 3000 steps move a value by sqrt(3000) 2^-24 / sqrt(3) of it, 1.9e-6, times
    two for the decays' own last bits."""
    B, H, K, V, steps = 4, 64, 16, 16, 3000
    state = 1 + rand(B, H, V, K, dtype=F32, seed=1).abs()
    start = state.double()
    q = k = rand(B, H, K, seed=2)
    v, beta = torch.zeros(B, H, V, dtype=BF16, device="cuda"), torch.full((B, H), float("-inf"), dtype=BF16, device="cuda")
    A = -rate * (1 + rand(H, dtype=F32, seed=3).abs())
    g, total = torch.Generator(device="cuda").manual_seed(4), torch.zeros(B, H, dtype=torch.float64, device="cuda")
    for _ in range(steps):
        delta = (0.5 + torch.rand(B, H, generator=g, device="cuda")).to(BF16)
        m.gated_delta_step(q, k, v, delta, beta, state, A, beta_sigmoid=True, qk_norm=True)
        total += delta.double() * A.double()
    want = start * torch.exp(total)[..., None, None]
    off = float((state.double() - want).norm() / want.norm())
    along = float(((state.double() - want) * want).sum() / want.square().sum())
    assert off < 4e-6, (off, along)


@pytest.mark.parametrize("rate", [1e-3, 3e-5])
def test_a_state_that_fades_slowly_in_chunks(rate):
    """The same over a prompt: a chunk's decay is rounded, and the state by it, 1024
    times: sqrt(1024) 2^-24 / sqrt(3), 1.1e-6, times two as above, and once more for
    the logarithms' sum of a chunk."""
    S, B, H, K, V = 65536, 1, 8, 16, 16
    state = 1 + rand(B, H, V, K, dtype=F32, seed=1).abs()
    q = k = rand(S, B, 1, K, seed=2)
    v, beta = torch.zeros(S, B, H, V, dtype=BF16, device="cuda"), torch.full((S, B, H), float("-inf"), dtype=BF16, device="cuda")
    A = -rate * (1 + rand(H, dtype=F32, seed=3).abs())
    delta = (0.5 + torch.rand(S, B, H, generator=torch.Generator(device="cuda").manual_seed(4), device="cuda")).to(BF16)
    _, final = m.gated_delta(q, k, v, delta, beta, A, state=state, return_state=True, beta_sigmoid=True, qk_norm=True)
    total = delta.double() * A.double()
    want = state.double() * torch.exp(total.sum(0))[..., None, None]
    head = (final.double() - want).norm(dim=(-1, -2)) / want.norm(dim=(-1, -2))
    # the heads' own chunks may all be rounded to one side (bf16 steps times one A are
    # few different numbers): what is off where nothing but each decay is rounded
    # to fp32 is no fault of the kernel's, and is allowed beside the rest
    decays = torch.exp(total.view(-1, 64, B, H).sum(1))
    rounded = (decays.float().double() / decays).log().sum(0).abs()
    there = want.norm(dim=(-1, -2)) > 1e-30
    assert there.any() and (head < 4.4e-6 + rounded)[there].all(), (head, rounded)
