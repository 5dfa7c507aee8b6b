"""The selective block of examples/selective_block.py: it learns, its gradients
are those of the same block in plain float64 torch, and prompts of unequal
lengths continue token by token."""
import os
import sys

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import ssm_reference as ref  # noqa: E402

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from causal_conv_backward_gb300 import build
    build.build()
    import selective_block
    return selective_block


def test_learns(example):
    torch.manual_seed(0)
    losses = example.train(example.SelectiveBlock(32), steps=40, S=32, B=8)
    assert losses[-1] < 0.9 * losses[0]


def test_prompts_continue_token_by_token(example):
    torch.manual_seed(0)
    # a handful of bf16 roundings between the two ways, each 2^-8 of a value
    assert example.continue_prompts(example.SelectiveBlock(32)) < 16 * 2.0 ** -8


def test_gradients_of_the_block(example):
    """Against the block in float64 from the operators' definitions. What the
    block rounds to bf16 between its parts is not rounded there, so whole
    gradients are compared, to a few roundings (2^-8 each) of their norm."""
    torch.manual_seed(0)
    block = example.SelectiveBlock(16, states=8)
    x = torch.randn(20, 2, 16, device="cuda").to(torch.bfloat16)
    w = torch.randn(20, 2, 16, device="cuda")
    (block(x).float() * w).sum().backward()

    p = {k: ref.to64(v, grad=True) for k, v in block.named_parameters()}
    h, z = (ref.to64(x) @ p["in_proj.weight"].T).chunk(2, dim=-1)
    u, _ = ref.conv(h, p["conv_weight"], p["conv_bias"])
    dt, B, C = (u @ p["x_proj.weight"].T).split([block.R, block.N, block.N], dim=-1)
    y, _ = ref.scan(u, dt @ p["dt_proj.weight"].T, -torch.exp(p["A_log"]), B.unsqueeze(-2), C.unsqueeze(-2), p["D"], z,
                    p["delta_bias"])
    ((y @ p["out_proj.weight"].T) * ref.to64(w)).sum().backward()
    for k, v in block.named_parameters():
        off = (ref.to64(v.grad) - p[k].grad).norm() / p[k].grad.norm()
        assert off < 8 * 2.0 ** -8, (k, float(off))
