"""The blocks of examples/gated_delta_block.py: they train, their gradients are
those of the same blocks in plain float64 torch, and prompts of unequal lengths
continue token by token."""
import os
import sys

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import delta_reference  # noqa: E402
import norm_reference  # noqa: E402
import ssm_reference as ref  # noqa: E402

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from causal_conv_backward_gb300 import build
    build.build()
    import gated_delta_block
    return gated_delta_block


def test_trains(example):
    torch.manual_seed(0)
    losses = example.train(example.GatedDeltaStack(32), steps=5, S=40, B=4)
    assert all(v == v and v < float("inf") for v in losses)


def test_prompts_continue_token_by_token(example):
    torch.manual_seed(0)
    # two blocks, each with some eight bf16 roundings between the two ways, 2^-8 of a value
    assert example.continue_prompts(example.GatedDeltaStack(32)) < 16 * 2.0 ** -8


def test_gradients(example):
    """Against the blocks in float64 from the operators' definitions. What they
    round to bf16 between their parts is not rounded there, so whole gradients
    are compared, to a few roundings (2^-8 each, at some ten places of a block)
    of their norm."""
    torch.manual_seed(0)
    S, B, width = 20, 2, 16
    stack = example.GatedDeltaStack(width, layers=1, heads=4, key_heads=2, K=16, V=24)
    x = torch.randn(S, B, width, device="cuda").to(torch.bfloat16)
    w = torch.randn(S, B, width, device="cuda")
    (stack(x).float() * w).sum().backward()

    p = {k: ref.to64(v, grad=True) for k, v in stack.named_parameters()}
    block = stack.blocks[0]
    x6 = ref.to64(x)
    y = norm_reference.rms(x6, 1e-6) * p["pre.0"]
    qkv, z, delta, beta = (y @ p["blocks.0.in_proj.weight"].T).split([block.channels, block.H * block.V, block.H, block.H], dim=-1)
    qkv, _ = ref.conv(qkv, p["blocks.0.conv_weight"])
    q, k, v = block._heads(qkv)
    o, _ = delta_reference.delta_rule(q, k, v, delta, beta, -torch.exp(p["blocks.0.A_log"]), p["blocks.0.delta_bias"])
    o = norm_reference.gated(o, z.unflatten(-1, (block.H, block.V)), p["blocks.0.norm_weight"], 1e-6)
    out, _ = norm_reference.residual(o.flatten(-2) @ p["blocks.0.out_proj.weight"].T, x6, p["pre.1"], p["post.0"], p["scale.0"])
    (out * ref.to64(w)).sum().backward()
    for k, v in stack.named_parameters():
        off = (ref.to64(v.grad) - p[k].grad).norm() / p[k].grad.norm()
        assert off < 10 * 2.0 ** -8, (k, float(off))
