"""The example's operators have first derivatives only: asking for a second one
is an error, not a zero."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_ssm_example_gpu import example  # noqa: E402,F401


def rand(*shape, dtype=torch.bfloat16):
    return torch.randn(shape, device="cuda").to(dtype)


def test_second_derivatives_are_refused(example):
    S, B, H, N = 12, 2, 16, 4
    x, f32 = rand(S, B, H).requires_grad_(), torch.float32
    conv = example.ShortConv.apply(x, rand(4, H), rand(H))
    scan = example.SelectiveScan.apply(x, rand(S, B, H), -torch.exp(rand(H, N, dtype=f32)), rand(S, B, 1, N), rand(S, B, 1, N),
                                       rand(H, dtype=f32), rand(S, B, H), rand(H, dtype=f32))
    for y in (conv, scan):
        loss = y.float().square().sum() + x.float().square().sum()      # x itself has a second derivative
        first, = torch.autograd.grad(loss, x, create_graph=True)
        with pytest.raises(RuntimeError, match="once_differentiable"):
            first.float().square().sum().backward()
