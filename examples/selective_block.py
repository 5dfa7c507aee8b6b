"""A selective state space block on the library's short convolution and selective
scan: trained, run over prompts of unequal lengths, and continued token by token.

    python examples/selective_block.py

The projections are torch matrix products; everything between them is the
library's. One state per sequence (the convolution's window and the scan's
state) carries a sequence from a prompt to single tokens.
"""
import math
import os
import sys

import torch
from torch.autograd.function import once_differentiable

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import causal_conv_backward_gb300 as mcc  # noqa: E402


class ShortConv(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias):
        ctx.save_for_backward(x, weight, bias)
        return mcc.short_conv(x, weight, bias)

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_y):
        g = mcc.short_conv_backward(grad_y.contiguous(), *ctx.saved_tensors)
        return g.x, g.weight, g.bias


class SelectiveScan(torch.autograd.Function):
    @staticmethod
    def forward(ctx, u, delta, A, B, C, D, z, delta_bias):
        ctx.save_for_backward(u, delta, A, B, C, D, z, delta_bias)
        return mcc.selective_scan(u, delta, A, B, C, D, z, delta_bias, delta_softplus=True)

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_y):
        g = mcc.selective_scan_backward(grad_y.contiguous(), *ctx.saved_tensors, delta_softplus=True)
        return g.u, g.delta, g.A, g.B, g.C, g.D, g.z, g.delta_bias


class SelectiveBlock(torch.nn.Module):
    """x [S,B,width] -> [S,B,width]; channels = expand * width."""

    def __init__(self, width, *, expand=2, states=16, taps=4, rank=None, dtype=torch.bfloat16, device="cuda"):
        super().__init__()
        H, N = expand * width, states
        R = rank or math.ceil(width / 16)
        self.H, self.N, self.R, self.W = H, N, R, taps

        def linear(i, o):
            return torch.nn.Linear(i, o, bias=False, dtype=dtype, device=device)

        self.in_proj, self.x_proj, self.dt_proj, self.out_proj = linear(width, 2 * H), linear(H, R + 2 * N), linear(R, H), linear(H, width)
        self.conv_weight = torch.nn.Parameter((torch.rand(taps, H, device=device) * 2 - 1).mul_(taps ** -0.5).to(dtype))
        self.conv_bias = torch.nn.Parameter(torch.zeros(H, dtype=dtype, device=device))
        step = torch.exp(torch.rand(H, device=device) * math.log(100.0) + math.log(1e-3))
        self.delta_bias = torch.nn.Parameter(step + torch.log(-torch.expm1(-step)))
        self.A_log = torch.nn.Parameter(torch.arange(1, N + 1, dtype=torch.float32, device=device).log().repeat(H, 1))
        self.D = torch.nn.Parameter(torch.ones(H, device=device))

    def _split(self, u):
        """delta [..,H] and B, C [..,1,N] of the convolved input."""
        dt, B, C = self.x_proj(u).split([self.R, self.N, self.N], dim=-1)
        return self.dt_proj(dt), B.unsqueeze(-2), C.unsqueeze(-2)

    def forward(self, x):
        x, z = self.in_proj(x).chunk(2, dim=-1)
        u = ShortConv.apply(x, self.conv_weight, self.conv_bias)
        delta, B, C = self._split(u)
        y = SelectiveScan.apply(u, delta, -torch.exp(self.A_log), B, C, self.D, z, self.delta_bias)
        return self.out_proj(y)

    def cache(self, rows):
        """Windows and states of `rows` sequences that have not begun."""
        p = self.conv_weight
        return (torch.zeros(rows, self.W - 1, self.H, dtype=p.dtype, device=p.device),
                torch.zeros(rows, self.H, self.N, dtype=torch.float32, device=p.device))

    @torch.no_grad()
    def prompt(self, x, cache=None, lengths=None):
        """Outputs of whole prompts (x [S,B,width], sequence b ending after
        lengths[b] tokens) and the cache they leave behind."""
        window, state = cache if cache is not None else (None, None)
        x, z = self.in_proj(x).chunk(2, dim=-1)
        u, window = mcc.short_conv(x, self.conv_weight, self.conv_bias, lengths=lengths, state=window, return_state=True)
        delta, B, C = self._split(u)
        y, state = mcc.selective_scan(u, delta, -torch.exp(self.A_log), B, C, self.D, z, self.delta_bias,
                                      delta_softplus=True, lengths=lengths, state=state, return_state=True)
        return self.out_proj(y), (window, state)

    @torch.no_grad()
    def step(self, x, cache, slots=None):
        """One token per sequence (x [B,width]); the cache moves on in place."""
        window, state = cache
        x, z = self.in_proj(x).chunk(2, dim=-1)
        u = mcc.short_conv_step(x, window, self.conv_weight, self.conv_bias, slots=slots)
        delta, B, C = self._split(u)
        y = mcc.selective_scan_step(u, delta, state, -torch.exp(self.A_log), B, C, self.D, z, self.delta_bias,
                                    delta_softplus=True, slots=slots)
        return self.out_proj(y)


def train(block, steps=60, S=64, B=16, lag=2, lr=1e-2):
    """Learns to give back its input of `lag` tokens ago; returns the losses."""
    g = torch.Generator(device="cuda").manual_seed(0)
    width = block.in_proj.in_features
    opt = torch.optim.Adam(block.parameters(), lr=lr)
    losses = []
    for _ in range(steps):
        x = torch.randn(S, B, width, generator=g, device="cuda").to(torch.bfloat16)
        out = block(x)
        loss = (out[lag:].float() - x[:-lag].float()).square().mean()
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(loss.detach())
    return [float(v) for v in losses]


def continue_prompts(block, S=48, B=4, new=6):
    """The largest difference between running whole sequences at once and their
    prompts first, token by token after, relative to the outputs' size."""
    g = torch.Generator(device="cuda").manual_seed(1)
    width = block.in_proj.in_features
    lengths = torch.tensor([S - new, 7, 1, 0][:B], dtype=torch.int32, device="cuda")
    x = torch.randn(S, B, width, generator=g, device="cuda").to(torch.bfloat16)
    whole, _ = block.prompt(x)
    _, cache = block.prompt(x[:S - new], lengths=lengths)
    rows, worst = torch.arange(B, device="cuda"), 0.0
    for i in range(new):
        at = (lengths + i).long()
        y = block.step(x[at, rows], cache)
        worst = max(worst, float((y.float() - whole[at, rows].float()).abs().max()))
    return worst / float(whole.float().abs().max())


def main():
    torch.manual_seed(0)
    block = SelectiveBlock(64)
    losses = train(block)
    print(f"loss: {losses[0]:.3f} after 1 step, {losses[-1]:.3f} after {len(losses)}")
    print(f"prompts continued token by token against whole sequences: {continue_prompts(block):.2e} of the largest output")


if __name__ == "__main__":
    main()
