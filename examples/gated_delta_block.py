"""Blocks whose sequence mixer is the gated delta rule, behind the library's short
convolution and between its norms: trained, run over prompts of unequal lengths,
and continued token by token.

    python examples/gated_delta_block.py

    h, y   = residual stream, and what a block reads of it   (residual_norm)
    q,k,v  = short convolution of projections of y           (short_conv)
    o      = gated delta rule of q, k, v                     (gated_delta)
    branch = projection of o / rms(o) weight silu(z)         (gated_norm)

The projections are torch matrix products; everything between them is the
library's. A sequence's cache is the convolution's window and the heads' states.
"""
import math
import os
import sys

import torch
from torch.autograd.function import once_differentiable

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))

import causal_conv_backward_gb300 as mcc  # noqa: E402
from selective_block import ShortConv  # noqa: E402

FORMS = dict(delta_softplus=True, beta_sigmoid=True, qk_norm=True)


class GatedDelta(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, delta, beta, A, delta_bias):
        ctx.save_for_backward(q, k, v, delta, beta, A, delta_bias)
        return mcc.gated_delta(q, k, v, delta, beta, A, delta_bias, **FORMS)

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_y):
        g = mcc.gated_delta_backward(grad_y.contiguous(), *ctx.saved_tensors, **FORMS)
        return g.q, g.k, g.v, g.delta, g.beta, g.A, g.delta_bias


class GatedNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, z, weight):
        ctx.save_for_backward(x, z, weight)
        return mcc.gated_norm(x, z, weight)

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_y):
        return tuple(mcc.gated_norm_backward(grad_y.contiguous(), *ctx.saved_tensors))


class ResidualNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, residual, weight, post_weight, scale):
        ctx.save_for_backward(x, residual, weight, post_weight, scale)
        return mcc.residual_norm(x, residual, weight, post_weight=post_weight, scale=scale)

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_y, grad_h):
        x, residual, weight, post_weight, scale = ctx.saved_tensors
        g = mcc.residual_norm_backward(grad_y.contiguous(), grad_h.contiguous(), x, residual, weight, post_weight=post_weight,
                                       scale=scale)
        return g.x, g.residual, g.weight, g.post_weight, g.scale


class GatedDeltaBlock(torch.nn.Module):
    """What a block adds to the residual stream: y [S,B,width] -> [S,B,width]."""

    def __init__(self, width, *, heads=4, key_heads=2, K=32, V=32, taps=4, dtype=torch.bfloat16, device="cuda"):
        super().__init__()
        self.H, self.G, self.K, self.V, self.W = heads, key_heads, K, V, taps
        self.channels = 2 * key_heads * K + heads * V          # of q, k and v, which the convolution takes together

        def linear(i, o):
            return torch.nn.Linear(i, o, bias=False, dtype=dtype, device=device)

        self.in_proj = linear(width, self.channels + heads * V + 2 * heads)
        self.out_proj = linear(heads * V, width)
        self.conv_weight = torch.nn.Parameter((torch.rand(taps, self.channels, device=device) * 2 - 1).mul_(taps ** -0.5).to(dtype))
        self.norm_weight = torch.nn.Parameter(torch.ones(V, dtype=dtype, device=device))
        step = torch.exp(torch.rand(heads, device=device) * math.log(100.0) + math.log(1e-3))
        self.delta_bias = torch.nn.Parameter(step + torch.log(-torch.expm1(-step)))
        self.A_log = torch.nn.Parameter(torch.log(1 + 15 * torch.rand(heads, device=device)))

    def _split(self, y):
        """q, k, v side by side, the output gate [..,H,V], delta and beta [..,H]."""
        qkv, z, delta, beta = self.in_proj(y).split([self.channels, self.H * self.V, self.H, self.H], dim=-1)
        return qkv, z.unflatten(-1, (self.H, self.V)), delta, beta

    def _heads(self, qkv):
        q, k, v = qkv.split([self.G * self.K, self.G * self.K, self.H * self.V], dim=-1)
        return q.unflatten(-1, (self.G, self.K)), k.unflatten(-1, (self.G, self.K)), v.unflatten(-1, (self.H, self.V))

    def forward(self, y):
        qkv, z, delta, beta = self._split(y)
        q, k, v = self._heads(ShortConv.apply(qkv, self.conv_weight, None))
        o = GatedDelta.apply(q, k, v, delta, beta, -torch.exp(self.A_log), self.delta_bias)
        return self.out_proj(GatedNorm.apply(o, z, self.norm_weight).flatten(-2))

    def cache(self, rows):
        """Windows and states of `rows` sequences that have not begun."""
        p = self.conv_weight
        return (torch.zeros(rows, self.W - 1, self.channels, dtype=p.dtype, device=p.device),
                torch.zeros(rows, self.H, self.V, self.K, dtype=torch.float32, device=p.device))

    def prompt(self, y, cache=None, lengths=None):
        """Whole prompts (sequence b ending after lengths[b] tokens), and the cache they leave behind."""
        window, state = cache if cache is not None else (None, None)
        qkv, z, delta, beta = self._split(y)
        qkv, window = mcc.short_conv(qkv, self.conv_weight, lengths=lengths, state=window, return_state=True)
        o, state = mcc.gated_delta(*self._heads(qkv), delta, beta, -torch.exp(self.A_log), self.delta_bias, lengths=lengths,
                                   state=state, return_state=True, **FORMS)
        return self.out_proj(mcc.gated_norm(o, z, self.norm_weight).flatten(-2)), (window, state)

    def step(self, y, cache, slots=None):
        """One token per sequence (y [B,width]); the cache moves on in place."""
        window, state = cache
        qkv, z, delta, beta = self._split(y)
        qkv = mcc.short_conv_step(qkv, window, self.conv_weight, slots=slots)
        o = mcc.gated_delta_step(*self._heads(qkv), delta, beta, state, -torch.exp(self.A_log), self.delta_bias, slots=slots, **FORMS)
        return self.out_proj(mcc.gated_norm(o, z, self.norm_weight).flatten(-2))


class GatedDeltaStack(torch.nn.Module):
    """Blocks on an fp32 residual stream, each one's output normed and scaled
    before it is added: x [S,B,width] -> [S,B,width]."""

    def __init__(self, width, layers=2, *, dtype=torch.bfloat16, device="cuda", **kw):
        super().__init__()
        self.blocks = torch.nn.ModuleList(GatedDeltaBlock(width, dtype=dtype, device=device, **kw) for _ in range(layers))
        ones = lambda: torch.nn.Parameter(torch.ones(width, dtype=dtype, device=device))  # noqa: E731
        self.pre = torch.nn.ParameterList(ones() for _ in range(layers + 1))
        self.post = torch.nn.ParameterList(ones() for _ in range(layers))
        self.scale = torch.nn.ParameterList(torch.nn.Parameter(torch.full((width,), 0.5, device=device)) for _ in range(layers))

    def forward(self, x):
        h = x.float()
        y = GatedNorm.apply(x, None, self.pre[0])
        for block, post, scale, pre in zip(self.blocks, self.post, self.scale, list(self.pre)[1:]):
            y, h = ResidualNorm.apply(block(y), h, pre, post, scale)
        return y

    def cache(self, rows):
        return [b.cache(rows) for b in self.blocks]

    @torch.no_grad()
    def prompt(self, x, caches=None, lengths=None):
        h, y, after = x.float(), mcc.gated_norm(x, None, self.pre[0]), []
        for n, block in enumerate(self.blocks):
            out, cache = block.prompt(y, caches[n] if caches is not None else None, lengths)
            after.append(cache)
            y, h = mcc.residual_norm(out, h, self.pre[n + 1], post_weight=self.post[n], scale=self.scale[n])
        return y, after

    @torch.no_grad()
    def step(self, x, caches, slots=None):
        h, y = x.float(), mcc.gated_norm(x, None, self.pre[0])
        for n, block in enumerate(self.blocks):
            y, h = mcc.residual_norm(block.step(y, caches[n], slots), h, self.pre[n + 1], post_weight=self.post[n], scale=self.scale[n])
        return y


def train(stack, steps=40, S=64, B=8, lag=2, lr=3e-3):
    """Learns to give back its input of `lag` tokens ago; returns the losses."""
    g = torch.Generator(device="cuda").manual_seed(0)
    width = stack.pre[0].shape[0]
    opt = torch.optim.Adam(stack.parameters(), lr=lr)
    losses = []
    for _ in range(steps):
        x = torch.randn(S, B, width, generator=g, device="cuda").to(torch.bfloat16)
        loss = (stack(x)[lag:].float() - x[:-lag].float()).square().mean()
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(loss.detach())
    return [float(v) for v in losses]


def continue_prompts(stack, S=70, B=4, new=6):
    """The largest difference between running whole sequences at once and their
    prompts first, token by token after, relative to the outputs' size."""
    g = torch.Generator(device="cuda").manual_seed(1)
    width = stack.pre[0].shape[0]
    lengths = torch.tensor([S - new, 7, 1, 0][:B], dtype=torch.int32, device="cuda")
    x = torch.randn(S, B, width, generator=g, device="cuda").to(torch.bfloat16)
    whole, _ = stack.prompt(x)
    _, caches = stack.prompt(x[:S - new], lengths=lengths)
    rows, worst = torch.arange(B, device="cuda"), 0.0
    for i in range(new):
        at = (lengths + i).long()
        y = stack.step(x[at, rows], caches)
        worst = max(worst, float((y.float() - whole[at, rows].float()).abs().max()))
    return worst / float(whole.float().abs().max())


def main():
    torch.manual_seed(0)
    stack = GatedDeltaStack(64)
    losses = train(stack)
    print(f"loss: {losses[0]:.3f} after 1 step, {losses[-1]:.3f} after {len(losses)}")
    print(f"prompts continued token by token against whole sequences: {continue_prompts(stack):.2e} of the largest output")


if __name__ == "__main__":
    main()
