"""A small hybrid language-model stack on this library's operators: blocks of gated long convolution and blocks of linear
attention with rotary positions, each behind a layer norm, with plain torch products for the projections.

    python examples/hybrid_block.py            # a few training steps, then a prompt and single tokens from its state

The autograd functions below are all that is needed to train through the operators."""
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from fft_long_convolution_amd import lconv  # noqa: E402

once = torch.autograd.function.once_differentiable     # the gradients have no gradient of their own: asking for one is an error


def rows(t):
    """A gradient as the calls take it: strided, but with contiguous rows (a sum's gradient is one element, repeated)."""
    return t if t.stride(-1) == 1 or t.shape[-1] == 1 else t.contiguous()


class LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias):
        y, mean, rstd = lconv.layer_norm(x, weight, bias)
        ctx.save_for_backward(x, weight, mean, rstd)
        return y

    @staticmethod
    @once
    def backward(ctx, dy):
        x, weight, mean, rstd = ctx.saved_tensors
        dx, dw, db = lconv.layer_norm_bwd(dy.contiguous(), x, weight, mean, rstd)
        return dx, dw.to(weight.dtype), db.to(weight.dtype)


class Rotary(torch.autograd.Function):
    """q and k of [B, heads, N, D], turned together."""

    @staticmethod
    def forward(ctx, q, k, positions, inv_freq):
        ctx.save_for_backward(positions, inv_freq)
        return lconv.rotary(q, k, positions, inv_freq)

    @staticmethod
    @once
    def backward(ctx, dq, dk):
        dq, dk = lconv.rotary(rows(dq), rows(dk), *ctx.saved_tensors, inverse=True)
        return dq, dk, None, None


class LinearAttention(torch.autograd.Function):
    """y and the state after the last token, from a state or none; either result may be used, and each state has its gradient."""

    @staticmethod
    def forward(ctx, q, k, v, log_decay, lengths, state):
        y, last = lconv.linear_attention(q, k, v, log_decay, state=state, lengths=lengths)
        ctx.save_for_backward(q, k, v, log_decay, lengths, state)
        ctx.set_materialize_grads(False)
        return y, last

    @staticmethod
    @once
    def backward(ctx, dy, dlast):
        q, k, v, log_decay, lengths, state = ctx.saved_tensors
        dy = torch.zeros(q.shape[:-1] + v.shape[-1:], dtype=q.dtype, device=q.device) if dy is None else rows(dy)
        g = lconv.linear_attention_bwd(dy, q, k, v, log_decay, state=state, dstate=None if dlast is None else dlast.contiguous(),
                                       lengths=lengths, need_dlog_decay=ctx.needs_input_grad[3])
        return g.dq, g.dk, g.dv, g.dlog_decay, None, g.dstate


class LongConv(torch.autograd.Function):
    """v * ((k * (q u)) + D (q u)) over rows [B, H, N]."""

    @staticmethod
    def forward(ctx, u, k, D, q, v):
        k_f = lconv.filter_fft(k)
        ctx.save_for_backward(u, k_f, D, q, v)
        return lconv.fftconv(u, k_f, D, q=q, v=v)

    @staticmethod
    @once
    def backward(ctx, dy):
        u, k_f, D, q, v = ctx.saved_tensors
        du, dq, dv, dk, dD = lconv.fftconv_bwd(dy.contiguous(), u, k_f, D, q=q, v=v)
        return du, dk.to(D.dtype), dD.to(D.dtype), dq, dv


class AttentionBlock(torch.nn.Module):
    def __init__(self, width, heads, shared, rot, dtype):
        super().__init__()
        self.heads, self.shared, self.D = heads, shared, width // heads
        p = lambda *shape: torch.nn.Parameter((torch.randn(shape) / math.sqrt(shape[-1])).to("cuda", dtype))  # noqa: E731
        self.norm_w = torch.nn.Parameter(torch.ones(width, device="cuda", dtype=dtype))
        self.norm_b = torch.nn.Parameter(torch.zeros(width, device="cuda", dtype=dtype))
        self.inp = p((heads + 2 * shared) * self.D, width)
        self.out = p(width, width)
        # memories from a few tokens to a few hundred
        self.decay = torch.nn.Parameter(torch.linspace(-0.5, -5.0, heads, device="cuda"))
        self.inv_freq, _ = lconv.rotary_frequencies(rot)

    def log_decay(self):
        return -self.decay.exp()

    def project(self, x):
        """q, k, v of x [B, N, width] as slices of one product: [B, heads, N, D] views, read where they are."""
        B, N, _ = x.shape
        h = (LayerNorm.apply(x, self.norm_w, self.norm_b) @ self.inp.t()).view(B, N, self.heads + 2 * self.shared, self.D)
        return (t.transpose(1, 2) for t in h.split((self.heads, self.shared, self.shared), dim=2))

    def forward(self, x, positions, lengths=None, state=None):
        q, k, v = self.project(x)
        q, k = Rotary.apply(q, k, positions, self.inv_freq)
        y, state = LinearAttention.apply(q, k, v, self.log_decay(), lengths, state)
        return x + y.transpose(1, 2).reshape(x.shape) @ self.out.t(), state

    def step(self, x, positions, state, slots=None):
        """One token of every sequence: x [B, width], positions [B]; the states move on in place."""
        q, k, v = self.project(x[:, None])
        q, k = lconv.rotary(q, k, positions[:, None], self.inv_freq)
        y = lconv.linear_attention_step(q[:, :, 0], k[:, :, 0], v[:, :, 0], self.log_decay(), state, slots=slots)
        return x + y.reshape(x.shape) @ self.out.t()


class ConvBlock(torch.nn.Module):
    def __init__(self, width, N, dtype):
        super().__init__()
        p = lambda *shape: torch.nn.Parameter((torch.randn(shape) / math.sqrt(shape[-1])).to("cuda", dtype))  # noqa: E731
        self.norm_w = torch.nn.Parameter(torch.ones(width, device="cuda", dtype=dtype))
        self.norm_b = torch.nn.Parameter(torch.zeros(width, device="cuda", dtype=dtype))
        self.inp, self.out = p(3 * width, width), p(width, width)
        taps = torch.randn(width, N) * torch.exp(-torch.arange(N) / 64.0)
        self.k = torch.nn.Parameter((taps / 8).to("cuda", dtype))
        self.D = torch.nn.Parameter(torch.ones(width, device="cuda", dtype=dtype))

    def forward(self, x):
        h = LayerNorm.apply(x, self.norm_w, self.norm_b) @ self.inp.t()
        u, q, v = (t.transpose(1, 2).contiguous() for t in h.chunk(3, dim=-1))
        return x + LongConv.apply(u, self.k, self.D, q, v).transpose(1, 2) @ self.out.t()


class Hybrid(torch.nn.Module):
    def __init__(self, width=256, heads=4, shared=2, N=512, dtype=torch.bfloat16):
        super().__init__()
        self.conv = ConvBlock(width, N, dtype)
        self.attention = AttentionBlock(width, heads, shared, (width // heads) // 2, dtype)

    def forward(self, x, positions):
        return self.attention(self.conv(x), positions)[0]


def train(steps=8, B=2, N=512, width=256, dtype=torch.bfloat16, seed=0):
    """Fits a running mean of the input's past; returns the losses."""
    torch.manual_seed(seed)
    model = Hybrid(width=width, N=N, dtype=dtype)
    opt = torch.optim.Adam(model.parameters(), lr=3e-3)
    x = torch.randn(B, N, width, device="cuda").to(dtype)
    target = (x.float().cumsum(1) / torch.arange(1, N + 1, device="cuda")[:, None]).to(dtype)
    positions = torch.arange(N, dtype=torch.int32, device="cuda")
    losses = []
    for _ in range(steps):
        opt.zero_grad()
        loss = (model(x, positions) - target).float().square().mean()
        loss.backward()
        opt.step()
        losses.append(float(loss.detach()))
    return losses


@torch.no_grad()
def serve(B=3, prompt=200, tokens=20, width=256, dtype=torch.bfloat16, seed=1):
    """A prompt of ragged lengths, then tokens one at a time from its states in a pool, against the whole sequences at once:
    the largest relative difference of a row."""
    torch.manual_seed(seed)
    block = AttentionBlock(width, 4, 2, width // 8, dtype)
    lengths = torch.tensor([prompt - 17 * b for b in range(B)], dtype=torch.int32, device="cuda")
    x = torch.randn(B, prompt + tokens, width, device="cuda").to(dtype)
    positions = torch.arange(prompt + tokens, dtype=torch.int32, device="cuda")
    whole, _ = block(x, positions)
    _, state = block(x[:, :prompt].contiguous(), positions[:prompt].contiguous(), lengths)
    slots = torch.arange(B, dtype=torch.int32, device="cuda") * 2 + 1          # the pool's states 1, 3, 5, ..
    pool = torch.zeros((2 * B + 1,) + state.shape[1:], device="cuda")
    pool[slots.long()] = state
    rows, worst = torch.arange(B, device="cuda"), 0.0
    for t in range(tokens):
        at = lengths + t
        y = block.step(x[rows, at.long()], at, pool, slots)
        want = whole[rows, at.long()].float()
        worst = max(worst, float(((y.float() - want).norm(dim=-1) / want.norm(dim=-1)).max()))
    return worst


if __name__ == "__main__":
    print("losses " + " ".join(f"{v:.4f}" for v in train()))
    print(f"single tokens against the whole sequences: {serve():.2e}")
