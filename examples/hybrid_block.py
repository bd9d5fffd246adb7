"""A small hybrid language-model stack on this library's operators: blocks of gated long convolution, blocks of linear
attention with rotary positions (with norms of q and k where asked for) and recurrent blocks (a short convolution, then a gated
recurrence), each behind a layer norm, with plain torch products for the projections.

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


class QkNormRotary(torch.autograd.Function):
    """q and k of [B, heads, N, D], every head's row over its root mean square, times a weight, turned."""

    @staticmethod
    def forward(ctx, q, k, q_weight, k_weight, positions, inv_freq):
        ctx.save_for_backward(q, k, q_weight, k_weight, positions, inv_freq)
        return lconv.qk_norm_rotary(q, k, q_weight, k_weight, positions, inv_freq)

    @staticmethod
    @once
    def backward(ctx, dq, dk):
        q, k, wq, wk, positions, inv_freq = ctx.saved_tensors
        g = lconv.qk_norm_rotary_bwd(rows(dq), rows(dk), q, k, wq, wk, positions, inv_freq)
        return g.dq, g.dk, g.dq_weight.to(wq.dtype), g.dk_weight.to(wk.dtype), None, None


class ShortConv(torch.autograd.Function):
    """y and the last inputs, from the inputs before or none; either result may be used."""

    @staticmethod
    def forward(ctx, x, weight, bias, lengths, state):
        y, last = lconv.short_conv(x, weight, bias, "silu", state=state, lengths=lengths)
        ctx.save_for_backward(x, weight, bias, lengths, state)
        ctx.set_materialize_grads(False)
        return y, last

    @staticmethod
    @once
    def backward(ctx, dy, dlast):
        x, weight, bias, lengths, state = ctx.saved_tensors
        dy = torch.zeros(x.shape, dtype=x.dtype, device=x.device) if dy is None else rows(dy)
        g = lconv.short_conv_bwd(dy, x, weight, bias, "silu", state=state, dstate=None if dlast is None else dlast.contiguous(),
                                 lengths=lengths)
        return g.dx, g.dweight.to(weight.dtype), g.dbias.to(bias.dtype), None, g.dstate


class GatedScan(torch.autograd.Function):
    """y and the state after the last token, from a state or none; either result may be used."""

    @staticmethod
    def forward(ctx, x, z, input_gate, rate, lengths, state):
        y, last, marks = lconv.gated_scan(x, z, "rate", "norm", input_gate, rate, state=state, lengths=lengths, need_marks=True)
        ctx.save_for_backward(x, z, input_gate, rate, lengths, marks)
        ctx.has_state = state is not None
        ctx.set_materialize_grads(False)
        return y, last

    @staticmethod
    @once
    def backward(ctx, dy, dlast):
        x, z, input_gate, rate, lengths, marks = ctx.saved_tensors
        dy = torch.zeros(x.shape, dtype=x.dtype, device=x.device) if dy is None else rows(dy)
        g = lconv.gated_scan_bwd(dy, x, z, marks, "rate", "norm", input_gate, rate,
                                 dstate=None if dlast is None else dlast.contiguous(), lengths=lengths, need_dstate=ctx.has_state)
        return g.dx, g.dz, g.dinput_gate, g.drate, None, g.dstate


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
    def __init__(self, width, heads, shared, rot, dtype, qk_norm=False):
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
        weights = (torch.nn.Parameter(torch.ones(self.D, device="cuda", dtype=dtype)) for _ in range(2))
        self.q_norm, self.k_norm = weights if qk_norm else (None, None)

    def turn(self, q, k, positions):
        if self.q_norm is None:
            return Rotary.apply(q, k, positions, self.inv_freq)
        return QkNormRotary.apply(q, k, self.q_norm, self.k_norm, positions, self.inv_freq)

    def log_decay(self):
        return -self.decay.exp()

    def project(self, x):
        """q, k, v of x [B, N, width] as slices of one product: [B, heads, N, D] views, read where they are."""
        B, N, _ = x.shape
        h = (LayerNorm.apply(x, self.norm_w, self.norm_b) @ self.inp.t()).view(B, N, self.heads + 2 * self.shared, self.D)
        return (t.transpose(1, 2) for t in h.split((self.heads, self.shared, self.shared), dim=2))

    def forward(self, x, positions, lengths=None, state=None):
        q, k, v = self.project(x)
        q, k = self.turn(q, k, positions)
        y, state = LinearAttention.apply(q, k, v, self.log_decay(), lengths, state)
        return x + y.transpose(1, 2).reshape(x.shape) @ self.out.t(), state

    def step(self, x, positions, state, slots=None):
        """One token of every sequence: x [B, width], positions [B]; the states move on in place."""
        q, k, v = self.project(x[:, None])
        q, k = self.turn(q, k, positions[:, None])
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


class RecurrentBlock(torch.nn.Module):
    """A short convolution, then a recurrence whose decays and inputs are gated by the token, then an output gate."""

    def __init__(self, width, dtype, taps=4):
        super().__init__()
        p = lambda *shape: torch.nn.Parameter((torch.randn(shape) / math.sqrt(shape[-1])).to("cuda", dtype))  # noqa: E731
        self.norm_w = torch.nn.Parameter(torch.ones(width, device="cuda", dtype=dtype))
        self.norm_b = torch.nn.Parameter(torch.zeros(width, device="cuda", dtype=dtype))
        self.inp, self.out = p(4 * width, width), p(width, width)
        self.conv_w, self.conv_b = p(width, taps), torch.nn.Parameter(torch.zeros(width, device="cuda", dtype=dtype))
        # decays of 0.9 to 0.999 at a half-open gate
        self.log_rate = torch.nn.Parameter(torch.log(-2.0 * torch.log(torch.linspace(0.9, 0.999, width, device="cuda"))))

    def project(self, x):
        """The convolution's input, the two gates of the recurrence and the output's, as slices of one product."""
        return (LayerNorm.apply(x, self.norm_w, self.norm_b) @ self.inp.t()).chunk(4, dim=-1)

    def forward(self, x, lengths=None, state=None):
        """x [B, N, width]; state: the convolution's last inputs and the recurrence's state, of an earlier piece."""
        u, z, i, o = self.project(x)
        inputs, h = (None, None) if state is None else state
        u, inputs = ShortConv.apply(u, self.conv_w, self.conv_b, lengths, inputs)
        y, h = GatedScan.apply(u, z, i, self.log_rate.exp(), lengths, h)
        return x + (y * torch.nn.functional.silu(o)) @ self.out.t(), (inputs, h)

    def step(self, x, inputs, h, slots=None):
        """One token of every sequence: x [B, width]; both pools move on in place."""
        u, z, i, o = self.project(x)
        u = lconv.short_conv_step(u, self.conv_w, inputs, self.conv_b, "silu", slots=slots)
        y = lconv.gated_scan_step(u, z, h, "rate", "norm", i, self.log_rate.exp(), slots=slots)
        return x + (y * torch.nn.functional.silu(o)) @ self.out.t()


class Hybrid(torch.nn.Module):
    def __init__(self, width=256, heads=4, shared=2, N=512, dtype=torch.bfloat16, recurrent=False):
        """recurrent: a recurrent block in front of the attention, whose q and k are then normed."""
        super().__init__()
        self.conv = ConvBlock(width, N, dtype)
        self.recurrent = RecurrentBlock(width, dtype) if recurrent else None
        self.attention = AttentionBlock(width, heads, shared, (width // heads) // 2, dtype, qk_norm=recurrent)

    def forward(self, x, positions):
        x = self.conv(x)
        if self.recurrent is not None:
            x = self.recurrent(x)[0]
        return self.attention(x, positions)[0]


def train(steps=8, B=2, N=512, width=256, dtype=torch.bfloat16, seed=0, recurrent=False):
    """Fits a running mean of the input's past; returns the losses."""
    torch.manual_seed(seed)
    model = Hybrid(width=width, N=N, dtype=dtype, recurrent=recurrent)
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


@torch.no_grad()
def serve_recurrent(B=3, prompt=200, tokens=20, width=256, dtype=torch.bfloat16, seed=2):
    """serve for a recurrent block and an attention block with norms of q and k behind it."""
    torch.manual_seed(seed)
    first, second = RecurrentBlock(width, dtype), AttentionBlock(width, 4, 2, width // 8, dtype, qk_norm=True)
    lengths = torch.tensor([prompt - 17 * b for b in range(B)], dtype=torch.int32, device="cuda")
    x = torch.randn(B, prompt + tokens, width, device="cuda").to(dtype)
    positions = torch.arange(prompt + tokens, dtype=torch.int32, device="cuda")
    whole = second(first(x)[0], positions)[0]
    y, (inputs, h) = first(x[:, :prompt].contiguous(), lengths)
    _, state = second(y, positions[:prompt].contiguous(), lengths)
    slots = torch.arange(B, dtype=torch.int32, device="cuda") * 2 + 1          # the pools' states 1, 3, 5, ..
    pools = [torch.zeros((2 * B + 1,) + t.shape[1:], dtype=t.dtype, device="cuda") for t in (inputs, h, state)]
    for pool, t in zip(pools, (inputs, h, state)):
        pool[slots.long()] = t
    rows, worst = torch.arange(B, device="cuda"), 0.0
    for t in range(tokens):
        at = lengths + t
        y = second.step(first.step(x[rows, at.long()], *pools[:2], slots), at, pools[2], slots)
        want = whole[rows, at.long()].float()
        worst = max(worst, float(((y.float() - want).norm(dim=-1) / want.norm(dim=-1)).max()))
    return worst


if __name__ == "__main__":
    print("losses " + " ".join(f"{v:.4f}" for v in train()))
    print("with a recurrent block " + " ".join(f"{v:.4f}" for v in train(recurrent=True)))
    print(f"single tokens against the whole sequences: {serve():.2e}, with a recurrent block {serve_recurrent():.2e}")
