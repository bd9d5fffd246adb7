"""The hybrid example with a recurrent block (short convolution and gated recurrence) and norms of q and k: it trains, its gradients
are those of a plain float64 model, single tokens continue a prompt, and pieces of a sequence give what the whole does."""
import numpy as np
import pytest

from tests.mixer_util import TOL, rel, say, wide
from tests.test_hybrid_example_gpu import ex  # noqa: F401

pytestmark = pytest.mark.gpu


def test_it_trains(ex):  # noqa: F811
    losses = ex.train(steps=4, N=256, recurrent=True)
    say("[recurrent train] " + " ".join(f"{v:.4f}" for v in losses))
    assert all(np.isfinite(losses))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_tokens_continue_the_prompt(ex, dtype):  # noqa: F811
    """Two blocks of some four roundings each in a row of the output, which also holds the input itself."""
    import torch
    worst = ex.serve_recurrent(dtype={"f32": torch.float32, "bf16": torch.bfloat16}[dtype])
    say(f"[recurrent serve] {dtype} {worst:.2e}")
    assert worst <= 8 * TOL[dtype]


def norm(x, w, b):
    return (x - x.mean(-1, keepdim=True)) / (x.var(-1, unbiased=False, keepdim=True) + 1e-5).sqrt() * w + b


def plain_recurrent(x, P, inputs, h):
    """The recurrent block in float64 torch, token by token, from the convolution's inputs and a state."""
    import torch
    K, N = P["conv_w"].shape[1], x.shape[1]
    u, z, i, o = (norm(x, P["norm_w"], P["norm_b"]) @ P["inp"].t()).chunk(4, dim=-1)
    seen = torch.cat((inputs, u), 1)
    p = P["conv_b"] + sum(P["conv_w"][:, j] * seen[:, j:j + N] for j in range(K))
    u = p * torch.sigmoid(p)
    rate, ys = P["log_rate"].exp(), []
    for t in range(N):
        a = torch.exp(-rate * torch.sigmoid(z[:, t]))
        h = a * h + (1 - a * a).sqrt() * torch.sigmoid(i[:, t]) * u[:, t]
        ys.append(h)
    return x + (torch.stack(ys, 1) * o * torch.sigmoid(o)) @ P["out"].t(), seen[:, N:], h


def leaves(module):
    return {n: p.detach().cpu().double().requires_grad_() for n, p in module.named_parameters()}


def test_gradients_of_the_recurrent_block(ex):  # noqa: F811
    """fp32 against float64, through the states on both ends, in one call and in two pieces.  About ten operators stand between
    loss and input, each with sums of at most 512 products (64 half-units allowed as for one operator): ten times that."""
    import torch
    torch.manual_seed(13)
    block = ex.RecurrentBlock(128, torch.float32)
    x, dy = torch.randn(2, 75, 128, device="cuda"), torch.randn(2, 75, 128, device="cuda")
    inputs, h = torch.randn(2, 3, 128, device="cuda"), torch.randn(2, 128, device="cuda")
    dinputs, dh = torch.randn(2, 3, 128, device="cuda"), torch.randn(2, 128, device="cuda")
    P = leaves(block)
    rx, ri, rh = (t.cpu().double().requires_grad_() for t in (x, inputs, h))
    ry, rl, rlast = plain_recurrent(rx, P, ri, rh)
    torch.autograd.backward([ry, rl, rlast], [t.cpu().double() for t in (dy, dinputs, dh)])
    for cuts in ([0, 75], [0, 2, 33, 75]):
        block.zero_grad()
        gx, gi, gh = (t.clone().requires_grad_() for t in (x, inputs, h))
        state, ys = (gi, gh), []
        for a, b in zip(cuts, cuts[1:]):
            y, state = block(gx[:, a:b].contiguous(), None, state)
            ys.append(y)
        torch.autograd.backward([torch.cat(ys, 1), *state], [dy, dinputs, dh])
        errs = {"y": rel(torch.cat(ys, 1), wide(ry)), "x": rel(gx.grad, wide(rx.grad)), "inputs": rel(gi.grad, wide(ri.grad)),
                "h": rel(gh.grad, wide(rh.grad))}
        for n, p in block.named_parameters():
            errs[n] = rel(p.grad, wide(P[n].grad))
        say(f"[recurrent grads] {cuts} " + " ".join(f"{n} {e:.1e}" for n, e in errs.items()))
        assert all(e <= 10 * TOL["f32"] for e in errs.values()), errs


def test_gradients_of_normed_attention(ex):  # noqa: F811
    """As above, for the attention block with norms of q and k."""
    import torch
    torch.manual_seed(14)
    B, N, W, H, G, D, rot = 2, 60, 128, 4, 2, 32, 16
    block = ex.AttentionBlock(W, H, G, rot, torch.float32, qk_norm=True)
    with torch.no_grad():
        block.q_norm.add_(0.2 * torch.randn(D, device="cuda"))
        block.k_norm.add_(0.2 * torch.randn(D, device="cuda"))
    x, dy = torch.randn(B, N, W, device="cuda", requires_grad=True), torch.randn(B, N, W, device="cuda")
    positions = torch.arange(5, 5 + N, dtype=torch.int32, device="cuda")
    y, _ = block(x, positions)
    y.backward(dy)
    P, rx = leaves(block), x.detach().cpu().double().requires_grad_()
    t = (norm(rx, P["norm_w"], P["norm_b"]) @ P["inp"].t()).view(B, N, H + 2 * G, D)
    q, k, v = t.split((H, G, G), dim=2)
    a = positions.cpu().double()[:, None] * block.inv_freq.cpu().double()
    c, s = a.cos()[None, :, None], a.sin()[None, :, None]

    def turned(u, w):
        u = u / ((u * u).mean(-1, keepdim=True) + 1e-6).sqrt() * w
        lo, hi = u[..., : rot // 2], u[..., rot // 2: rot]
        return torch.cat((lo * c - hi * s, hi * c + lo * s, u[..., rot:]), -1)

    q, k = turned(q, P["q_norm"]), turned(k, P["k_norm"])
    k, v = (u.repeat_interleave(H // G, dim=2) for u in (k, v))
    gamma, S, ys = (-P["decay"].exp()).exp()[None, :, None, None], torch.zeros(B, H, D, D, dtype=torch.float64), []
    for n in range(N):
        S = gamma * S + k[:, n, :, :, None] * v[:, n, :, None, :]
        ys.append((S * q[:, n, :, :, None]).sum(2) / D ** 0.5)
    ry = rx + torch.stack(ys, 1).reshape(B, N, W) @ P["out"].t()
    ry.backward(dy.cpu().double())
    errs = {"y": rel(y, wide(ry)), "x": rel(x.grad, wide(rx.grad))}
    for n, p in block.named_parameters():
        errs[n] = rel(p.grad, wide(P[n].grad))
    say("[normed grads] " + " ".join(f"{n} {e:.1e}" for n, e in errs.items()))
    assert all(e <= 10 * TOL["f32"] for e in errs.values()), errs


def test_only_the_states_are_used(ex):  # noqa: F811
    import torch
    say("[recurrent states alone]")
    torch.manual_seed(15)
    block = ex.RecurrentBlock(64, torch.float32)
    x = torch.randn(2, 30, 64, device="cuda", requires_grad=True)
    _, (inputs, h) = block(x)
    h.sum().backward(retain_graph=True)
    assert bool(x.grad.isfinite().all()) and float(x.grad.abs().max()) > 0
    x.grad = None
    inputs.sum().backward()
    assert bool(x.grad.isfinite().all()) and float(x.grad[:, :-3].abs().max()) == 0
