"""The hybrid example (long convolution, layer norm, rotary positions and linear attention together): training falls, its
gradients are those of a plain float64 model, and single tokens continue a prompt."""
import importlib.util
import os

import numpy as np
import pytest

from tests.mixer_util import TOL, rel, say, wide

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ex():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    spec = importlib.util.spec_from_file_location("hybrid_block", os.path.join(ROOT, "examples", "hybrid_block.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    m.lconv.load()
    return m


def test_training_falls(ex):
    losses = ex.train(steps=8, N=256)
    say("[hybrid train] " + " ".join(f"{v:.4f}" for v in losses))
    assert all(np.isfinite(losses)) and losses[-1] < 0.8 * losses[0]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_tokens_continue_the_prompt(ex, dtype):
    """Differences are roundings of y, of the projected sum and, in the prompt, of scores and states as operands: at
    most four of them in a row of the block's output, which also holds the input itself."""
    import torch
    worst = ex.serve(dtype={"f32": torch.float32, "bf16": torch.bfloat16}[dtype])
    say(f"[hybrid serve] {dtype} {worst:.2e}")
    assert worst <= 4 * TOL[dtype]


def plain_block(block, x, positions):
    """The attention block in float64 torch on the CPU, token by token; parameters as leaves."""
    import torch
    P = {n: p.detach().cpu().double().requires_grad_() for n, p in block.named_parameters()}
    x = x.detach().cpu().double().requires_grad_()
    B, N, W = x.shape
    H, G, D = block.heads, block.shared, block.D
    h = (x - x.mean(-1, keepdim=True)) / (x.var(-1, unbiased=False, keepdim=True) + 1e-5).sqrt() * P["norm_w"] + P["norm_b"]
    h = (h @ P["inp"].t()).view(B, N, H + 2 * G, D)
    f = block.inv_freq.cpu().double()
    a = positions.cpu().double()[:, None] * f
    c, s, half = a.cos()[None, :, None], a.sin()[None, :, None], f.numel()

    def turn(t):
        x1, x2 = t[..., :half], t[..., half:2 * half]
        return torch.cat((x1 * c - x2 * s, x2 * c + x1 * s, t[..., 2 * half:]), -1)

    q, k, v = turn(h[:, :, :H]), turn(h[:, :, H:H + G]), h[:, :, H + G:]
    k, v = (t.repeat_interleave(H // G, dim=2) for t in (k, v))
    gamma = (-P["decay"].exp()).exp()[None, :, None, None]
    S, ys = torch.zeros(B, H, D, D, dtype=torch.float64), []
    for t in range(N):
        S = gamma * S + k[:, t, :, :, None] * v[:, t, :, None, :]
        ys.append((S * q[:, t, :, :, None]).sum(2) / D ** 0.5)
    y = torch.stack(ys, 1).reshape(B, N, W)
    return x + y @ P["out"].t(), x, P


def test_gradients_of_the_block(ex):
    """fp32 against float64.  About ten operators stand between loss and input, each with sums of at most 256 products
    (16 half-units where roundings add like a random walk; 64 allowed as for one operator): ten times that."""
    import torch
    torch.manual_seed(3)
    block = ex.AttentionBlock(128, 4, 2, 16, torch.float32)
    x = torch.randn(2, 75, 128, device="cuda", requires_grad=True)
    positions = torch.arange(5, 80, dtype=torch.int32, device="cuda")
    dy = torch.randn(2, 75, 128, device="cuda")
    y, _ = block(x, positions)
    y.backward(dy)
    ry, rx, P = plain_block(block, x, positions)
    ry.backward(dy.cpu().double())
    errs = {"y": rel(y, wide(ry)), "x": rel(x.grad, wide(rx.grad))}
    for n, p in block.named_parameters():
        errs[n] = rel(p.grad, wide(P[n].grad))
    say("[hybrid grads] " + " ".join(f"{n} {e:.1e}" for n, e in errs.items()))
    assert all(e <= 10 * TOL["f32"] for e in errs.values()), errs
