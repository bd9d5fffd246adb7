"""The hybrid example's autograd functions: gradients that come as repeated elements, gradients through the state between two
pieces of a sequence, and second derivatives, which there are not."""
import pytest

from tests.mixer_util import TOL, rel, say, wide
from tests.test_hybrid_example_gpu import ex  # noqa: F401

pytestmark = pytest.mark.gpu


def test_gradient_of_a_plain_sum(ex):  # noqa: F811
    """y.sum().backward() hands every function a gradient of stride 0."""
    import torch
    say("[hybrid sum]")
    torch.manual_seed(5)
    block = ex.AttentionBlock(128, 4, 2, 16, torch.float32)
    q, k, v = (torch.randn(2, h, 40, 32, device="cuda", requires_grad=True) for h in (4, 2, 2))
    y, state = ex.LinearAttention.apply(q, k, v, block.log_decay(), None, None)
    y.sum().backward()
    want = ex.lconv.linear_attention_bwd(torch.ones_like(y), q.detach(), k.detach(), v.detach(), block.log_decay().detach())
    assert all(bool((a.grad == b).all()) for a, b in zip((q, k, v), want[:3]))
    f = block.inv_freq
    a, b = (torch.randn(2, h, 40, 32, device="cuda", requires_grad=True) for h in (4, 2))
    yq, yk = ex.Rotary.apply(a, b, torch.arange(40, dtype=torch.int32, device="cuda"), f)
    (yq.sum() + yk.sum()).backward()
    assert bool(torch.isfinite(a.grad).all()) and bool(torch.isfinite(b.grad).all())
    x = torch.randn(3, 5, 128, device="cuda", requires_grad=True)
    ex.LayerNorm.apply(x, block.norm_w, block.norm_b).sum().backward()
    assert float(x.grad.abs().max()) < 1e-4                     # the sum of a normalised row does not depend on it


def test_gradients_through_the_state_of_two_pieces(ex):  # noqa: F811
    """A sequence in one call, and in two whose state passes on: the same gradients.  fp32 sums of some hundred products, ten
    operators deep, as in the example's own test."""
    import torch
    say("[hybrid pieces]")
    torch.manual_seed(6)
    block = ex.AttentionBlock(128, 4, 2, 16, torch.float32)
    x = torch.randn(2, 90, 128, device="cuda")
    start = torch.randn(2, 4, 32, 32, device="cuda")
    dy, ds = torch.randn(2, 90, 128, device="cuda"), torch.randn(2, 4, 32, 32, device="cuda")
    pos = torch.arange(90, dtype=torch.int32, device="cuda")
    grads = []
    for cuts in ([0, 90], [0, 37, 90]):
        block.zero_grad()
        xi, si = x.clone().requires_grad_(), start.clone().requires_grad_()
        s, ys = si, []
        for a, b in zip(cuts, cuts[1:]):
            y, s = block(xi[:, a:b].contiguous(), pos[a:b].contiguous(), None, s)
            ys.append(y)
        torch.autograd.backward([torch.cat(ys, 1), s], [dy, ds])
        grads.append([xi.grad, si.grad] + [p.grad.clone() for p in block.parameters()])
    errs = [rel(a, wide(b)) for a, b in zip(*grads)]
    say("   " + " ".join(f"{e:.1e}" for e in errs))
    assert max(errs) <= 10 * TOL["f32"]
    # only the state used: its gradient alone
    q, k, v = (torch.randn(2, h, 40, 32, device="cuda", requires_grad=True) for h in (4, 2, 2))
    _, s = ex.LinearAttention.apply(q, k, v, block.log_decay().detach(), None, start)
    s.backward(ds)
    assert float(q.grad.abs().max()) == 0 and float(k.grad.abs().max()) > 0 and float(v.grad.abs().max()) > 0


def test_second_derivatives_are_refused(ex):  # noqa: F811
    import torch
    say("[hybrid second]")
    q, k, v = (torch.randn(1, 2, 20, 16, device="cuda", requires_grad=True) for _ in range(3))
    y, _ = ex.LinearAttention.apply(q, k, v, torch.full((2,), -0.1, device="cuda"), None, None)
    g, = torch.autograd.grad(y.square().sum(), q, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        g.sum().backward()
