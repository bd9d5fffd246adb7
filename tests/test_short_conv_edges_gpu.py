"""Gradients of the short convolution at the ends: SiLU's slope far out, values that are not finite."""
import numpy as np
import pytest

from oracle import block
from tests.mixer_util import ULP, host, say, tdtype, wide
from tests.test_short_conv_gpu import SLACK, cuda

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lc():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from fft_long_convolution_amd import lconv
    lconv.load()
    return lconv


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_slopes_far_out(lc, dtype):
    """dx behind one tap of weight one, to its own size down to sigmoid(p) = 2^-126: the exponent log2(e) p is off by 1.22 2^-24 of
    itself (log2(e) as a float, the product), which makes the exponential off by |p| times that."""
    import torch
    say(f"[conv edges] slopes {dtype}")
    rng = np.random.default_rng(1400)
    B, N, K = 2, 19, 4
    p = np.array([-87.0, -84.0, -80.0, -75.0, -71.0, -68.0, -40.0, -9.0, -1.25, 0.0, 3.0, 40.0, 87.0], np.float32)
    x = torch.from_numpy(np.broadcast_to(p, (B, N, len(p))).copy()).to(tdtype(dtype))
    w = torch.zeros((len(p), K), dtype=tdtype(dtype))
    w[:, K - 1] = 1
    dy = host(rng, x.shape, dtype)
    gx, gw, gdy = cuda(x, w, dy)
    got = wide(lc.short_conv_bwd(gdy, gx, gw, activation="silu").dx)
    want = block.short_conv_bwd(wide(dy), wide(x), wide(w), None, True)[0]
    P = wide(x)
    size = np.abs(wide(dy)) * (1.0 + np.abs(P)) / (1.0 + np.exp(-P))
    least = -14 if dtype == "f16" else -126
    over = np.abs(got - want) - ULP[dtype] * 2.0 ** np.maximum(np.floor(np.log2(np.maximum(np.abs(want), 1e-300))), least)
    off = float(np.max(over / (size * (SLACK + 1.25 * 2.0 ** -24 * np.abs(P)))))
    say(f"   {off:.2f}")
    assert np.all(np.isfinite(got)) and off <= 1


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("C", [3, 24])
@pytest.mark.parametrize("silu", [False, True])
def test_values_that_are_not_finite(lc, dtype, C, silu):
    """A weight that is not finite reaches its channel's tokens and none behind a row's length; an input reaches the gradients of the
    taps that met it: the last one's alone, for a row's last token."""
    import torch
    rng = np.random.default_rng(1401)
    act = "silu" if silu else None
    for K in (2, 4, 8):
        for B, N, ends in ((5, 45, [45, 0, 1, 17, 33]), (2, 300, [300, 299])):
            say(f"[conv edges] not finite {dtype} K={K} silu={silu} {(B, N, C)}")
            n = torch.tensor(ends, dtype=torch.int32)
            x, dy, w = host(rng, (B, N, C), dtype), host(rng, (B, N, C), dtype), host(rng, (C, K), dtype)
            s, ds = host(rng, (B, K - 1, C), dtype), host(rng, (B, K - 1, C), dtype)
            gx, gdy, gw, gn, gs, gds = cuda(x, dy, w, n, s, ds)
            clean = lc.short_conv_bwd(gdy, gx, gw, activation=act, state=gs, dstate=gds, lengths=gn)
            for bad in (float("nan"), float("inf")):
                for j in (0, K - 1):
                    v = gw.clone()
                    v[1, j] = bad
                    g = lc.short_conv_bwd(gdy, gx, v, activation=act, state=gs, dstate=gds, lengths=gn)
                    for b, end in enumerate(ends):
                        assert not bool(g.dx[b, end:].any()), (K, end)
                        if end == 0:
                            assert bool((g.dstate[b] == gds[b]).all())
                        if end > 1:
                            # token t's own tap K - 1 - j meets dp of token s + K - 1 - j
                            hit = g.dx[b, :max(end - (K - 1 - j), 0), 1]
                            past = g.dx[b, max(end - (K - 1 - j), 0):end, 1]
                            assert silu or (not bool(hit.isfinite().any()) and bool(past.isfinite().all()))
                    rest = [c for c in range(C) if c != 1]
                    assert bool((g.dx[..., rest] == clean.dx[..., rest]).all())
                    assert bool((g.dweight[rest] == clean.dweight[rest]).all())
            if silu:
                continue
            # a row's last input: tap K - 1 alone meets it
            for b, end in enumerate(ends):
                if end == 0:
                    continue
                y = gx.clone()
                y[b, end - 1, 2] = float("inf")
                g = lc.short_conv_bwd(gdy, y, gw, activation=act, state=gs, dstate=gds, lengths=gn)
                assert not bool(g.dweight[2, K - 1].isfinite())
                assert bool((g.dweight[2, :K - 1] == clean.dweight[2, :K - 1]).all()), (K, end)
                assert bool((g.dx == clean.dx).all())
