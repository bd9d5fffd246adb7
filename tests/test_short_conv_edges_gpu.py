"""Gradients of the short convolution at the ends: SiLU's slope far out."""
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
