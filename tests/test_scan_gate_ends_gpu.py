"""Gates of the recurrence at the ends of what fp32 holds, each result to its own size."""
import numpy as np
import pytest

from oracle import block
from tests.mixer_util import ULP, host, say, tdtype, wide
from tests.test_gated_scan_gpu import SLACK, cuda

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lc():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from fft_long_convolution_amd import lconv
    lconv.load()
    return lconv


def beyond(got, ref, dtype, size, extra):
    """The largest error beyond the rounding of the result, in units of SLACK size + extra."""
    got = wide(got)
    assert got.shape == ref.shape and np.all(np.isfinite(got))
    least = {"f32": -126, "f16": -14, "bf16": -126}[dtype]
    binade = np.maximum(np.floor(np.log2(np.maximum(np.abs(ref), 1e-300))), least)
    over = np.abs(got - ref) - ULP[dtype] * 2.0 ** binade
    return float(np.max(over / np.maximum(SLACK * size + extra, 1e-60), initial=0.0))


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_inputs_behind_closed_gates(lc, dtype):
    """sigmoid(input gate) and its slope to their own size, down to 2^-126.  The exponent log2(e) gate is off by 1.22 2^-24 of itself
    (log2(e) as a float, the product), which makes the exponential off by |gate| times that."""
    import torch
    say(f"[gate ends] input gates {dtype}")
    rng = np.random.default_rng(1303)
    B, N, C = 1, 9, 12
    ends = [-87.0, -85.0, -80.0, -75.0, -72.0, -70.0, -68.0, -40.0, 0.0, 12.0, 60.0, 90.0]
    i = torch.from_numpy(np.broadcast_to(np.array(ends, np.float32), (B, N, C)).copy()).to(tdtype(dtype))
    x, z, dy = (host(rng, (B, N, C), dtype) for _ in range(3))
    gx, gz, gdy, gi = cuda(x, z, dy, i)
    f = lc.gated_scan(gx, gz, "sigmoid", "convex", gi, need_marks=True)
    g = lc.gated_scan_bwd(gdy, gx, gz, f.marks, "sigmoid", "convex", gi)
    args = dict(gate="sigmoid", mix="convex")
    want = block.gated_scan_bwd(wide(dy), wide(x), wide(z), input_gate=wide(i), **args)
    a = lambda t: np.abs(wide(t))  # noqa: E731
    size = block.gated_scan_bwd(a(dy), a(x), wide(z), input_gate=wide(i), size=True, **args)
    di = want[0] * wide(x) / (1.0 + np.exp(wide(i)))                   # 1 - s to its own size, unlike 1.0 - s
    sdi = size[0] * a(x) / (1.0 + np.exp(wide(i)))
    # 1 + exp(-gate) has lost a gate of more than 87, and 1 - s with it; s is 1 there
    open_ = wide(i) > 87.0
    for name, got, r, m in (("dx", g.dx, want[0], size[0]), ("di", g.dinput_gate, di, sdi)):
        off = beyond(got, r, dtype, m, m * np.where(open_, 1.0, 1.25 * 2.0 ** -24 * np.abs(wide(i))))
        say(f"   {name} {off:.2f}")
        assert off <= 1, name
