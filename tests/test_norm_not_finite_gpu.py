"""Layer norm's statistics and gradients of rows that hold a NaN or an infinity, for every width's kernel."""
import numpy as np
import pytest

from tests.mixer_util import host, say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("C", [7, 100, 500, 1000, 1500, 4000, 8000, 9001])
def test_rows_that_are_not_finite_say_so(C, dtype):
    """mean as the values add up (an infinity, or NaN), rstd NaN, y and dx NaN; the other rows' bits are unchanged."""
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from fft_long_convolution_amd import lconv
    say(f"[norm not finite] {dtype} C={C}")
    rng = np.random.default_rng(560)
    x, dy = host(rng, (9, C), dtype).cuda(), host(rng, (9, C), dtype).cuda()
    w, b = host(rng, (C,), dtype).cuda(), host(rng, (C,), dtype).cuda()
    y0, m0, r0 = lconv.layer_norm(x, w, b)
    dx0, _, db0 = lconv.layer_norm_bwd(dy, x, w, m0, r0)
    bad = {1: float("nan"), 4: float("inf"), 6: float("-inf"), 7: "both"}
    for row, value in bad.items():
        if value == "both":
            x[row, 0], x[row, C - 1] = float("inf"), float("-inf")
        else:
            x[row, C // 2] = value
    y, m, r = lconv.layer_norm(x, w, b)
    dx, _, db = lconv.layer_norm_bwd(dy, x, w, m, r)
    want = {1: "nan", 4: "inf", 6: "-inf", 7: "nan"}
    for row in range(9):
        if row in bad:
            assert str(float(m[row])) == want[row] and bool(torch.isnan(r[row]))
            assert bool(torch.isnan(y[row]).all()) and bool(torch.isnan(dx[row]).all())
        else:
            for a, c in ((y, y0), (m, m0), (r, r0), (dx, dx0)):
                assert bool((a[row] == c[row]).all())
    assert bool((db == db0).all())              # dbias does not depend on x
