"""Frequencies by parts: which pairs keep theirs, which are divided, and the ramp between, also where the original context is
so short or so long that a bound lies outside the pairs (CPU)."""
import numpy as np
import pytest

pytest.importorskip("torch")

from fft_long_convolution_amd import lconv  # noqa: E402


@pytest.mark.parametrize("rot", [2, 8, 24, 64, 128])
@pytest.mark.parametrize("base", [10.0, 500.0, 10000.0, 1e6])
@pytest.mark.parametrize("original", [5, 40, 100, 2048, 131072, 10 ** 9])
@pytest.mark.parametrize("fast,slow", [(32.0, 1.0), (1.5, 1.4), (4.0, 0.25)])
def test_parts(rot, base, original, fast, slow):
    plain = lconv.rotary_frequencies(rot, base=base, device="cpu")[0].double().numpy()
    f, m = lconv.rotary_frequencies(rot, base=base, scaling="by_parts", factor=8.0, original=original, fast=fast, slow=slow, device="cpu")
    part = (1.0 - f.double().numpy() / plain) * 8.0 / 7.0         # 0: kept, 1: divided by the factor
    turns = original * plain / (2.0 * np.pi)
    assert np.all(np.abs(part[turns > fast * 1.0001]) < 1e-5) and np.all(np.abs(part[turns < slow * 0.9999] - 1.0) < 1e-5)
    assert np.all(np.diff(part) > -1e-5) and abs(m - (1.0 + 0.1 * np.log(8.0))) < 1e-12
    between = np.nonzero((part > 1e-4) & (part < 1 - 1e-4))[0]
    if len(between) > 2:                                        # a straight line in the index
        np.testing.assert_allclose(np.diff(part[between], 2), 0.0, atol=2e-5)


def test_refusals():
    for bad in (dict(fast=1.0), dict(slow=0.0), dict(base=1.0), dict(original=0)):
        with pytest.raises(ValueError, match="by_parts"):
            lconv.rotary_frequencies(8, scaling="by_parts", factor=2.0, device="cpu", **bad)
