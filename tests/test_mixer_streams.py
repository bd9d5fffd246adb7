"""A stream of another GPU than the operands' is refused before anything is launched on it (CPU: a stand-in for the stream)."""
from types import SimpleNamespace

import pytest

torch = pytest.importorskip("torch")

from fft_long_convolution_amd import lconv  # noqa: E402


def test_a_stream_of_another_device(monkeypatch):
    monkeypatch.setattr(torch.cuda, "stream", lambda s: s)
    other, own = (SimpleNamespace(device=torch.device("cuda", i), cuda_stream=64) for i in (1, 0))
    with pytest.raises(ValueError, match="cuda:1, the operands on cuda:0"):
        lconv._at(0, other)
    assert lconv._at(0, own)[1] == 64
