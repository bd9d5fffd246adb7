"""The size of the gated recurrence's marks: whatever the forward call takes, its query gives the room for, in every type (CPU;
the host code under the sanitizers, the built library, and the gradients of such a call on the GPU)."""
import os

import numpy as np
import pytest

from oracle import block
from tests.mixer_util import host, off_by, say, wide
from tests.test_gated_scan_gpu import SLACK
from tests.test_sanitizers import CSRC, HERE, ROOT, SAN, _run, _tool, outdir  # noqa: F401

# 16-bit calls take these with two channels to a lane; with one, as fp32 has them, they pass a grid's reach
LARGE = [(131072, 1, 2560), (131072, 8, 2560), (65536, 16, 5120)]


def test_marks_of_every_call_that_launches(outdir):  # noqa: F811
    cxx, rocm = _tool("clang++"), "/opt/rocm"
    exe = os.path.join(outdir, "block_sizes")
    _run([cxx, *SAN, "-std=c++17", "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(rocm, "include"),
          "-I", os.path.join(ROOT, "include"), "-I", CSRC, "-Wno-unused-result", "-Wno-unused-value",
          os.path.join(CSRC, "block_api.cpp"), os.path.join(HERE, "block_sizes_main.cpp"), "-o", exe])
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:abort_on_error=1", UBSAN_OPTIONS="print_stacktrace=1")
    assert "BLOCK_SIZES_OK" in _run([exe], env=env).stdout


def test_the_query_of_the_built_library():
    from fft_long_convolution_amd import lconv
    q = lconv.lconv_gated_scan_marks_bytes
    for B, N, C in LARGE + [(2, 65, 12), (1, 1, 1), (1, 64, 7)]:
        assert q(B, N, C) == B * ((N + 63) // 64) * C * 4
    # nothing for what no type takes
    for bad in ((0, 8, 8), (8, 0, 8), (8, 8, 0), (-1, 8, 8), (1, 2 ** 31, 8), (1, 8, 2 ** 24 + 1), (2 ** 24 + 1, 8, 8)):
        assert q(*bad) == 0, bad


@pytest.mark.gpu
def test_gradients_of_many_wide_rows():
    """The first of these calls in bf16, trained; some rows and channels against float64."""
    import torch
    from fft_long_convolution_amd import lconv
    B, N, C = LARGE[0]
    say(f"[sizes] {(B, N, C)}")
    rng = np.random.default_rng(1200)
    rows = np.unique(np.r_[0, B - 1, rng.integers(0, B, 30)])
    # the same few rows over and over
    x, z, dy = (host(rng, (16, N, C), "bf16") for _ in range(3))
    gx, gz, gdy = (t.cuda().repeat(B // 16, 1, 1) for t in (x, z, dy))
    f = lconv.gated_scan(gx, gz, "sigmoid", "convex", need_marks=True)
    assert f.marks.numel() == B * C
    g = lconv.gated_scan_bwd(gdy, gx, gz, f.marks, "sigmoid", "convex")
    X, Z, D = (wide(t)[rows % 16] for t in (x, z, dy))
    want, last = block.gated_scan(X, Z, "sigmoid", "convex")
    size, _ = block.gated_scan(np.abs(X), Z, "sigmoid", "convex")
    at = torch.from_numpy(rows).cuda()
    e = off_by(f.y[at], want, "bf16", np.maximum(size, 1e-6))
    want = block.gated_scan_bwd(D, X, Z, gate="sigmoid", mix="convex")
    size = block.gated_scan_bwd(np.abs(D), np.abs(X), Z, gate="sigmoid", mix="convex", size=True)
    for got, r, s in zip(g[:2], want, size):
        e = max(e, off_by(got[at], r, "bf16", np.maximum(s, 1e-6)))
    say(f"   beyond the rounding: {e:.1e} (at most {SLACK:.1e})")
    assert e <= SLACK
    for t in (f.y, g.dx, g.dz):
        assert bool((t.view(-1, 16, N, C) == t[:16]).all())
