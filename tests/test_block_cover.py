"""Every variant of the recurrence's, the q/k norms' and the short convolution's kernels that a plan can choose, run: the first
test holds the GPU tests' shapes, with those below, against the plans over a wide range of calls (CPU), so that a retuned plan
cannot leave a variant without a case."""
import os
import subprocess

import pytest

from tests import test_gated_scan_gpu as scan
from tests import test_qk_norm_gpu as norm
from tests import test_short_conv_gpu as conv
from tests.test_sanitizers import CSRC, HERE, ROOT, _run, _tool, outdir  # noqa: F401

# many rows of one channel to a lane; of two, short ones too and a width that ends inside a wave; two channels in segments
SCAN = [(520, 70, 3), (257, 70, 66), (256, 30, 130), (130, 70, 66), (130, 30, 128), (3, 600, 70), (1, 1537, 130)]
# more runs, and more rows, than the gradients' waves
CONV = [(2100, 40, 3), (4200, 9, 4)]
# lanes that a head's units fill or not, items of four heads
NORM = [(2, 3, 2, 50, 8, 0, "bnhd", 0), (3, 3, 2, 50, 32, 32, "bhnd", 3), (2, 4, 4, 70, 256, 256, "bhnd", 3),
        (5, 4, 1, 30, 160, 24, "bnhd", 3), (110, 4, 0, 300, 64, 64, "bnhd", 3)]


def variants(outdir, calls):  # noqa: F811
    exe = os.path.join(outdir, "block_cover")
    if not os.path.exists(exe):
        _run([_tool("clang++"), "-O2", "-std=c++17", "-D__HIP_PLATFORM_AMD__", "-I", "/opt/rocm/include",
              "-I", os.path.join(ROOT, "include"), "-I", CSRC, os.path.join(HERE, "block_cover.cpp"), "-o", exe])
    out = subprocess.run([exe], input="\n".join(calls) + "\n", stdout=subprocess.PIPE, text=True, check=True).stdout
    return set(out.splitlines())


def test_the_cases_reach_every_variant_that_plans_choose(outdir):  # noqa: F811
    tested = [f"scan {t} {B} {N} {C}" for t in range(3) for B, N, C in scan.SHAPES + SCAN]
    tested += [f"conv {B} {N} {C} {K}" for K in range(2, 9) for B, N, C in conv.SHAPES + CONV]
    tested += [f"norm {B} {N} {H} {G} {D} {rot}" for B, H, G, N, D, rot, _, _ in norm.CASES + NORM]
    rows, lengths = (1, 2, 5, 16, 64, 300, 1000, 5000), (1, 7, 50, 64, 100, 129, 300, 1000, 5000, 70000)
    swept = [f"scan {t} {B} {N} {C}" for t in range(3) for B in rows for N in lengths for C in (1, 2, 64, 65, 130, 1000, 4096, 20001)]
    swept += [f"conv {B} {N} {C} {K}" for K in range(2, 9) for B in rows for N in lengths for C in (1, 3, 4, 7, 130, 1000, 4096)]
    swept += [f"norm {B} {N} {H} {G} {D} {rot}" for B in rows for N in lengths for H, G in ((1, 0), (1, 1), (4, 1), (16, 16), (32, 8))
              for D in range(8, 513, 8) for rot in sorted({0, 2, D // 4 * 2, D // 16 * 8, D})]
    left = variants(outdir, swept) - variants(outdir, tested)
    assert not left, "\n".join(sorted(left))


@pytest.fixture(scope="module")
def lc():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from fft_long_convolution_amd import lconv
    lconv.load()
    return lconv


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("how", scan.HOW, ids=lambda h: "-".join(map(str, h)))
def test_scan(lc, monkeypatch, dtype, how):
    monkeypatch.setattr(scan, "SHAPES", SCAN)
    scan.test_prompts(lc, dtype, how)
    scan.test_gradients(lc, dtype, how)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("K", [2, 3, 4, 5, 6, 7, 8])
def test_conv(lc, monkeypatch, dtype, K):
    monkeypatch.setattr(conv, "SHAPES", CONV)
    conv.test_prompts_and_gradients(lc, dtype, K, K % 2 == 0)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("case", NORM, ids=lambda c: "-".join(map(str, c)))
def test_norm(lc, dtype, case):
    i = NORM.index(case)
    norm.test_forward_and_gradients(lc, dtype, i % 2 == 0, i % 3 == 0, case)
