"""Every chunk kernel of linear attention that a plan can choose, run: the cases below reach each (type, contraction tiles,
column tiles, whole rows or segments, forward or gradients) with segments long enough for the pipelined loop.  The first test
holds the list against the plans (CPU), so that a retuned plan cannot leave a kernel without a case."""
import os
import subprocess

import numpy as np
import pytest

from oracle import mixer
from tests.linattn_ref import linattn_all
from tests.mixer_util import TOL, TOL_F32, rel_rows, say, wide
from tests.test_linattn_gpu import inputs
from tests.test_sanitizers import CSRC, HERE, ROOT, _run, _tool, outdir  # noqa: F401

# (type, rows, N, Dk, Dv); rows are batch rows of up to four heads
COVER = [
    ("bf16", 1, 170, 8, 40), ("bf16", 1, 170, 72, 128), ("bf16", 1, 170, 136, 200), ("bf16", 1, 170, 40, 8),
    ("bf16", 64, 170, 200, 40), ("bf16", 96, 170, 72, 200), ("bf16", 96, 170, 128, 8), ("bf16", 96, 170, 8, 136),
    ("bf16", 96, 170, 40, 136), ("bf16", 96, 170, 200, 136), ("bf16", 128, 263, 128, 192), ("bf16", 256, 263, 192, 128),
    ("bf16", 16, 700, 200, 136), ("bf16", 8, 1500, 128, 200), ("bf16", 8, 1500, 136, 200), ("bf16", 16, 1500, 64, 192),
    ("bf16", 16, 1500, 128, 136), ("bf16", 16, 1500, 200, 136), ("bf16", 32, 1500, 24, 40), ("bf16", 32, 1500, 24, 72),
    ("bf16", 32, 1500, 72, 128), ("bf16", 32, 1500, 64, 64), ("bf16", 32, 1500, 72, 64), ("bf16", 32, 8200, 192, 128),
    ("f16", 1, 170, 8, 40), ("f16", 1, 170, 72, 128), ("f16", 1, 170, 136, 200), ("f16", 1, 170, 40, 8),
    ("f16", 32, 170, 200, 200), ("f16", 96, 170, 128, 8), ("f16", 96, 170, 40, 136), ("f16", 96, 170, 8, 136),
    ("f16", 96, 170, 200, 136), ("f16", 400, 170, 72, 128), ("f16", 400, 170, 128, 72), ("f16", 16, 700, 128, 256),
    ("f16", 16, 700, 200, 200), ("f16", 8, 1500, 192, 256), ("f16", 16, 1500, 200, 136), ("f16", 32, 1500, 40, 136),
    ("f16", 32, 1500, 40, 200), ("f16", 32, 1500, 128, 200), ("f16", 64, 1500, 8, 40), ("f16", 64, 1500, 8, 72),
    ("f16", 64, 1500, 72, 40), ("f16", 16, 6001, 72, 128), ("f32", 1, 170, 8, 40), ("f32", 1, 170, 72, 128),
    ("f32", 1, 170, 136, 200), ("f32", 1, 170, 40, 8), ("f32", 1, 170, 128, 8), ("f32", 1, 170, 200, 8),
    ("f32", 96, 170, 136, 136), ("f32", 128, 170, 200, 136), ("f32", 64, 700, 200, 8), ("f32", 16, 1500, 136, 200),
    ("f32", 32, 1500, 136, 8), ("f32", 32, 1500, 200, 72), ("f32", 32, 1500, 96, 192), ("f32", 32, 1500, 128, 160),
    ("f32", 64, 1500, 40, 128), ("f32", 32, 8200, 8, 8),
]

TYPES = ("f32", "f16", "bf16")          # the order of lconv_dtype_t


def test_the_cases_reach_every_kernel_that_plans_choose(outdir):  # noqa: F811
    exe = os.path.join(outdir, "mixer_cover")
    _run([_tool("clang++"), "-O2", "-std=c++17", "-D__HIP_PLATFORM_AMD__", "-I", "/opt/rocm/include", "-I", os.path.join(ROOT, "include"),
          "-I", CSRC, os.path.join(HERE, "mixer_cover.cpp"), "-o", exe])
    text = "".join(f"{TYPES.index(t)} {r} {N} {Dk} {Dv}\n" for t, r, N, Dk, Dv in COVER)
    out = subprocess.run([exe], input=text, stdout=subprocess.PIPE, text=True, check=True).stdout
    assert out.strip().endswith("missing 0"), out
    none = subprocess.run([exe], input="", stdout=subprocess.PIPE, text=True, check=True).stdout
    assert not none.strip().endswith("missing 0")


def test_the_chunked_reference_is_the_oracle():
    r = np.random.default_rng(3)
    n = r.standard_normal
    d = dict(q=n((2, 4, 150, 3)), k=n((2, 2, 150, 3)), v=n((2, 2, 150, 5)), dy=n((2, 4, 150, 5)), ld=-np.exp(n(4) - 2), state=n((2, 4, 3, 5)),
             dstate=n((2, 4, 3, 5)), lengths=np.array([150, 77]))
    y, S = mixer.linattn(d["q"], d["k"], d["v"], d["ld"], 0.7, d["state"], d["lengths"])
    want = (y, S) + mixer.linattn_bwd(d["dy"], d["q"], d["k"], d["v"], d["ld"], 0.7, d["state"], d["dstate"], d["lengths"])[:4]
    for a, b in zip(linattn_all(d, 0.7), want):
        np.testing.assert_allclose(a, b, rtol=1e-10, atol=1e-11)


@pytest.mark.gpu
@pytest.mark.parametrize("case", COVER, ids=lambda c: "-".join(map(str, c)))
def test_kernel(case):
    """First and last batch row against float64, everything against a second run bit for bit; every third case with rows of
    different lengths, every other one with shared heads."""
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from fft_long_convolution_amd import lconv
    dtype, rows, N, Dk, Dv = case
    i = COVER.index(case)
    H = min(rows, 4)
    B, G = rows // H, max(H // 2, 1) if i % 2 else H
    lengths = [N - (37 * b) % min(N, 150) for b in range(B)] if i % 3 == 2 else None
    say(f"[linattn cover] {case} B={B} H={H} G={G} {'ragged' if lengths else ''}")
    d = inputs(1000 + i, B, H, G, N, Dk, Dv, dtype, ("bnhd", "bhnd")[i % 2], True, lengths)

    def run():
        y, S = lconv.linear_attention(d["q"], d["k"], d["v"], d["ld"], state=d["state"], lengths=d["lengths"])
        g = lconv.linear_attention_bwd(d["dy"], d["q"], d["k"], d["v"], d["ld"], state=d["state"], dstate=d["dstate"], lengths=d["lengths"])
        return y, S, g.dq, g.dk, g.dv, g.dstate

    got, again = run(), run()
    names = "y S dq dk dv dS".split()
    for name, a, b in zip(names, got, again):
        assert bool((a == b).all()), name
    for b in sorted({0, B - 1}):
        e = {n: (wide(t) if n == "ld" else t if n == "scale" or t is None else wide(t[b:b + 1])) for n, t in d.items()}
        for name, a, want in zip(names, got, linattn_all(e, d["scale"])):
            err, tol = rel_rows(a[b:b + 1], want), TOL_F32 if name in ("S", "dS") else TOL[dtype]
            say(f"   row {b} {name} {err:.2e}")
            assert err <= tol, (name, err, tol)
