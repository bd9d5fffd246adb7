"""Every form of the gated recurrence -- kind of gate, mix, with and without an input gate, each a kernel of its own -- against its
float64 definition, at sizes that take one and two channels to a lane, whole rows and segments; the first tests (CPU) hold the list
of forms against all that there are, and the sizes against what the plans can choose.  Gradients under memories of thousands of
tokens."""
import itertools

import numpy as np
import pytest

from tests import test_gated_scan_gpu as scan
from tests.mixer_util import say, wide
from tests.test_block_cover import SCAN, lc, variants  # noqa: F401
from tests.test_gated_scan_gpu import HOW
from tests.test_sanitizers import outdir  # noqa: F401

# beside HOW, whose forms run at test_gated_scan_gpu.py's and test_block_cover.py's sizes
MORE = [("sigmoid", "plain", False), ("sigmoid", "convex", True), ("sigmoid", "norm", True), ("rate", "plain", True),
        ("rate", "convex", True), ("rate", "norm", False), ("log", "plain", True), ("log", "convex", False), ("log", "norm", False)]
SIZES = [(2, 3, 2), (2, 64, 130), (1, 1000, 16), (257, 70, 66), (130, 30, 128), (520, 70, 3), (3, 600, 70)]


def test_every_form_has_a_case():
    forms = set(itertools.product(("log", "sigmoid", "rate"), ("plain", "convex", "norm"), (False, True)))
    assert set(HOW) | set(MORE) == forms and len(HOW) + len(MORE) == len(forms)


def test_every_form_runs_at_every_width_and_cut(outdir):  # noqa: F811
    """A kernel is chosen by type, pass, form, channels to a lane, and whether a row is cut."""
    def kernels(shapes):
        shapes = list(shapes)
        lines = variants(outdir, [f"scan {t} {B} {N} {C}" for t in range(3) for B, N, C in shapes])
        return {(v.split(":")[0], v.split("channels ")[1][0], v.split(", ")[-1]) for v in lines}
    rows, lengths = (1, 2, 5, 16, 64, 300, 1000, 5000), (1, 7, 50, 64, 100, 129, 300, 1000, 5000, 70000)
    swept = kernels(itertools.product(rows, lengths, (1, 2, 64, 65, 130, 1000, 4096, 20001)))
    assert len(swept) == 4 + 2 * 8      # fp32 has one channel to a lane
    assert not swept - kernels(SIZES) and not swept - kernels(scan.SHAPES + SCAN)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("how", MORE, ids=lambda h: "-".join(map(str, h)))
def test_forms(lc, monkeypatch, dtype, how):  # noqa: F811
    monkeypatch.setattr(scan, "SHAPES", SIZES)
    scan.test_prompts(lc, dtype, how)
    scan.test_gradients(lc, dtype, how)
    scan.test_single_tokens(lc, dtype, how)


@pytest.mark.gpu
@pytest.mark.parametrize("gate", ["log", "sigmoid", "rate"])
@pytest.mark.parametrize("B", [1, 40])
def test_gradients_of_long_memories_do_not_drift(lc, gate, B):  # noqa: F811
    """4096 silent tokens under gates that stay where they are, memories of 500 to 30000 tokens, a state of one that enters and a
    gradient of one at the last token, in segments (one row) and in one piece: with g = log a, dx_t = exp(g (N - 1 - t)), dz_t by
    dlog a = exp(g N), dstate = exp(g N).  Two roundings a token walk 64 times 2^-23, taken four times as for the states; a decay's
    logarithm, off by at most 16 2^-24 of itself (a sigmoid's exponent of up to 10.4), times 8.2 memories is within that."""
    import torch
    say(f"[scan drift of gradients] {gate} {B}")
    rng = np.random.default_rng(708)
    N, C = 4096, 256
    assert (lc.lconv_gated_scan_bwd_workspace_bytes(B, N, C, 0, lc.F32) > 0) == (B == 1)
    g = -np.exp(rng.uniform(np.log(3e-5), np.log(2e-3), C))
    rate, slope = None, np.ones(C)
    if gate == "log":
        z = g.astype(np.float32)
        g = z.astype(np.float64)
    elif gate == "sigmoid":
        z = (-np.log(np.expm1(-g))).astype(np.float32)
        g = -np.logaddexp(0.0, -z.astype(np.float64))
        slope = -np.expm1(g)                                # dlog a / dz
    else:
        z, r = np.zeros(C, np.float32), (-2.0 * g).astype(np.float32)
        g, slope, rate = -0.5 * r.astype(np.float64), -0.25 * r.astype(np.float64), torch.from_numpy(r).cuda()
    gz = torch.from_numpy(np.broadcast_to(z, (B, N, C)).copy()).cuda()
    x, dy = torch.zeros((B, N, C), device="cuda"), torch.zeros((B, N, C), device="cuda")
    dy[:, N - 1] = 1.0
    marks = lc.gated_scan(x, gz, gate, "plain", None, rate, torch.ones((B, C), device="cuda"), need_marks=True).marks
    got = lc.gated_scan_bwd(dy, x, gz, marks, gate, "plain", None, rate)
    whole = np.exp(g * N)
    want = {"dx": np.exp(g * (N - 1 - np.arange(N))[:, None]), "dz": np.broadcast_to(whole * slope, (N, C)), "dstate": whole}
    bound = 4 * 64 * 2.0 ** -23
    for name, w in want.items():
        e = np.abs(wide(getattr(got, name)) / w - 1.0).max()
        say(f"   {name}: {e:.1e} (at most {bound:.1e})")
        assert e <= bound, name
    if rate is not None:
        e = np.abs(wide(got.drate) / (-0.5 * B * N * whole) - 1.0).max()
        say(f"   drate: {e:.1e}")
        assert e <= bound
