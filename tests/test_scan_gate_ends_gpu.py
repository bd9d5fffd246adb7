"""Gates of the recurrence at the ends of what fp32 holds, among them those whose 1 - a^2 the hardware's root instructions take for
zero: forward, gradients and single tokens, each result to its own size."""
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


def check(lc, x, z, dy, gate, rate, dtype, extra, gated):
    """Every result of a call with mix "norm"; extra [N, C]: what sqrt(1 - a^2) of a token may be off by beside SLACK, relative:
    it enters h with x, and so do dz, dinput_gate and drate."""
    import torch
    rng = np.random.default_rng(1301)
    i = host(rng, x.shape, dtype) if gated else None
    gx, gz, gdy, gr, gi = cuda(x, z, dy, rate, i)
    f = lc.gated_scan(gx, gz, gate, "norm", gi, gr, need_marks=True)
    g = lc.gated_scan_bwd(gdy, gx, gz, f.marks, gate, "norm", gi, gr)
    args = dict(gate=gate, mix="norm", rate=wide(rate), input_gate=wide(i))
    y, last = block.gated_scan(wide(x), wide(z), **args)
    X, D = np.abs(wide(x)), np.abs(wide(dy))
    (sy, sl), (ey, el) = (block.gated_scan(v, wide(z), **args) for v in (X, X * extra))
    want = block.gated_scan_bwd(wide(dy), wide(x), wide(z), **args)
    size, more = (block.gated_scan_bwd(D, v, wide(z), size=True, **args) for v in (X, X * extra))
    more = (size[0] * extra,) + more[1:4] + (0.0,)
    off = {"y": beyond(f.y, y, dtype, sy, ey), "state": beyond(f.state, last, "f32", sl, el)}
    for name, got, r, s, e in zip(("dx", "dz", "di", "drate", "dstate"), g, want, size, more):
        assert (got is None) == (r is None), name
        if got is not None:
            off[name] = beyond(got, r, "f32" if name in ("drate", "dstate") else dtype, s, e)
    # the first token by itself
    pool = torch.zeros((x.shape[0], x.shape[2]), device="cuda")
    t = lc.gated_scan_step(gx[:, 0], gz[:, 0], pool, gate, "norm", None if gi is None else gi[:, 0], gr)
    off["token"] = beyond(t, y[:, 0], dtype, sy[:, 0], ey[:, 0])
    say("   " + ", ".join(f"{k} {v:.2f}" for k, v in off.items()))
    assert max(off.values()) <= 1
    return f, g


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("gated", [False, True])
def test_decays_next_to_one(lc, dtype, gated):
    """log a down to the smallest number there is.  Its product with log2(e) and the one after are each rounded to a multiple of
    2^-149, off by 2^-150 at most: relative to a decay's distance from one, (1 / 1.44 + 1) 2^-150 / |log a|, and a root halves that."""
    import torch
    rng = np.random.default_rng(1300)
    ends = [-1e-44, -1e-43, -1e-41, -1e-39, -5.8e-39, -5.9e-39, -1.2e-38, -1e-30, -1e-12, -0.0]
    if dtype == "bf16":
        ends = [-1e-40, -1e-39, -5.7e-39, -5.9e-39, -1.2e-38, -1e-30, -1e-12, -0.0]
    for B, N, C in ((1, 1, 16), (2, 29, 20), (1, 70, 130), (1, 600, 20)):
        say(f"[gate ends] log {dtype} gated={gated} {(B, N, C)}")
        z = -np.exp(rng.standard_normal((B, N, C)) - 3.0)
        for t in range(N):
            for c in range(C):
                if (t + c) % 3 == 0:
                    z[:, t, c] = ends[(t * 7 + c) % len(ends)]
        z = torch.from_numpy(z.astype(np.float32)).to(tdtype(dtype))
        x, dy = host(rng, (B, N, C), dtype), host(rng, (B, N, C), dtype)
        w = np.abs(wide(z)).min(0)
        extra = np.where(w > 0, 2.0 ** -150 / np.maximum(w, 2.0 ** -149), 0.0)
        f, g = check(lc, x, z, dy, "log", None, dtype, extra, gated)
        closed = (z == 0).cuda()
        assert not bool(g.dx[closed].any()), "1 - a^2 of nothing is nothing"


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("gated", [False, True])
def test_rates_behind_closed_gates(lc, dtype, gated):
    """sigmoid(z) down to 2^-126; below, it and what it multiplies may be zero.  rate sigmoid(z) log2(e) and the product after are
    rounded as above; sigmoid(z) is off by 1.22 2^-24 |z| (log2(e) as a float, the product in the exponent), dz and drate by that
    and, through the root, half as much again."""
    import torch
    rng = np.random.default_rng(1302)
    ends = [-60.0, -68.0, -72.0, -75.0, -80.0, -83.0, -85.0, -86.0, -87.0, -90.0, -100.0]
    for B, N, C in ((1, 1, 22), (2, 29, 22), (1, 70, 130), (1, 600, 22)):
        say(f"[gate ends] rate {dtype} gated={gated} {(B, N, C)}")
        z = rng.standard_normal((B, N, C)) * 1.5
        for t in range(N):
            for c in range(C):
                if (t + c) % 3 == 0:
                    z[:, t, c] = ends[(t * 7 + c) % len(ends)]
        z = torch.from_numpy(z.astype(np.float32)).to(tdtype(dtype))
        rate = torch.from_numpy(np.where(np.arange(C) % 2, 0.002, 0.1).astype(np.float32))
        x, dy = host(rng, (B, N, C), dtype), host(rng, (B, N, C), dtype)
        zz = wide(z)[0]
        l = wide(rate) / (1.0 + np.exp(-zz))
        extra = np.where(zz < -87.3, 1.0, 2.0 ** -150 / np.maximum(l, 2.0 ** -149) + 2.0 ** -23 * np.abs(zz))
        check(lc, x, z, dy, "rate", rate, dtype, extra, gated)


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
