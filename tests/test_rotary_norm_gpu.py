"""Rotary positions and layer norm on the GPU against their float64 definitions."""
import numpy as np
import pytest

from oracle import mixer
from tests.mixer_util import TOL, TOL_F32, host, off_by, rel, say, wide

pytestmark = pytest.mark.gpu

# Beyond the one rounding of the result (half a unit in the last place, element by element): the fp32
# arithmetic before it -- a sine, two products and a sum, or sums over a row whose roundings add like a
# random walk within lanes -- in fractions of the terms' size.
SLACK = 16 * 2.0 ** -24


@pytest.fixture(scope="module")
def lc():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from fft_long_convolution_amd import lconv
    lconv.load()
    return lconv


def heads(rng, B, H, N, D, dtype, order):
    if order == "bnhd":
        return host(rng, (B, N, H, D), dtype).cuda().transpose(1, 2)
    return host(rng, (B, H, N, D), dtype).cuda()


# (B, H, G, N, D, rot, order, first position)
ROTARY = [
    (1, 1, 1, 1, 8, 2, "bhnd", 0),
    (2, 3, 1, 5, 24, 6, "bnhd", 7),             # odd half, pairs that no vector holds
    (2, 4, 2, 33, 64, 64, "bhnd", 0),
    (1, 4, 4, 130, 128, 128, "bnhd", 1000),
    (3, 2, 1, 7, 96, 24, "bhnd", 30000),
    (1, 2, 2, 3, 80, 50, "bnhd", 123),          # halves at odd places
    (64, 4, 2, 1, 128, 128, "bhnd", 2 ** 30),   # positions float32 does not hold
    (1, 1, 1, 4, 1000, 1000, "bhnd", 5),
    (1, 2, 1, 9, 256, 130, "bnhd", 100),
]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("case", ROTARY, ids=lambda c: "-".join(map(str, c)))
def test_rotary(lc, dtype, interleaved, case):
    import torch
    B, H, G, N, D, rot, order, first = case
    say(f"[rotary] {dtype} interleaved={interleaved} {case}")
    rng = np.random.default_rng(400 + D)
    q, k = heads(rng, B, H, N, D, dtype, order), heads(rng, B, G, N, D, dtype, order)
    pos = torch.from_numpy(first + rng.integers(0, 50, (B, N)).astype(np.int32)).cuda()
    f, _ = lc.rotary_frequencies(rot, device="cuda")
    for inverse in (False, True):
        yq, yk = lc.rotary(q, k, pos, f, interleaved=interleaved, inverse=inverse, magnitude=1.25)
        for x, y in ((q, yq), (k, yk)):
            r = mixer.rotary(wide(x), wide(pos), wide(f), interleaved, inverse, 1.25)
            size = np.abs(mixer.rotary(np.abs(wide(x)), 0 * wide(pos), wide(f), interleaved, False, 1.25))
            lo, hi = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
            size[..., lo] += size[..., hi]
            size[..., hi] = size[..., lo]
            e = off_by(y, r, dtype, size)
            say(f"   {e:.2e} beyond the rounding (at most {SLACK:.1e})")
            assert e <= SLACK
            assert all(a == b for n, a, b in zip(x.shape, x.stride(), y.stride()) if n > 1)
            assert bool((y[..., rot:] == x[..., rot:]).all())


def test_rotary_in_place_shared_positions_and_gradient(lc):
    import torch
    say("[rotary in place]")
    rng = np.random.default_rng(410)
    B, H, G, N, D, rot = 2, 4, 2, 40, 64, 48
    packed = host(rng, (B, N, H + 2 * G, D), "bf16").cuda().transpose(1, 2)
    kept = packed.clone()
    q, k = packed[:, :H], packed[:, H:H + G]
    pos = torch.arange(100, 100 + N, dtype=torch.int32, device="cuda")
    f, _ = lc.rotary_frequencies(rot)
    yq, yk = lc.rotary(q, k, pos, f)
    zq, zk = lc.rotary(q, k, pos[None].expand(B, N), f)
    assert bool((yq == zq).all()) and bool((yk == zk).all())
    lc.rotary(q, k, pos, f, out=(q, k))
    assert bool((q == yq).all()) and bool((k == yk).all())
    assert bool((packed[:, H + G:] == kept[:, H + G:]).all())
    only, none = lc.rotary(kept[:, :H], None, pos, f)
    assert none is None and bool((only == yq).all())
    at0, _ = lc.rotary(kept[:, :H], None, None, f)
    assert bool((at0 == lc.rotary(kept[:, :H], None, torch.arange(N, dtype=torch.int32, device="cuda"), f)[0]).all())
    # <dy, R x> = <R^-1 dy, x>: the inverse turn is the gradient
    x, dy = host(rng, (B, H, N, D), "f32").cuda(), host(rng, (B, H, N, D), "f32").cuda()
    a = (dy.double() * lc.rotary(x, None, pos, f, magnitude=1.1)[0].double()).sum()
    b = (lc.rotary(dy, None, pos, f, magnitude=1.1, inverse=True)[0].double() * x.double()).sum()
    assert abs(float(a - b)) <= 1e-6 * float((dy * x).abs().sum())


def test_rotary_offsets_past_32_bits(lc):
    import torch
    say("[rotary 64-bit offsets]")
    rng = np.random.default_rng(411)
    x = host(rng, (1, 2, 6, 64), "bf16").cuda()
    buf = torch.empty(2 ** 31 + 1024, dtype=torch.bfloat16, device="cuda")
    far = buf.as_strided((1, 2, 6, 64), (0, 2 ** 31 + 64, 64, 1))
    far.copy_(x)
    f, _ = lc.rotary_frequencies(64)
    want = lc.rotary(x, None, None, f)[0]
    assert bool((lc.rotary(far, None, None, f)[0] == want).all())
    lc.rotary(far, None, None, f, out=(far, None))
    assert bool((far == want).all())


NORM = [(1, 1), (3, 2), (5, 7), (2, 63), (4, 64), (7, 100), (33, 256), (300, 257), (2, 1001), (9, 1024), (5, 2048),
        (3, 4096), (2, 4100), (2, 8192), (2, 12289), (1, 65536), (2000, 48), (1030, 768),
        # more rows than the gradient's workgroups have in hand
        (3100, 520), (1600, 1100), (520, 4096), (600, 2056), (530, 4104)]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,C", NORM)
def test_layer_norm(lc, dtype, rows, C):
    say(f"[norm] {dtype} {rows} x {C}")
    rng = np.random.default_rng(500 + C)
    x = (host(rng, (rows, C), "f32", 1.5) + host(rng, (rows, 1), "f32", 2.0)).to(host(rng, (1,), dtype).dtype).cuda()
    w, b, dy = host(rng, (C,), dtype).cuda(), host(rng, (C,), dtype).cuda(), host(rng, (rows, C), dtype).cuda()
    for weight, bias in ((w, b), (w, None), (None, b), (None, None)):
        y, mean, rstd = lc.layer_norm(x, weight, bias, eps=1e-5)
        ww = 1.0 if weight is None else wide(weight)
        ry, rm, rr = mixer.layer_norm(wide(x), ww, 0.0 if bias is None else wide(bias), 1e-5)
        # y: the terms are |x| rstd |w|, those of the mean, and |b|
        xh = (np.abs(wide(x)) + np.abs(wide(x)).mean(1, keepdims=True)) * rr[:, None]
        sy = xh * np.abs(ww) + (0.0 if bias is None else np.abs(wide(bias)))
        ey, em, er = off_by(y, ry, dtype, sy), rel(mean, rm), rel(rstd, rr)
        dx, dw, db = lc.layer_norm_bwd(dy, x, weight, mean, rstd)
        rx, rw, rb = mixer.layer_norm_bwd(wide(dy), wide(x), ww, wide(mean), wide(rstd))
        # dx: three terms that may cancel (C = 1: dx = 0); what was added up is the measure
        h = np.abs(ww * wide(dy))
        sx = rr[:, None] * (h + h.mean(1, keepdims=True) + xh * (h * xh).mean(1, keepdims=True))
        ex = off_by(dx, rx, dtype, sx)
        ew, eb = 0.0 if dw is None else rel(dw, rw), rel(db, rb)
        say(f"   y {ey:.2e} mean {em:.2e} rstd {er:.2e} dx {ex:.2e} dw {ew:.2e} db {eb:.2e}")
        assert ey <= SLACK and ex <= SLACK
        assert em <= TOL_F32 and er <= TOL_F32
        assert ew <= TOL_F32 and eb <= TOL_F32


def test_layer_norm_keeps_a_small_spread_on_a_large_mean(lc):
    """Values 1000 +- 0.1 in fp32: the variance comes from centred values."""
    say("[norm offset]")
    rng = np.random.default_rng(510)
    x = (1000.0 + 0.1 * host(rng, (20, 1000), "f32")).cuda()
    y, mean, rstd = lc.layer_norm(x, eps=1e-12)
    ry, rm, rr = mixer.layer_norm(wide(x), 1.0, 0.0, 1e-12)
    # the mean is stored to half a unit of 1000 (3e-5), a fraction 3e-4 of the spread
    assert rel(rstd, rr) <= 1e-5 and rel(y, ry) <= 3e-4


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_layer_norm_strided_in_place_and_shapes(lc, dtype):
    import torch
    say(f"[norm strided] {dtype}")
    rng = np.random.default_rng(520)
    wide_x = host(rng, (50, 999), dtype).cuda()
    x = wide_x[:, :300]                          # rows 999 apart: no two alike in their alignment
    w, b = host(rng, (300,), dtype).cuda(), host(rng, (300,), dtype).cuda()
    dy = host(rng, (50, 300), dtype).cuda()
    y, mean, rstd = lc.layer_norm(x, w, b)
    z, m2, r2 = lc.layer_norm(x.contiguous(), w, b)
    assert rel(y, wide(z)) <= TOL[dtype] and rel(mean, wide(m2)) <= TOL_F32
    dx, dw, db = lc.layer_norm_bwd(dy, x, w, mean, rstd)
    ex, ew, eb = lc.layer_norm_bwd(dy, x.contiguous(), w, mean, rstd)
    assert rel(dx, wide(ex)) <= 2 * TOL[dtype] and rel(dw, wide(ew)) <= TOL_F32 and rel(db, wide(eb)) <= TOL_F32
    keep = wide_x.clone()
    lc.layer_norm(x, w, b, out=x)
    assert bool((x == y).all()) and bool((wide_x[:, 300:] == keep[:, 300:]).all())
    g = dy.clone()
    out, dw2, db2 = lc.layer_norm_bwd(g, keep[:, :300], w, mean, rstd, out=g)
    assert out.data_ptr() == g.data_ptr() and bool((g == dx).all()) and bool((dw2 == dw).all()) and bool((db2 == db).all())
    t = host(rng, (3, 4, 300), dtype).cuda()
    y3, m3, _ = lc.layer_norm(t, w, b)
    y2, m2, _ = lc.layer_norm(t.reshape(12, 300), w, b)
    assert m3.shape == (3, 4) and bool((y3.reshape(12, 300) == y2).all())
    y0, m0, r0 = lc.layer_norm(t[:0], w, b)
    d0, w0, b0 = lc.layer_norm_bwd(t[:0], t[:0], w, m0, r0)
    assert y0.shape == (0, 4, 300) and float(w0.abs().max()) == 0 and float(b0.abs().max()) == 0
    assert torch.isfinite(y3.float()).all()


def test_layer_norm_nan_and_inf_stay_in_their_row(lc):
    import torch
    say("[norm nan]")
    rng = np.random.default_rng(530)
    x = host(rng, (8, 500), "f32").cuda()
    clean = lc.layer_norm(x)[0]
    x[2, 17] = float("nan")
    x[5, 400] = float("inf")
    y = lc.layer_norm(x)[0]
    for r in range(8):
        assert bool(torch.isnan(y[r]).any()) if r in (2, 5) else bool((y[r] == clean[r]).all())


def test_layer_norm_gradient_against_differences(lc):
    say("[norm differences]")
    rng = np.random.default_rng(540)
    x, dy, w, b = (host(rng, s, "f32").cuda() for s in ((6, 200), (6, 200), (200,), (200,)))
    y, mean, rstd = lc.layer_norm(x, w, b)
    dx, dw, db = lc.layer_norm_bwd(dy, x, w, mean, rstd)
    loss = lambda x, w, b: float((lc.layer_norm(x, w, b)[0].double() * dy.double()).sum())  # noqa: E731
    for i, g in enumerate((dx, dw, db)):
        args = [x, w, b]
        step = host(rng, tuple(args[i].shape), "f32").cuda()
        eps = 1e-2 if i == 0 else 1.0            # y is linear in weight and bias
        at = [[a + s * eps * step if j == i else a for j, a in enumerate(args)] for s in (1, -1)]
        want = (loss(*at[0]) - loss(*at[1])) / (2 * eps)
        got = float((g.double() * step.double()).sum())
        size = float((g.double() * step.double()).abs().sum())
        say(f"   {got:.6g} against {want:.6g}")
        # rounding of the two losses over the step; for x the third-order term, eps^2
        assert abs(got - want) <= (5e-4 if i == 0 else 1e-5) * size


def test_rotary_and_norm_repeat_in_a_captured_graph(lc):
    import torch
    say("[rotary, norm graph]")
    rng = np.random.default_rng(550)
    x = host(rng, (2, 40, 4, 64), "bf16").cuda()
    w, b = host(rng, (64,), "bf16").cuda(), host(rng, (64,), "bf16").cuda()
    f, _ = lc.rotary_frequencies(64)

    def go():
        y, mean, rstd = lc.layer_norm(x, w, b)
        q, k = lc.rotary(y.transpose(1, 2), y.transpose(1, 2)[:, :2], None, f)
        return (y, q, k) + tuple(lc.layer_norm_bwd(q.transpose(1, 2).contiguous(), x, w, mean, rstd))

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        go()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = go()
    for i in range(3):
        x.copy_(host(np.random.default_rng(60 + i), tuple(x.shape), "bf16").cuda())
        graph.replay()
        torch.cuda.synchronize()
        kept = [t.clone() for t in out]
        for a, b2 in zip(kept, go()):
            assert bool((a == b2).all()), i
        torch.cuda.synchronize()
