"""Norms of q and k with their rotary positions on the GPU, and their gradients, against the float64 definitions."""
import numpy as np
import pytest

from oracle import block
from tests.mixer_util import host, off_by, say, wide

pytestmark = pytest.mark.gpu

# Beyond the one rounding of the result, relative to the magnitude of its terms: a mean and a mean square of a row (roundings
# that walk within lanes), a root and a quotient, a sine, three products and a sum.
SLACK = 16 * 2.0 ** -24
# Sums over rows: a few hundred roundings in a lane, then in a fixed tree.
SUMS = 64 * 2.0 ** -24

# (B, H, G, N, D, rot, order, first position)
CASES = [
    (1, 1, 1, 1, 8, 2, "bhnd", 0),
    (2, 3, 1, 5, 24, 6, "bnhd", 7),              # odd half
    (2, 4, 2, 33, 64, 64, "bhnd", 0),
    (1, 4, 4, 130, 128, 128, "bnhd", 1000),
    (3, 2, 1, 7, 96, 24, "bhnd", 30000),
    (1, 2, 2, 3, 80, 50, "bnhd", 123),           # halves at odd places
    (64, 4, 2, 1, 128, 128, "bhnd", 2 ** 30),    # positions that float32 does not hold
    (2, 5, 0, 9, 16, 0, "bnhd", 0),              # no k, no turn
    (1, 2, 1, 9, 256, 130, "bnhd", 100),
    (1, 2, 2, 4, 512, 512, "bhnd", 5),
    (2, 1, 1, 3, 512, 2, "bhnd", 5),             # the most units of a head
    (40, 6, 2, 300, 40, 40, "bnhd", 3),          # many items to a workgroup
]


@pytest.fixture(scope="module")
def lc():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from fft_long_convolution_amd import lconv
    lconv.load()
    return lconv


def heads(rng, B, H, N, D, dtype, order, scale=1.0):
    if order == "bnhd":
        return host(rng, (B, N, H, D), dtype, scale).cuda().transpose(1, 2)
    return host(rng, (B, H, N, D), dtype, scale).cuda()


def weight(rng, D, dtype):
    return (1.0 + 0.2 * host(rng, (D,), "f32")).to(host(rng, (1,), dtype).dtype).cuda()


def turned_size(v, rot, interleaved, magnitude):
    """Magnitudes of what a turn adds up."""
    v = np.abs(v).copy()
    lo, hi = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    v[..., lo] = magnitude * (v[..., lo] + v[..., hi])
    v[..., hi] = v[..., lo]
    return v


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("centred", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_forward_and_gradients(lc, dtype, centred, interleaved, case):
    import torch
    B, H, G, N, D, rot, order, first = case
    say(f"[qk norm] {dtype} centred={centred} interleaved={interleaved} {case}")
    rng = np.random.default_rng(800 + D)
    x = [heads(rng, B, n, N, D, dtype, order, 1.5) if n else None for n in (H, G)]
    dy = [heads(rng, B, n, N, D, dtype, order) if n else None for n in (H, G)]
    w = [weight(rng, D, dtype) if n else None for n in (H, G)]
    pos = torch.from_numpy(first + rng.integers(0, 50, (B, N)).astype(np.int32)).cuda()
    f = lc.rotary_frequencies(rot)[0] if rot else None
    mag, eps = 1.25, 1e-5
    how = dict(eps=eps, centred=centred, interleaved=interleaved, magnitude=mag)
    y = lc.qk_norm_rotary(x[0], x[1], w[0], w[1], pos, f, **how)
    g = lc.qk_norm_rotary_bwd(dy[0], dy[1], x[0], x[1], w[0], w[1], pos, f, **how)
    fr = wide(f) if rot else np.zeros(0)
    for i in range(2):
        if x[i] is None:
            assert y[i] is None and g[i] is None and g[2 + i] is None
            continue
        a, d, v = wide(x[i]), wide(dy[i]), wide(w[i])
        ry = block.qk_norm_rotary(a, v, wide(pos), fr, eps, centred, interleaved, mag)
        # a mean's terms are the values: its roundings go by sum |x| / D (each partial sum is at most sum |x|), however
        # small the mean itself is
        mean = np.abs(a).mean(-1, keepdims=True) if centred else 0.0
        u = a - a.mean(-1, keepdims=True) if centred else a
        r = 1.0 / np.sqrt((u * u).mean(-1, keepdims=True) + eps)
        sy = turned_size(r * (np.abs(a) + mean) * v, rot, interleaved, mag)
        e = off_by(y[i], ry, dtype, np.maximum(sy, 1e-6))
        rd, rw = block.qk_norm_rotary_bwd(d, a, v, wide(pos), fr, eps, centred, interleaved, mag)
        n = turned_size(d, rot, interleaved, mag)
        h, ub = n * v, np.abs(a) + mean
        sd = r * (h + ub * r * r * (h * ub).mean(-1, keepdims=True) + (h.mean(-1, keepdims=True) if centred else 0.0))
        sw = (n * ub * r).sum((0, 1, 2))
        ed, ew = off_by(g[i], rd, dtype, np.maximum(sd, 1e-6)), off_by(g[2 + i], rw, "f32", sw)
        say(f"   beyond the rounding: y {e:.1e}, dx {ed:.1e} (at most {SLACK:.1e}), dweight {ew:.1e} (at most {SUMS:.1e})")
        assert e <= SLACK and ed <= SLACK and ew <= SUMS
        assert all(p == q for m, p, q in zip(x[i].shape, x[i].stride(), y[i].stride()) if m > 1)


def test_alike_with_rotary_and_in_place(lc):
    """Weights of ones, rows of mean square one and a shared row of positions: what rotary gives; slices of one buffer, in place."""
    import torch
    say("[qk norm in place]")
    rng = np.random.default_rng(810)
    B, H, G, N, D = 2, 4, 2, 40, 64
    packed = host(rng, (B, N, H + 2 * G, D), "bf16").cuda().transpose(1, 2)
    kept = packed.clone()
    q, k = packed[:, :H], packed[:, H:H + G]
    pos = torch.arange(100, 100 + N, dtype=torch.int32, device="cuda")
    f, _ = lc.rotary_frequencies(48)
    wq, wk = weight(rng, D, "bf16"), weight(rng, D, "bf16")
    y = lc.qk_norm_rotary(q, k, wq, wk, pos, f)
    z = lc.qk_norm_rotary(q.contiguous(), k.contiguous(), wq, wk, pos[None].expand(B, N), f)
    assert all(bool((a == b).all()) for a, b in zip(y, z))
    lc.qk_norm_rotary(q, k, wq, wk, pos, f, out=(q, k))
    assert bool((q == y[0]).all()) and bool((k == y[1]).all()) and bool((packed[:, H + G:] == kept[:, H + G:]).all())
    ones = torch.ones(B, H, N, D, device="cuda")
    a = lc.qk_norm_rotary(ones, None, None, None, None, f, eps=0.0)[0]
    assert bool((a == lc.rotary(ones, None, None, f)[0]).all())
    assert lc.qk_norm_rotary_bwd(ones, None, ones, None, None, None, None, f).dq_weight is None
    only = lc.qk_norm_rotary_bwd(y[0], None, kept[:, :H], None, wq, None, pos, f)
    both = lc.qk_norm_rotary_bwd(y[0], y[1], kept[:, :H], kept[:, H:H + G], wq, wk, pos, f)
    assert bool((only.dq == both.dq).all()) and only.dk is None
    bare = lc.qk_norm_rotary_bwd(y[0], y[1], kept[:, :H], kept[:, H:H + G], wq, wk, pos, f, need_dweight=False)
    assert bare.dq_weight is None and bool((bare.dk == both.dk).all())


def test_rows_that_are_zero_or_not_finite(lc):
    import torch
    say("[qk norm not finite]")
    rng = np.random.default_rng(811)
    x = host(rng, (2, 3, 5, 48), "f32").cuda()
    f, _ = lc.rotary_frequencies(32)
    for centred in (False, True):
        want = lc.qk_norm_rotary(x, None, None, None, None, f, centred=centred)[0]
        bad = x.clone()
        bad[1, 2, 3, 7], bad[0, 0, 0, 47] = float("nan"), float("inf")
        bad[0, 1, 1] = 0.0
        y = lc.qk_norm_rotary(bad, None, None, None, None, f, centred=centred)[0]
        assert not bool(y[1, 2, 3].isfinite().any()) and not bool(y[0, 0, 0].isfinite().all()) and not bool(y[0, 1, 1].any())
        same = torch.ones(2, 3, 5, dtype=torch.bool, device="cuda")
        same[1, 2, 3] = same[0, 0, 0] = same[0, 1, 1] = False
        assert bool((y[same] == want[same]).all())
        g = lc.qk_norm_rotary_bwd(torch.ones_like(x), None, bad, None, None, None, None, f, centred=centred).dq
        assert bool(g[same].isfinite().all()) and bool(g[0, 1, 1].isfinite().all()) and not bool(g[1, 2, 3].isfinite().any())
    # a constant row, centred, is zero up to the roundings of its mean: eps keeps it there
    c = torch.full((1, 1, 1, 64), 1000.1, device="cuda")
    assert float(lc.qk_norm_rotary(c, None, None, None, None, None, eps=1e-6, centred=True)[0].abs().max()) <= 1e-3


def test_offsets_past_32_bits_and_empty_calls(lc):
    import torch
    say("[qk norm 64-bit offsets]")
    rng = np.random.default_rng(812)
    x = host(rng, (1, 2, 6, 64), "bf16").cuda()
    buf = torch.empty(2 ** 31 + 1024, dtype=torch.bfloat16, device="cuda")
    far = buf.as_strided((1, 2, 6, 64), (0, 2 ** 31 + 64, 64, 1))
    far.copy_(x)
    f, _ = lc.rotary_frequencies(64)
    want = lc.qk_norm_rotary(x, x, None, None, None, f)
    g = lc.qk_norm_rotary_bwd(x, x, x, x, None, None, None, f)
    h = lc.qk_norm_rotary_bwd(far, far, far, far, None, None, None, f)
    assert bool((h.dq == g.dq).all()) and bool((h.dk == g.dk).all())
    lc.qk_norm_rotary(far, None, None, None, None, f, out=(far, None))
    assert bool((far == want[0]).all())
    w = torch.ones(64, device="cuda", dtype=torch.bfloat16)
    e = lc.qk_norm_rotary_bwd(x[:, :, :0], x[:, :, :0], x[:, :, :0], x[:, :, :0], w, w, None, f)
    assert e.dq.shape == (1, 2, 0, 64) and not bool(e.dq_weight.any()) and not bool(e.dk_weight.any())
    assert lc.qk_norm_rotary(x[:0], None, None, None, None, f)[0].shape == (0, 2, 6, 64)


def test_graph_stream_and_repeats(lc):
    import torch
    say("[qk norm graph]")
    rng = np.random.default_rng(813)
    B, H, G, N, D = 4, 8, 2, 500, 128
    new = lambda n: heads(rng, B, n, N, D, "f16", "bnhd")  # noqa: E731
    q, k, dq, dk = new(H), new(G), new(H), new(G)
    wq, wk = weight(rng, D, "f16"), weight(rng, D, "f16")
    f, _ = lc.rotary_frequencies(D)

    def step():
        return (*lc.qk_norm_rotary(q, k, wq, wk, None, f), *lc.qk_norm_rotary_bwd(dq, dk, q, k, wq, wk, None, f))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        first = [t.clone() for t in step()]
    torch.cuda.current_stream().wait_stream(side)
    assert all(bool((a == b).all()) for a, b in zip(first, step()))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for _ in range(3):
        q.copy_(new(H))
        dk.copy_(new(G))
        want = [t.clone() for t in step()]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(bool((a == b).all()) for a, b in zip(held, want))


def test_against_differences(lc):
    """<dy, y(v + e d) - y(v - e d)> / 2e from forward calls in fp32, e = 1/64: its own error is e^2 / 6 of third derivatives of
    order one (4e-5) and 2^-24 / e of the terms (4e-6)."""
    import torch
    say("[qk norm differences]")
    rng = np.random.default_rng(814)
    x, dy = heads(rng, 2, 3, 7, 48, "f32", "bhnd"), heads(rng, 2, 3, 7, 48, "f32", "bhnd")
    w = weight(rng, 48, "f32")
    f, _ = lc.rotary_frequencies(32)
    for centred in (False, True):
        at = lambda x, w: lc.qk_norm_rotary(x, None, w, None, None, f, centred=centred, magnitude=1.1)[0].double()  # noqa: E731
        g = lc.qk_norm_rotary_bwd(dy, None, x, None, w, None, None, f, centred=centred, magnitude=1.1)
        for k, grad in ((0, g.dq), (1, g.dq_weight)):
            d = torch.from_numpy(rng.standard_normal(grad.shape).astype(np.float32)).cuda()
            e = 1.0 / 64
            hi, lo = ([v + (s * e * d if j == k else 0) for j, v in enumerate((x, w))] for s in (1, -1))
            want = float(((at(*hi) - at(*lo)) * dy.double()).sum()) / (2 * e)
            got, terms = float((grad.double() * d.double()).sum()), float((grad.double() * d.double()).abs().sum())
            say(f"   {got:.5f} against {want:.5f} of {terms:.1f}")
            assert abs(got - want) <= 2e-4 * terms
