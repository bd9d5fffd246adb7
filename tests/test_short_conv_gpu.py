"""The short causal convolution on the GPU against its float64 definition: prompts, gradients, single tokens."""
import numpy as np
import pytest

from oracle import block
from tests.mixer_util import host, off_by, say, wide

pytestmark = pytest.mark.gpu

# Beyond the one rounding of the result, relative to the magnitude of its terms: at most nine products added up, an exponential,
# a reciprocal and a few products.
SLACK = 16 * 2.0 ** -24
# Sums over tokens: some hundred roundings in a lane, then in a fixed tree.
SUMS = 64 * 2.0 ** -24

# (B, N, C): single tokens, rows shorter than the filter, ends of a run, widths that one lane's channels do not divide
SHAPES = [(1, 1, 1), (2, 3, 4), (3, 8, 7), (2, 33, 65), (5, 31, 256), (1, 200, 260), (40, 70, 12), (3, 1000, 20), (1, 16, 1030),
          (600, 40, 8)]


@pytest.fixture(scope="module")
def lc():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from fft_long_convolution_amd import lconv
    lconv.load()
    return lconv


def cuda(*ts):
    return [None if t is None else t.cuda() for t in ts]


def inputs(rng, B, N, C, K, dtype, some):
    x, w = host(rng, (B, N, C), dtype), host(rng, (C, K), dtype, K ** -0.5)
    return x, w, host(rng, (C,), dtype, 0.3) if some else None, host(rng, (B, K - 1, C), dtype) if some else None


def some_lengths(rng, B, N):
    import torch
    n = rng.integers(0, N + 1, B)
    n[: min(B, 4)] = [0, 1, min(2, N), N][: min(B, 4)]
    return torch.from_numpy(n.astype(np.int32))


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("K", [2, 3, 4, 5, 6, 7, 8])
@pytest.mark.parametrize("silu", [False, True])
def test_prompts_and_gradients(lc, dtype, K, silu):
    rng = np.random.default_rng(900 + K)
    act = "silu" if silu else None
    for k, (B, N, C) in enumerate(SHAPES):
        some, ragged = k % 2 == 0, k % 3 != 1
        x, w, b, s = inputs(rng, B, N, C, K, dtype, some)
        dy, ds = host(rng, (B, N, C), dtype), host(rng, (B, K - 1, C), dtype) if some else None
        n = some_lengths(rng, B, N) if ragged else None
        say(f"[conv] {dtype} K={K} silu={silu} {(B, N, C)} state={some} ragged={ragged}")
        gx, gw, gb, gs, gdy, gds, gn = cuda(x, w, b, s, dy, ds, n)
        y, last = lc.short_conv(gx, gw, gb, act, gs, gn)
        a = [wide(t) for t in (x, w, b, s)]
        ry, rl = block.short_conv(a[0], a[1], a[2], silu, a[3], n)
        m = [None if t is None else np.abs(t) for t in a]
        sp, _ = block.short_conv(m[0], m[1], m[2], False, m[3], n)
        e = off_by(y, ry, dtype, np.maximum(sp, 1e-6))
        assert np.array_equal(wide(last), rl) and e <= SLACK, e
        g = lc.short_conv_bwd(gdy, gx, gw, gb, act, gs, gds, gn)
        want = block.short_conv_bwd(wide(dy), a[0], a[1], a[2], silu, a[3], wide(ds), n)
        # p' is at most 1.1 and its own slope at most 1/2, times what p's terms are off by
        md = np.abs(wide(dy)) * (1.1 + 0.5 * sp if silu else 1.0)
        size = block.short_conv_bwd(md, m[0], m[1], None, False, m[3], None if ds is None else np.abs(wide(ds)), n)
        for name, got, r, z, kind, most in zip(("dx", "dweight", "dbias", "dstate"), g, want, size, (dtype, "f32", "f32", dtype),
                                               (SLACK, SUMS, SUMS, SLACK)):
            assert (got is None) == (name in ("dbias", "dstate") and not some), name
            if got is not None:
                e = off_by(got, r, kind, np.maximum(z, 1e-6))
                assert e <= most, (name, e)
        if ragged:
            for i in range(B):
                assert not bool(y[i, int(n[i]):].any()) and not bool(g.dx[i, int(n[i]):].any())
        # the state in place; what is not asked for is not made
        if some:
            t = gs.clone()
            again = lc.short_conv(gx, gw, gb, act, t, gn, state_out=t)
            assert again[1] is t and bool((t == last).all()) and bool((again[0] == y).all())
        bare = lc.short_conv_bwd(gdy, gx, gw, gb, act, gs, gds, gn, need_dweight=False)
        assert bare.dweight is None and bare.dbias is None and bool((bare.dx == g.dx).all())
        assert lc.short_conv(gx, gw, gb, act, gs, gn, need_state=False)[1] is None


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("K", [2, 4, 7])
def test_single_tokens(lc, dtype, K):
    """A prompt token by token, its inputs in a pool, idle rows among them."""
    import torch
    rng = np.random.default_rng(910 + K)
    for B, C in ((1, 1), (5, 7), (3, 132), (64, 4)):
        say(f"[conv tokens] {dtype} K={K} {(B, C)}")
        N = 10
        x, w, b, _ = inputs(rng, B, N, C, K, dtype, True)
        slots = torch.from_numpy(rng.permutation(2 * B)[:B].astype(np.int32))
        pool = host(rng, (2 * B, K - 1, C), dtype)
        first = pool[slots.long()]
        if B > 1:
            slots[1] = -1 if B % 2 else 2 * B
        gx, gw, gb, gs, gp = cuda(x, w, b, slots, pool.clone())
        ry, rl = block.short_conv(wide(x), wide(w), wide(b), True, wide(first))
        sp, _ = block.short_conv(*(np.abs(wide(t)) for t in (x, w, b)), False, np.abs(wide(first)))
        live = [i for i in range(B) if not (B > 1 and i == 1)]
        for t in range(N):
            y = lc.short_conv_step(gx[:, t], gw, gp, gb, "silu", gs)
            assert off_by(y[live], ry[live, t], dtype, np.maximum(sp[live, t], 1e-6)) <= SLACK
            if B > 1:
                assert not bool(y[1].any())
        assert np.array_equal(wide(gp[slots[live].long().cuda()]), rl[live])
        others = sorted(set(range(2 * B)) - {int(s) for s in slots})
        assert bool((gp.cpu()[others] == pool[others]).all())
        p = first.cuda()
        plain = lc.short_conv_step(gx[:, 0], gw, p)
        r, _ = block.short_conv(wide(x)[:, :1], wide(w), None, False, wide(first))
        assert off_by(plain, r[:, 0], dtype, np.maximum(sp[:, 0], 1e-6)) <= SLACK


def test_slices_padding_and_offsets(lc):
    import torch
    say("[conv slices]")
    rng = np.random.default_rng(920)
    B, N, C, K = 3, 50, 24, 4
    packed = host(rng, (B, N, 3 * C), "bf16").cuda()
    kept = packed.clone()
    w, n = host(rng, (C, K), "bf16").cuda(), torch.tensor([50, 0, 17], dtype=torch.int32, device="cuda")
    x, out, rest = packed.split(C, dim=-1)
    want = lc.short_conv(x.contiguous(), w, lengths=n)
    got = lc.short_conv(x, w, lengths=n, out=out)
    assert bool((out == want[0]).all()) and bool((got[1] == want[1]).all())
    assert bool((x == kept[..., :C]).all()) and bool((rest == kept[..., 2 * C:]).all())
    dy = host(rng, (B, N, 2 * C), "bf16").cuda()[..., C:]
    a, b = lc.short_conv_bwd(dy, x, w, lengths=n), lc.short_conv_bwd(dy.contiguous(), x.contiguous(), w, lengths=n)
    assert bool((a.dx == b.dx).all()) and bool((a.dweight == b.dweight).all())
    # an odd column to begin with, and a width that no vector holds
    v = packed[..., 1:8]
    w7 = w[:7].contiguous()
    assert bool((lc.short_conv(v, w7)[0] == lc.short_conv(v.contiguous(), w7)[0]).all())
    # padding may hold anything
    bad, bdy = x.contiguous(), dy.contiguous()
    for i in range(B):
        bad[i, int(n[i]):] = float("nan")
        bdy[i, int(n[i]):] = float("nan")
    c = lc.short_conv(bad, w, activation="silu", lengths=n)
    d = lc.short_conv(x.contiguous(), w, activation="silu", lengths=n)
    assert bool((c[0] == d[0]).all()) and bool((c[1] == d[1]).all())
    e = lc.short_conv_bwd(bdy, bad, w, activation="silu", lengths=n)
    f = lc.short_conv_bwd(dy, x, w, activation="silu", lengths=n)
    assert bool((e.dx == f.dx).all()) and bool((e.dweight == f.dweight).all())
    # a NaN reaches K tokens of its channel
    bad = x.contiguous().clone()
    bad[0, 20, 5] = float("nan")
    y = lc.short_conv(bad, w)[0]
    hit = torch.zeros_like(y, dtype=torch.bool)
    hit[0, 20:20 + K, 5] = True
    assert bool((y.isnan() == hit).all())
    # offsets past 32 bits
    buf = torch.empty(2 ** 31 + 64 * 50 + 4096, dtype=torch.bfloat16, device="cuda")
    far = buf.as_strided((2, 50, C), (2 ** 31 + 64, 48, 1))
    far.copy_(x[:2])
    assert bool((lc.short_conv(far, w)[0] == lc.short_conv(x[:2], w)[0]).all())
    g, h = lc.short_conv_bwd(far, far, w), lc.short_conv_bwd(x[:2], x[:2], w)
    assert bool((g.dx == h.dx).all()) and bool((g.dweight == h.dweight).all())


def test_empty_calls(lc):
    import torch
    say("[conv empty]")
    x, w, s = torch.randn(3, 20, 8, device="cuda"), torch.randn(8, 4, device="cuda"), torch.randn(3, 3, 8, device="cuda")
    y, last = lc.short_conv(x[:, :0], w, state=s)
    assert y.shape == (3, 0, 8) and bool((last == s).all())
    assert not bool(lc.short_conv(x[:, :0], w)[1].any())
    g = lc.short_conv_bwd(x[:, :0], x[:, :0], w, bias=w[:, 0].contiguous(), state=s, dstate=2 * s)
    assert bool((g.dstate == 2 * s).all()) and not bool(g.dweight.any()) and not bool(g.dbias.any())
    assert lc.short_conv(x[:0], w)[0].shape == (0, 20, 8) and not bool(lc.short_conv_bwd(x[:0], x[:0], w).dweight.any())
    assert lc.short_conv_step(x[:0, 0], w, s).shape == (0, 8)


def test_graph_stream_and_repeats(lc):
    import torch
    say("[conv graph]")
    rng = np.random.default_rng(930)
    B, N, C, K = 4, 300, 64, 4
    new = lambda: host(rng, (B, N, C), "bf16").cuda()  # noqa: E731
    x, dy, w, b = new(), new(), host(rng, (C, K), "bf16").cuda(), host(rng, (C,), "bf16").cuda()
    pool = torch.zeros(B, K - 1, C, dtype=torch.bfloat16, device="cuda")

    def step():
        y, s = lc.short_conv(x, w, b, "silu")
        pool.copy_(s)
        t = lc.short_conv_step(x[:, 5], w, pool, b, "silu")
        g = lc.short_conv_bwd(dy, x, w, b, "silu")
        return y, s, t, pool, g.dx, g.dweight, g.dbias

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        first = [t.clone() for t in step()]
    torch.cuda.current_stream().wait_stream(side)
    assert all(bool((p == q).all()) for p, q in zip(first, step()))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for _ in range(3):
        x.copy_(new())
        dy.copy_(new())
        want = [t.clone() for t in step()]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(bool((p == q).all()) for p, q in zip(held, want))


def test_against_differences(lc):
    """<dy, y(v + e d) - y(v - e d)> / 2e from forward calls in fp32, e = 1/64: its own error is e^2 / 6 of third derivatives of
    order one (4e-5) and 2^-24 / e of the terms (4e-6)."""
    import torch
    say("[conv differences]")
    rng = np.random.default_rng(931)
    B, N, C, K = 2, 40, 20, 5
    args = cuda(*inputs(rng, B, N, C, K, "f32", True))
    dy = host(rng, (B, N, C), "f32").cuda()
    f = lambda x, w, b, s: lc.short_conv(x, w, b, "silu", s)[0].double()  # noqa: E731
    g = lc.short_conv_bwd(dy, *args[:3], "silu", args[3])
    for k, grad in enumerate(g):
        d = torch.from_numpy(rng.standard_normal(grad.shape).astype(np.float32)).cuda()
        e = 1.0 / 64
        hi, lo = ([a + (s * e * d if j == k else 0) for j, a in enumerate(args)] for s in (1, -1))
        want = float(((f(*hi) - f(*lo)) * dy.double()).sum()) / (2 * e)
        got, terms = float((grad.double() * d.double()).sum()), float((grad.double() * d.double()).abs().sum())
        say(f"   argument {k}: {got:.5f} against {want:.5f} of {terms:.1f}")
        assert abs(got - want) <= 2e-4 * terms
