"""The gated linear recurrence on the GPU against its float64 definition: prompts, gradients, single tokens."""
import numpy as np
import pytest

from oracle import block
from tests.mixer_util import host, off_by, say, tdtype, wide

pytestmark = pytest.mark.gpu

# Beyond the one rounding of the result, relative to the magnitude of its terms: gates are off by a few units of 2^-24 to
# their own size (an exponential, a reciprocal, a root of one unit in the last place each, a handful of products), decays by
# as much in 1 - a, which over their whole memory adds up to once that; the state is rounded at every token, twice, which over
# a memory of a few hundred tokens walks some 20 units.
SLACK = 64 * 2.0 ** -24

HOW = [("sigmoid", "convex", False), ("rate", "norm", True), ("log", "plain", False), ("log", "norm", True),
       ("rate", "convex", False), ("sigmoid", "plain", True), ("sigmoid", "norm", False), ("rate", "plain", False),
       ("log", "convex", True)]

# (B, N, C): single tokens, ends inside a wave's turn and a tile, odd widths, more rows than one lane's channel covers,
# few rows cut into segments
SHAPES = [(1, 1, 1), (2, 3, 2), (3, 8, 64), (2, 9, 5), (1, 63, 65), (2, 64, 130), (3, 65, 7), (2, 200, 129), (257, 70, 2),
          (256, 130, 6), (1, 1000, 16), (2, 1537, 9), (1, 4100, 3)]


@pytest.fixture(scope="module")
def lc():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from fft_long_convolution_amd import lconv
    lconv.load()
    return lconv


def inputs(rng, B, N, C, dtype, gate, gated):
    """x, z, input_gate, rate on the host, memories of a few to a few hundred tokens."""
    import torch
    x = host(rng, (B, N, C), dtype)
    g = rng.standard_normal((B, N, C), dtype=np.float32)
    z = -np.exp(g - 3.0) if gate == "log" else g * np.float32(1.5) + np.float32(2.0 if gate == "sigmoid" else 0.0)
    rate = torch.from_numpy(rng.uniform(0.002, 0.5, C).astype(np.float32)) if gate == "rate" else None
    return x, torch.from_numpy(z).to(tdtype(dtype)), host(rng, (B, N, C), dtype) if gated else None, rate


def cuda(*ts):
    return [None if t is None else t.cuda() for t in ts]


def some_lengths(rng, B, N):
    import torch
    n = rng.integers(0, N + 1, B)
    n[: min(B, 3)] = [0, 1, N][: min(B, 3)]
    n[B - 1] = N if B != 2 else N - 1
    return torch.from_numpy(n.astype(np.int32))


def magnitude(x, z, i, rate, state, gate, mix, n):
    a = lambda t: None if t is None else np.abs(wide(t))  # noqa: E731
    return block.gated_scan(a(x), wide(z), gate, mix, wide(i), wide(rate), a(state), n)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("how", HOW, ids=lambda h: "-".join(map(str, h)))
def test_prompts(lc, dtype, how):
    gate, mix, gated = how
    rng = np.random.default_rng(700)
    for k, (B, N, C) in enumerate(SHAPES):
        x, z, i, rate = inputs(rng, B, N, C, dtype, gate, gated)
        state = host(rng, (B, C), "f32") if k % 2 else None
        n = some_lengths(rng, B, N) if k % 3 else None
        say(f"[scan] {dtype} {how} {(B, N, C)} state={state is not None} ragged={n is not None}")
        dx, dz, di, dr, ds, dn = cuda(x, z, i, rate, state, n)
        y, last, marks = lc.gated_scan(dx, dz, gate, mix, di, dr, ds, dn)
        assert marks is None
        args = [wide(t) for t in (i, rate, state)]
        ry, rl = block.gated_scan(wide(x), wide(z), gate, mix, *args, n)
        sy, sl = magnitude(x, z, i, rate, state, gate, mix, n)
        e = off_by(y, ry, dtype, np.maximum(sy, 1e-6)), off_by(last, rl, "f32", np.maximum(sl, 1e-6))
        say(f"   beyond the rounding: {e[0]:.1e} {e[1]:.1e} (at most {SLACK:.1e})")
        assert max(e) <= SLACK
        if n is not None:
            for b in range(B):
                assert not bool(y[b, int(n[b]):].any())
        # with marks, and the state in place
        again = lc.gated_scan(dx, dz, gate, mix, di, dr, ds, dn, need_marks=True, state_out=ds)
        assert bool((again.y == y).all()) and bool((again.state == last).all())
        if ds is not None:
            assert again.state is ds


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("how", HOW, ids=lambda h: "-".join(map(str, h)))
def test_gradients(lc, dtype, how):
    gate, mix, gated = how
    rng = np.random.default_rng(701)
    for k, (B, N, C) in enumerate(SHAPES):
        x, z, i, rate = inputs(rng, B, N, C, dtype, gate, gated)
        dy = host(rng, (B, N, C), dtype)
        state, dstate = (host(rng, (B, C), "f32"), host(rng, (B, C), "f32")) if k % 2 else (None, None)
        n = some_lengths(rng, B, N) if k % 3 else None
        say(f"[scan gradients] {dtype} {how} {(B, N, C)} state={state is not None} ragged={n is not None}")
        gx, gz, gi, gr, gs, gds, gn, gdy = cuda(x, z, i, rate, state, dstate, n, dy)
        marks = lc.gated_scan(gx, gz, gate, mix, gi, gr, gs, gn, need_marks=True).marks
        g = lc.gated_scan_bwd(gdy, gx, gz, marks, gate, mix, gi, gr, gds, gn)
        args = dict(gate=gate, mix=mix, input_gate=wide(i), rate=wide(rate), lengths=n)
        want = block.gated_scan_bwd(wide(dy), wide(x), wide(z), state=wide(state), dstate=wide(dstate), **args)
        a = lambda t: None if t is None else np.abs(wide(t))  # noqa: E731
        size = block.gated_scan_bwd(a(dy), a(x), wide(z), state=a(state), dstate=a(dstate), size=True, **args)
        for name, got, r, s in zip(("dx", "dz", "di", "drate", "dstate"), g, want, size):
            assert (got is None) == (r is None), name
            if got is None:
                continue
            kind = "f32" if name in ("drate", "dstate") else dtype
            # dz of a saturated gate is small beside G h: its factor 1 - s is right to its own size, so is the product
            e = off_by(got, r, kind, np.maximum(s, 1e-6))
            say(f"   {name}: {e:.1e} beyond the rounding (at most {SLACK:.1e})")
            assert e <= SLACK, name
        if n is not None:
            for b in range(B):
                assert not bool(g.dx[b, int(n[b]):].any()) and not bool(g.dz[b, int(n[b]):].any())
        # what is not asked for is not made, and leaves the rest as it is
        h = lc.gated_scan_bwd(gdy, gx, gz, marks, gate, mix, gi, gr, gds, gn, need_drate=False, need_dstate=False)
        assert h.drate is None and h.dstate is None and bool((h.dx == g.dx).all()) and bool((h.dz == g.dz).all())


def test_slices_of_a_packed_projection(lc):
    """Operands and outputs as slices of one token-major buffer; nothing beside them is touched."""
    import torch
    say("[scan slices]")
    rng = np.random.default_rng(702)
    B, N, C = 3, 100, 40
    packed = host(rng, (B, N, 5 * C), "bf16").cuda()
    kept = packed.clone()
    x, z, i, out, rest = packed.split(C, dim=-1)
    want = lc.gated_scan(x.contiguous(), z.contiguous(), "sigmoid", "norm", i.contiguous(), need_marks=True)
    got = lc.gated_scan(x, z, "sigmoid", "norm", i, out=out, need_marks=True)
    assert got.y.data_ptr() == out.data_ptr() and bool((out == want.y).all()) and bool((got.marks == want.marks).all())
    assert bool((packed[..., : 3 * C] == kept[..., : 3 * C]).all()) and bool((rest == kept[..., 4 * C:]).all())
    dy = host(rng, (B, N, 2 * C), "bf16").cuda()[..., C:]
    a = lc.gated_scan_bwd(dy, x, z, got.marks, "sigmoid", "norm", i)
    b = lc.gated_scan_bwd(dy.contiguous(), x.contiguous(), z.contiguous(), want.marks, "sigmoid", "norm", i.contiguous())
    assert all(bool((p == q).all()) for p, q in zip(a, b) if p is not None)
    # time-major memory
    t = host(rng, (N, B, C), "f32").cuda().transpose(0, 1)
    assert bool((lc.gated_scan(t, -t.abs(), "log").y == lc.gated_scan(t.contiguous(), -t.abs().contiguous(), "log").y).all())
    # one token's gate repeated over a row
    g = z[:, :1].expand(B, N, C)
    assert bool((lc.gated_scan(x, g, "sigmoid").y == lc.gated_scan(x, g.contiguous(), "sigmoid").y).all())
    only = torch.empty((B, N, C), dtype=torch.bfloat16, device="cuda")
    assert lc.gated_scan(x, z, out=only, need_state=False).state is None


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("how", HOW, ids=lambda h: "-".join(map(str, h)))
def test_single_tokens(lc, dtype, how):
    """A prompt token by token, from states in a pool, idle rows among them."""
    import torch
    gate, mix, gated = how
    rng = np.random.default_rng(703)
    for B, C in ((1, 1), (5, 7), (3, 130), (64, 2)):
        N = 6
        say(f"[scan tokens] {dtype} {how} {(B, C)}")
        x, z, i, rate = inputs(rng, B, N, C, dtype, gate, gated)
        slots = torch.from_numpy(rng.permutation(2 * B)[:B].astype(np.int32))
        pool = host(rng, (2 * B, C), "f32")
        first = pool[slots.long()]
        idle = B > 1
        if idle:
            slots[1] = -1 if B % 2 else 2 * B
        gx, gz, gi, gr, gs, gp = cuda(x, z, i, rate, slots, pool.clone())
        ry, rl = block.gated_scan(wide(x), wide(z), gate, mix, wide(i), wide(rate), wide(first))
        sy, sl = magnitude(x, z, i, rate, first, gate, mix, None)
        for t in range(N):
            y = lc.gated_scan_step(gx[:, t], gz[:, t], gp, gate, mix, None if gi is None else gi[:, t], gr, slots=gs)
            for b in range(B):
                if idle and b == 1:
                    assert not bool(y[b].any())
                else:
                    assert off_by(y[b], ry[b, t], dtype, np.maximum(sy[b, t], 1e-6)) <= SLACK
        for b in range(B):
            if not (idle and b == 1):
                assert off_by(gp[int(slots[b])], rl[b], "f32", np.maximum(sl[b], 1e-6)) <= SLACK
        others = sorted(set(range(2 * B)) - {int(s) for s in slots})
        assert bool((gp.cpu()[others] == pool[others]).all())
        if not idle:
            p = pool.cuda()
            assert bool((lc.gated_scan_step(gx[:, 0], gz[:, 0], p, gate, mix, None if gi is None else gi[:, 0], gr)).isfinite().all())


def test_long_memories_do_not_drift(lc):
    """4096 silent tokens under gates that stay where they are, memories of 10 to 30000 tokens: a decay's rounding to fp32
    would add up to 4096 times 2^-25 (1.2e-4); two roundings a token walk 64 times 2^-23 (8e-6), taken four times."""
    import torch
    say("[scan drift]")
    rng = np.random.default_rng(704)
    B, N, C = 1, 4096, 256
    la = -np.exp(rng.uniform(np.log(3e-5), np.log(2e-3), C)).astype(np.float32)
    z = torch.from_numpy(np.broadcast_to(la, (B, N, C)).copy()).cuda()
    state = torch.ones((B, C), device="cuda")
    x = torch.zeros((B, N, C), device="cuda")
    bound = 4 * 64 * 2.0 ** -23
    e = np.abs(wide(lc.gated_scan(x, z, "log", state=state).state)[0] / np.exp(N * la.astype(np.float64)) - 1)
    say(f"   largest drift {e.max():.1e} (at most {bound:.1e})")
    assert e.max() <= bound
    pool = torch.ones((1, C), device="cuda")
    for _ in range(N):
        lc.gated_scan_step(x[:, 0], z[:, 0], pool, "log")
    e = np.abs(wide(pool)[0] / np.exp(N * la.astype(np.float64)) - 1)
    say(f"   token by token {e.max():.1e}")
    assert e.max() <= bound


def test_values_that_are_not_finite(lc):
    """Padding may hold anything; a NaN reaches its own channel's later tokens (gradients: earlier ones) and nothing else."""
    import torch
    say("[scan not finite]")
    rng = np.random.default_rng(705)
    B, N, C = 2, 150, 70
    x, z, i, _ = inputs(rng, B, N, C, "bf16", "sigmoid", True)
    dy = host(rng, (B, N, C), "bf16")
    n = torch.tensor([100, 37], dtype=torch.int32)
    clean = cuda(x, z, i, dy)
    bad = [t.clone() for t in clean]
    for t in bad:
        for b in range(B):
            t[b, int(n[b]):] = float("nan")
    f = lambda t: lc.gated_scan(t[0], t[1], "sigmoid", "norm", t[2], lengths=n.cuda(), need_marks=True)  # noqa: E731
    a, b = f(clean), f(bad)
    assert bool((a.y == b.y).all()) and bool((a.state == b.state).all()) and bool(b.y.isfinite().all())
    g = lambda t, m: lc.gated_scan_bwd(t[3], t[0], t[1], m, "sigmoid", "norm", t[2], lengths=n.cuda())  # noqa: E731
    for p, q in zip(g(clean, a.marks), g(bad, b.marks)):
        assert p is None or bool((p == q).all())
    for where in range(3):
        t = [v.clone() for v in clean[:3]]
        t[where][0, 41, 13] = float("nan")
        y = lc.gated_scan(t[0], t[1], "sigmoid", "norm", t[2]).y
        w = lc.gated_scan(*clean[:2], "sigmoid", "norm", clean[2]).y
        hit = torch.zeros_like(y, dtype=torch.bool)
        hit[0, 41:, 13] = True
        assert bool((y.isnan() == hit).all()) and bool((y[~hit] == w[~hit]).all())
    d = clean[3].clone()
    d[1, 20, 5] = float("inf")
    m = lc.gated_scan(*clean[:2], "sigmoid", "norm", clean[2], need_marks=True).marks
    got = lc.gated_scan_bwd(d, *clean[:2], m, "sigmoid", "norm", clean[2])
    hit = torch.zeros_like(d, dtype=torch.bool)
    hit[1, :21, 5] = True
    assert bool((~got.dx.isfinite() == hit).all())
    # gates at their ends: no memory, nothing forgotten, no way in
    z = torch.zeros((1, 4, 2), device="cuda")
    z[:, :, 0], z[:, :, 1] = float("-inf"), float("inf")
    y = lc.gated_scan(torch.ones_like(z), z, "sigmoid", "norm", state=torch.full((1, 2), 3.0, device="cuda"), need_marks=True)
    assert y.y[0].tolist() == [[1.0, 3.0]] * 4
    g = lc.gated_scan_bwd(torch.ones_like(z), torch.ones_like(z), z, y.marks, "sigmoid", "norm")
    assert all(bool(t.isfinite().all()) for t in g if t is not None)
    y = lc.gated_scan(torch.ones_like(z), torch.full_like(z, float("-inf")), "log").y
    assert bool((y == 1.0).all())


def test_lengths_outside_the_row_and_empty_calls(lc):
    import torch
    say("[scan lengths]")
    x = torch.randn(3, 20, 8, device="cuda")
    n = torch.tensor([-5, 99, 4], dtype=torch.int32, device="cuda")
    m = torch.tensor([0, 20, 4], dtype=torch.int32, device="cuda")
    a, b = lc.gated_scan(x, x, lengths=n), lc.gated_scan(x, x, lengths=m)
    assert bool((a.y == b.y).all()) and bool((a.state == b.state).all())
    s = torch.randn(3, 8, device="cuda")
    e = lc.gated_scan(x[:, :0], x[:, :0], state=s, need_marks=True)
    assert e.y.shape == (3, 0, 8) and bool((e.state == s).all())
    g = lc.gated_scan_bwd(x[:, :0], x[:, :0], x[:, :0], e.marks, "rate", rate=torch.ones(8, device="cuda"), dstate=s)
    assert bool((g.dstate == s).all()) and not bool(g.drate.any())
    assert lc.gated_scan(x[:0], x[:0]).y.shape == (0, 20, 8)
    g = lc.gated_scan_bwd(x[:0], x[:0], x[:0], e.marks, "rate", rate=torch.ones(8, device="cuda"))
    assert not bool(g.drate.any())
    assert lc.gated_scan_step(x[:0, 0], x[:0, 0], s).shape == (0, 8)


def test_offsets_past_32_bits(lc):
    import torch
    say("[scan 64-bit offsets]")
    rng = np.random.default_rng(706)
    x = host(rng, (2, 70, 16), "bf16").cuda()
    buf = torch.empty(2 ** 31 + 70 * 64 + 4096, dtype=torch.bfloat16, device="cuda")
    far = buf.as_strided((2, 70, 16), (2 ** 31 + 64, 32, 1))
    far.copy_(x)
    out = buf.as_strided((2, 70, 16), (2 ** 31 + 64, 32, 1), 16)
    want = lc.gated_scan(x, x, "sigmoid", "norm", need_marks=True)
    got = lc.gated_scan(far, far, "sigmoid", "norm", out=out, need_marks=True)
    assert bool((out == want.y).all()) and bool((got.marks == want.marks).all()) and bool((far == x).all())
    a, b = lc.gated_scan_bwd(far, far, far, got.marks, "sigmoid", "norm"), lc.gated_scan_bwd(x, x, x, want.marks, "sigmoid", "norm")
    assert bool((a.dx == b.dx).all()) and bool((a.dz == b.dz).all())


def test_graphs_streams_and_repeats(lc):
    """Captured and replayed on new inputs, on a side stream, twice over: the same bits."""
    import torch
    say("[scan graphs]")
    rng = np.random.default_rng(707)
    B, N, C = 2, 700, 24                  # cut into segments: workspaces and both launches
    assert lc.lconv_gated_scan_workspace_bytes(B, N, C, lc.BF16) > 0
    new = lambda: cuda(*inputs(rng, B, N, C, "bf16", "rate", True)[:3], host(rng, (B, N, C), "bf16"))  # noqa: E731
    rate = torch.linspace(0.01, 0.4, C, device="cuda")
    x, z, i, dy = new()
    pool = torch.zeros((B, C), device="cuda")

    def step():
        f = lc.gated_scan(x, z, "rate", "norm", i, rate, need_marks=True)
        g = lc.gated_scan_bwd(dy, x, z, f.marks, "rate", "norm", i, rate, dstate=f.state)
        pool.copy_(f.state)
        t = lc.gated_scan_step(x[:, 0], z[:, 0], pool, "rate", "norm", i[:, 0], rate)
        return f.y, f.state, g.dx, g.dz, g.dinput_gate, g.drate, g.dstate, t, pool

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
        for t, v in zip((x, z, i, dy), new()):
            t.copy_(v)
        want = [t.clone() for t in step()]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(bool((a == b).all()) for a, b in zip(held, want))
    # a stream given by hand
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    y = lc.gated_scan(x, z, "rate", "norm", i, rate, stream=other).y
    torch.cuda.current_stream().wait_stream(other)
    assert bool((y == want[0]).all())


def test_against_differences(lc):
    """<dy, y(v + e d) - y(v - e d)> / 2e from forward calls in fp32 against the gradients: e = 1/64, so the difference's own
    error is e^2 / 6 of third derivatives of order one (4e-5) and 2^-24 / e of the terms (4e-6)."""
    import torch
    say("[scan differences]")
    rng = np.random.default_rng(708)
    B, N, C = 2, 40, 33
    x, z, i, rate = cuda(*inputs(rng, B, N, C, "f32", "rate", True))
    s, dy = host(rng, (B, C), "f32").cuda(), host(rng, (B, N, C), "f32").cuda()
    f = lambda x, z, i, rate, s: lc.gated_scan(x, z, "rate", "norm", i, rate, s)  # noqa: E731
    marks = lc.gated_scan(x, z, "rate", "norm", i, rate, s, need_marks=True).marks
    g = lc.gated_scan_bwd(dy, x, z, marks, "rate", "norm", i, rate)
    args = [x, z, i, rate, s]
    for k, grad in enumerate(g):
        d = torch.from_numpy(rng.standard_normal(args[k].shape).astype(np.float32)).cuda()
        e = 1.0 / 64
        if k == 3:
            d = d * rate                   # rates stay positive
        hi, lo = ([a + (sg * e * d if j == k else 0) for j, a in enumerate(args)] for sg in (1, -1))
        want = float(((f(*hi).y.double() - f(*lo).y.double()) * dy.double()).sum()) / (2 * e)
        terms = float((grad.double() * d.double()).abs().sum())
        got = float((grad.double() * d.double()).sum())
        say(f"   argument {k}: {got:.5f} against {want:.5f} of {terms:.1f}")
        assert abs(got - want) <= 2e-4 * terms


@pytest.mark.parametrize("N", [60, 3000])
def test_states_in_place(lc, N):
    """One buffer for the state that enters and the one that leaves, in one piece and cut into segments, many rows: the same
    bits as with two."""
    import torch
    say(f"[scan states in place] {N}")
    rng = np.random.default_rng(709)
    B, C = 2, 1400
    x, z, _, _ = cuda(*inputs(rng, B, N, C, "bf16", "sigmoid", False))
    assert (lc.lconv_gated_scan_workspace_bytes(B, N, C, lc.BF16) > 0) == (N > 60)
    s, dy = host(rng, (B, C), "f32").cuda(), host(rng, (B, N, C), "bf16").cuda()
    want = lc.gated_scan(x, z, state=s, need_marks=True)
    ds = lc.gated_scan_bwd(dy, x, z, want.marks, dstate=s)
    st = torch.cuda.current_stream().cuda_stream
    ws = torch.empty(lc.lconv_gated_scan_bwd_workspace_bytes(B, N, C, 1, lc.BF16) or 16, dtype=torch.uint8, device="cuda")
    for _ in range(5):
        t = s.clone()
        got = lc.gated_scan(x, z, state=t, state_out=t)
        assert bool((got.y == want.y).all()) and bool((t == want.state).all())
        t, dx, dz = s.clone(), torch.empty_like(x), torch.empty_like(x)
        assert lc.lconv_gated_scan_bwd(dy.data_ptr(), None, x.data_ptr(), None, z.data_ptr(), None, None, None, None,
                                       want.marks.data_ptr(), t.data_ptr(), None, dx.data_ptr(), None, dz.data_ptr(), None, None,
                                       None, None, t.data_ptr(), B, N, C, 1, lc.BF16, ws.data_ptr(), ws.numel(), st) == 0
        assert bool((t == ds.dstate).all()) and bool((dx == ds.dx).all()) and bool((dz == ds.dz).all())
