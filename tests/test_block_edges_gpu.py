"""The recurrence, the short convolution and the q/k norms at the edges of what a call may be: many and wide rows, operands that
are broadcast or of other orders, one tensor in several places, calls on two streams at once, graphs that share their memory."""
import numpy as np
import pytest

from oracle import block
from tests.mixer_util import host, off_by, say, wide
from tests.test_gated_scan_gpu import SLACK

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lc():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from fft_long_convolution_amd import lconv
    lconv.load()
    return lconv


def same(a, b):
    return all((p is None) == (q is None) and (p is None or bool((p == q).all())) for p, q in zip(a, b))


@pytest.mark.parametrize("B,N,C", [(70001, 1, 3), (33000, 2, 64), (2, 9, 100003), (1, 1, 70000)])
def test_many_and_wide_rows(lc, B, N, C):
    """Some rows and channels against float64: rows and channels do not meet."""
    import torch
    say(f"[edges] {(B, N, C)}")
    rng = np.random.default_rng(1100)
    x, z, dy = (host(rng, (B, N, C), "bf16") for _ in range(3))
    w = host(rng, (C, 4), "bf16", 0.5)
    gx, gz, gdy, gw = x.cuda(), z.cuda(), dy.cuda(), w.cuda()
    f = lc.gated_scan(gx, gz, "sigmoid", "convex", need_marks=True)
    g = lc.gated_scan_bwd(gdy, gx, gz, f.marks, "sigmoid", "convex")
    c, _ = lc.short_conv(gx, gw, activation="silu")
    h = lc.short_conv_bwd(gdy, gx, gw, activation="silu")
    rows = np.unique(np.r_[0, B - 1, rng.integers(0, B, 6)])
    cols = np.unique(np.r_[0, C - 1, max(C - 5, 0), rng.integers(0, C, 9)])
    at = lambda t: wide(t)[np.ix_(rows, range(N), cols)]  # noqa: E731
    X, Z, D, W = at(x), at(z), at(dy), wide(w)[cols]
    ry, rl = block.gated_scan(X, Z, "sigmoid", "convex")
    size, last = block.gated_scan(np.abs(X), Z, "sigmoid", "convex")
    e = off_by(f.y.cpu()[rows][:, :, cols], ry, "bf16", np.maximum(size, 1e-6))
    e = max(e, off_by(f.state.cpu()[rows][:, cols], rl, "f32", np.maximum(last, 1e-6)))
    want = block.gated_scan_bwd(D, X, Z, gate="sigmoid", mix="convex")
    size = block.gated_scan_bwd(np.abs(D), np.abs(X), Z, gate="sigmoid", mix="convex", size=True)
    for got, r, s in zip(g[:2], want, size):
        e = max(e, off_by(got.cpu()[rows][:, :, cols], r, "bf16", np.maximum(s, 1e-6)))
    p, _ = block.short_conv(X, W, None, True)
    terms, _ = block.short_conv(np.abs(X), np.abs(W), None, False)
    e = max(e, off_by(c.cpu()[rows][:, :, cols], p, "bf16", np.maximum(terms, 1e-6)))
    r = block.short_conv_bwd(D, X, W, None, True)
    # p' is at most 1.1 and its own slope at most 1/2, times what p's terms are off by
    s = block.short_conv_bwd(np.abs(D) * (1.1 + 0.5 * terms), np.abs(X), np.abs(W), None, False)
    e = max(e, off_by(h.dx.cpu()[rows][:, :, cols], r[0], "bf16", np.maximum(s[0], 1e-6)))
    say(f"   beyond the rounding: {e:.1e} (at most {SLACK:.1e})")
    assert e <= SLACK
    if N == 1:
        pool = torch.zeros((B, C), device="cuda")
        y = lc.gated_scan_step(gx[:, 0], gz[:, 0], pool, "sigmoid", "convex")
        assert off_by(y.cpu()[rows][:, cols], ry[:, 0], "bf16", np.maximum(np.abs(ry[:, 0]), 1e-6)) <= SLACK


@pytest.mark.parametrize("N", [37, 900])
def test_broadcast_operands_and_orders(lc, N):
    """Bit for bit what dense copies give."""
    import torch
    say(f"[edges] orders {N}")
    rng = np.random.default_rng(1101)
    B, C = 3, 70
    one = host(rng, (1, N, C), "bf16").cuda().expand(B, N, C)             # every row alike
    step = host(rng, (B, 1, C), "bf16").cuda().expand(B, N, C)            # every token alike
    late = host(rng, (N, B, C), "bf16").cuda().transpose(0, 1)            # tokens outside
    w = host(rng, (C, 5), "bf16").cuda()
    dense = lambda *t: [v.contiguous() for v in t]  # noqa: E731
    for x, z, i, dy in ((one, step, late, late), (late, one, step, one), (step, late, one, step), (late, late, late, late)):
        for gate, mix in (("sigmoid", "norm"), ("sigmoid", "plain")):
            f = lc.gated_scan(x, z, gate, mix, i, need_marks=True)
            a, b, c, d = dense(x, z, i, dy)
            want = lc.gated_scan(a, b, gate, mix, c, need_marks=True)
            assert same(f, want)
            assert same(lc.gated_scan_bwd(dy, x, z, f.marks, gate, mix, i), lc.gated_scan_bwd(d, a, b, want.marks, gate, mix, c))
        assert same(lc.short_conv(x, w), lc.short_conv(a, w))
        assert same(lc.short_conv_bwd(dy, x, w, activation="silu"), lc.short_conv_bwd(d, a, w, activation="silu"))
    # y in another order than its inputs
    y = torch.empty((N, B, C), dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    assert bool((lc.gated_scan(one, late, out=y).y == lc.gated_scan(*dense(one, late)).y).all())
    assert bool((lc.short_conv(late, w, out=y)[0] == lc.short_conv(late.contiguous(), w)[0]).all())
    # one k head for all, one position's q for all, and the same gradient for both
    H, D = 6, 64
    q = host(rng, (B, 1, N, D), "f16").cuda().expand(B, H, N, D)
    k = host(rng, (B, H, 1, D), "f16").cuda().expand(B, H, N, D)
    v = torch.ones(D, dtype=torch.float16, device="cuda")
    f, _ = lc.rotary_frequencies(D)
    assert same(lc.qk_norm_rotary(q, k, v, v, None, f), lc.qk_norm_rotary(*dense(q, k), v, v, None, f))
    assert same(lc.qk_norm_rotary_bwd(q, q, q, k, v, v, None, f), lc.qk_norm_rotary_bwd(*dense(q, q, q, k), v, v, None, f))


def work(lc, rng, seed):
    """A forward and backward pass of all three, with workspaces; returns a call that gives its results."""
    import torch
    B, N, C, H, D = 2, 1500 + 64 * seed, 96, 6, 16
    x, z, i, dy = (host(rng, (B, N, C), "bf16").cuda() for _ in range(4))
    w, v = host(rng, (C, 4), "bf16").cuda(), torch.ones(D, dtype=torch.bfloat16, device="cuda")
    rate = torch.linspace(0.01, 0.3, C, device="cuda")
    f, _ = lc.rotary_frequencies(D)
    assert lc.lconv_gated_scan_workspace_bytes(B, N, C, lc.BF16) > 0

    def run():
        c, _ = lc.short_conv(x, w, activation="silu", need_state=False)
        s = lc.gated_scan(c, z, "rate", "norm", i, rate, need_marks=True)
        heads = s.y.view(B, N, H, D).transpose(1, 2)
        q, _ = lc.qk_norm_rotary(heads, None, v, None, None, f)
        g = lc.qk_norm_rotary_bwd(dy.view(B, N, H, D).transpose(1, 2), None, heads, None, v, None, None, f)
        b = lc.gated_scan_bwd(g.dq.transpose(1, 2).reshape(B, N, C), c, z, s.marks, "rate", "norm", i, rate)
        e = lc.short_conv_bwd(b.dx, x, w, activation="silu")
        return c, s.y, s.state, q, g.dq, g.dq_weight, b.dx, b.dz, b.dinput_gate, b.drate, b.dstate, e.dx, e.dweight

    return run, (x, z, i, dy)


def test_two_streams_at_once(lc):
    import torch
    say("[edges] two streams")
    rng = np.random.default_rng(1102)
    runs = [work(lc, rng, k)[0] for k in range(2)]
    want = [[t.clone() for t in run()] for run in runs]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [[], []]
    for _ in range(8):
        for k, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[k].append(runs[k]())
    for s in streams:
        torch.cuda.current_stream().wait_stream(s)
    assert all(same(r, want[k]) for k in range(2) for r in got[k])


def test_graphs_that_share_their_memory(lc):
    """Two graphs from one pool, replayed in turn with eager calls between: workspaces hold nothing from one call to the next."""
    import torch
    say("[edges] graphs")
    rng = np.random.default_rng(1103)
    runs, data = zip(*(work(lc, rng, k) for k in range(2)))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for run in runs:
            run()
    torch.cuda.current_stream().wait_stream(side)
    graphs, held = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()], []
    for k in range(2):
        with torch.cuda.graph(graphs[k], pool=graphs[0].pool() if k else None):
            held.append(runs[k]())
    for _ in range(3):
        for k in range(2):
            for t in data[k]:
                t.copy_(torch.randn_like(t))
            want = [t.clone() for t in runs[k]()]
            torch.cuda.synchronize()
            graphs[k].replay()
            torch.cuda.synchronize()
            assert same(held[k], want)
