"""Linear attention with a decay for each head on the GPU (lconv_linattn_fwd, _bwd, _step) against the
float64 recurrence, at the sizes, masks, layouts and decays where it can go wrong."""
import numpy as np
import pytest

from oracle import mixer
from tests.mixer_util import TOL, TOL_F32, host, rel, rel_rows, say, tdtype, wide

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lc():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from fft_long_convolution_amd import lconv
    lconv.load()
    return lconv


def decays(H):
    """Memories from two tokens to about a thousand."""
    import torch
    return torch.from_numpy((-2.0 ** -np.linspace(1, 10, H)).astype(np.float32) if H > 1 else np.float32([-0.02]))


def inputs(seed, B, H, G, N, Dk, Dv, dtype, order="bhnd", state=True, lengths=None):
    import torch
    rng = np.random.default_rng(seed)
    d = {}
    for name, heads, D in (("q", H, Dk), ("k", G, Dk), ("v", G, Dv), ("dy", H, Dv)):
        if order == "bnhd":
            d[name] = host(rng, (B, N, heads, D), dtype).cuda().transpose(1, 2)
        else:
            d[name] = host(rng, (B, heads, N, D), dtype).cuda()
    d["ld"] = decays(H).cuda()
    d["state"] = host(rng, (B, H, Dk, Dv), "f32").cuda() if state else None
    d["dstate"] = host(rng, (B, H, Dk, Dv), "f32").cuda() if state else None
    d["lengths"] = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
    d["scale"] = Dk ** -0.5
    return d


def ref_fwd(d):
    return mixer.linattn(wide(d["q"]), wide(d["k"]), wide(d["v"]), wide(d["ld"]), d["scale"], wide(d["state"]),
                         wide(d["lengths"]))


def check_fwd(lc, d, dtype):
    y, S = lc.linear_attention(d["q"], d["k"], d["v"], d["ld"], state=d["state"], lengths=d["lengths"])
    ry, rS = ref_fwd(d)
    ey, eS = rel_rows(y, ry), rel_rows(S, rS)
    say(f"   y {ey:.2e} (tol {TOL[dtype]:.1e})  state {eS:.2e} (tol {TOL_F32:.1e})")
    assert y.dtype == d["q"].dtype and ey <= TOL[dtype] and eS <= TOL_F32
    return y, S


def check_bwd(lc, d, dtype, need_dl=True):
    g = lc.linear_attention_bwd(d["dy"], d["q"], d["k"], d["v"], d["ld"], state=d["state"], dstate=d["dstate"],
                                lengths=d["lengths"], need_dlog_decay=need_dl)
    r = mixer.linattn_bwd(wide(d["dy"]), wide(d["q"]), wide(d["k"]), wide(d["v"]), wide(d["ld"]), d["scale"],
                          wide(d["state"]), wide(d["dstate"]), wide(d["lengths"]))
    e = [rel_rows(g.dq, r[0]), rel_rows(g.dk, r[1]), rel_rows(g.dv, r[2])]
    es = rel_rows(g.dstate, r[3]) if g.dstate is not None else 0.0
    # a head's dlog_decay is a sum of products of either sign: measured against the root of the sum of
    # squares over the heads
    el = rel(g.dlog_decay, r[4]) if need_dl else 0.0
    say(f"   dq dk dv {e[0]:.2e} {e[1]:.2e} {e[2]:.2e}  dstate {es:.2e}  dlog_decay {el:.2e}")
    assert max(e) <= TOL[dtype] and es <= TOL_F32
    assert el <= (1e-4 if dtype == "f32" else TOL[dtype])
    return g


# (B, H, G, N, Dk, Dv, order, state, lengths)
CASES = [
    (1, 1, 1, 1, 8, 8, "bhnd", False, None),           # the smallest
    (2, 2, 1, 2, 16, 24, "bnhd", True, None),
    (1, 3, 3, 31, 64, 64, "bhnd", True, None),
    (1, 2, 2, 32, 128, 128, "bnhd", False, None),
    (1, 2, 2, 33, 40, 72, "bhnd", True, None),
    (2, 2, 2, 63, 128, 64, "bnhd", True, None),
    (1, 2, 1, 64, 64, 128, "bhnd", False, None),
    (1, 2, 2, 65, 88, 104, "bnhd", True, None),
    (1, 2, 2, 127, 256, 256, "bhnd", True, None),
    (1, 4, 2, 129, 136, 200, "bnhd", True, None),
    (6, 2, 1, 150, 48, 80, "bnhd", True, (0, 1, 150, 64, 65, 149)),   # rows of no and of one token
    (4, 3, 1, 77, 128, 128, "bhnd", False, (-5, 400, 0, 76)),         # taken as 0, N, 0, 76
    (1, 2, 2, 700, 64, 64, "bhnd", True, None),
    (3, 2, 2, 1030, 32, 16, "bnhd", True, (1030, 513, 3)),
    (1, 1, 1, 4100, 128, 128, "bhnd", True, None),     # a long row: split over its length
    (2, 4, 2, 1500, 72, 136, "bnhd", True, (1500, 700)),
    (3, 2, 1, 2600, 256, 128, "bnhd", True, (2600, 0, 1)),
    (1, 2, 2, 3001, 128, 24, "bhnd", False, None),
    # widths between the tiles', past the pipelined loop's start
    (1, 3, 3, 200, 24, 40, "bnhd", True, None),
    (1, 2, 2, 400, 16, 136, "bhnd", True, None),
    (2, 2, 2, 300, 96, 80, "bnhd", False, (300, 222)),
    (2, 2, 1, 333, 192, 192, "bnhd", True, None),
    (2, 2, 2, 257, 168, 184, "bhnd", True, (250, 257)),
    (1, 2, 2, 290, 248, 8, "bhnd", True, None),
]


# Enough rows for the wide column blocks, and lengths past the pipelined loop's start: checked on the first and the last
# batch row (every row is on its own)
MANY = [
    (9, 16, 4, 199, 128, 128, "bnhd", True, [199, 160, 1, 33, 64, 0, 199, 198, 193]),
    (25, 16, 16, 170, 128, 128, "bhnd", False, None),
    (25, 16, 8, 170, 128, 128, "bnhd", True, None),
    (13, 10, 5, 170, 256, 256, "bhnd", False, None),
    (33, 8, 2, 161, 64, 64, "bnhd", True, None),
]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("case", MANY, ids=lambda c: "-".join(map(str, c[:7])))
def test_many_rows(lc, dtype, case):
    B, H, G, N, Dk, Dv, order, state, lengths = case
    say(f"[linattn many] {dtype} {case}")
    d = inputs(700 + B, B, H, G, N, Dk, Dv, dtype, order, state, lengths)
    y, S = lc.linear_attention(d["q"], d["k"], d["v"], d["ld"], state=d["state"], lengths=d["lengths"])
    g = lc.linear_attention_bwd(d["dy"], d["q"], d["k"], d["v"], d["ld"], state=d["state"], dstate=d["dstate"],
                                lengths=d["lengths"])
    for b in (0, B - 1):
        e = {n: (t if n in ("ld", "scale") or t is None else t[b:b + 1]) for n, t in d.items()}
        ry, rS = ref_fwd(e)
        r = mixer.linattn_bwd(wide(e["dy"]), wide(e["q"]), wide(e["k"]), wide(e["v"]), wide(e["ld"]), e["scale"],
                              wide(e["state"]), wide(e["dstate"]), wide(e["lengths"]))
        errs = [rel_rows(t[b:b + 1], x) for t, x in zip((y, g.dq, g.dk, g.dv), (ry, r[0], r[1], r[2]))]
        eS = [rel_rows(S[b:b + 1], rS)] + ([rel_rows(g.dstate[b:b + 1], r[3])] if state else [])
        say(f"   row {b}: y dq dk dv " + " ".join(f"{v:.2e}" for v in errs) + " states " + " ".join(f"{v:.2e}" for v in eS))
        assert max(errs) <= TOL[dtype] and max(eS) <= TOL_F32


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c[:7])))
def test_forward(lc, dtype, case):
    B, H, G, N, Dk, Dv, order, state, lengths = case
    say(f"[linattn fwd] {dtype} {case}")
    check_fwd(lc, inputs(100 + N, B, H, G, N, Dk, Dv, dtype, order, state, lengths), dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c[:7])))
def test_gradients(lc, dtype, case):
    B, H, G, N, Dk, Dv, order, state, lengths = case
    say(f"[linattn bwd] {dtype} {case}")
    check_bwd(lc, inputs(200 + N, B, H, G, N, Dk, Dv, dtype, order, state, lengths), dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_what_lies_past_a_rows_length_is_not_read(lc, dtype):
    """NaN and infinities in the masked places change no bit."""
    say(f"[linattn masked] {dtype}")
    lengths = (0, 1, 64, 100, 191)
    d = inputs(7, 5, 4, 2, 191, 64, 72, dtype, "bnhd", True, lengths)
    y0, S0 = check_fwd(lc, d, dtype)
    g0 = check_bwd(lc, d, dtype)
    for i, n in enumerate(lengths):
        for name in ("q", "k", "v", "dy"):
            d[name][i, :, n:] = float("nan")
            d[name][i, :, n::3] = float("inf")
    y, S = lc.linear_attention(d["q"], d["k"], d["v"], d["ld"], state=d["state"], lengths=d["lengths"])
    g = lc.linear_attention_bwd(d["dy"], d["q"], d["k"], d["v"], d["ld"], state=d["state"], dstate=d["dstate"],
                                lengths=d["lengths"], need_dlog_decay=True)
    for a, b in zip((y0, S0) + tuple(g0), (y, S) + tuple(g)):
        assert bool((a == b).all())
    assert float(y[0].abs().max()) == 0.0 and bool((S[0] == d["state"][0]).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_decays_at_the_ends_of_their_range(lc, dtype):
    """No decay, the slightest, a fast one, and none of the past at all (minus infinity)."""
    import torch
    say(f"[linattn decays] {dtype}")
    d = inputs(8, 2, 5, 5, 200, 64, 64, dtype)
    d["ld"] = torch.tensor([0.0, -1e-7, -30.0, float("-inf"), -3e38], device="cuda")
    check_fwd(lc, d, dtype)
    # the decay's gradient at gamma = 0 is 0 in the oracle's units (d/dlog)
    check_bwd(lc, d, dtype)


def test_f16_scores_and_states_beyond_the_types_range(lc):
    """Scores of 1e6 and states past 65504 with results that fp16 holds: the operands are scaled."""
    say("[linattn f16 range]")
    d = inputs(9, 1, 2, 2, 300, 128, 64, "f16", state=False)
    for name, s in (("q", 100.0), ("k", 100.0), ("v", 1e-3)):
        d[name] = (d[name].float() * s).half()
    check_fwd(lc, d, "f16")
    d = inputs(10, 1, 2, 2, 300, 64, 64, "f16", state=False)
    d["q"], d["k"], d["v"] = (d["q"].float() * 2e-4).half(), (d["k"].float() * 300).half(), (d["v"].float() * 300).half()
    d["dy"] = (d["dy"].float() * 1e-3).half()
    d["ld"] = d["ld"] * 0
    check_fwd(lc, d, "f16")


def test_packed_projection_and_repeated_heads(lc):
    """q, k, v as slices of one [B, N, H + 2G, D] buffer, and k, v repeated over heads by a zero stride."""
    import torch
    say("[linattn packed]")
    rng = np.random.default_rng(11)
    B, H, G, N, D = 2, 4, 2, 100, 64
    packed = host(rng, (B, N, H + 2 * G, D), "bf16").cuda().transpose(1, 2)
    d = inputs(12, B, H, G, N, D, D, "bf16")
    d["q"], d["k"], d["v"] = packed[:, :H], packed[:, H:H + G], packed[:, H + G:]
    y, S = check_fwd(lc, d, "bf16")
    check_bwd(lc, d, "bf16")
    one = packed[:, H:H + 1].expand(B, H, N, D)
    d["k"] = one
    d["v"] = packed[:, H + G:H + G + 1].expand(B, H, N, D)
    check_fwd(lc, d, "bf16")
    # an output inside a wider buffer, between other data
    buf = torch.full((B, N, 3, H, D), 7.0, device="cuda", dtype=torch.bfloat16)
    out = buf[:, :, 1].transpose(1, 2)
    y1, _ = lc.linear_attention(d["q"], d["k"], d["v"], d["ld"], state=d["state"])
    y2, _ = lc.linear_attention(d["q"], d["k"], d["v"], d["ld"], state=d["state"], out=out)
    assert y2.data_ptr() == out.data_ptr() and bool((y1 == out).all())
    assert bool((buf[:, :, 0] == 7).all()) and bool((buf[:, :, 2] == 7).all())


def test_offsets_past_32_bits(lc):
    """Heads and tokens more than 2^31 elements apart."""
    import torch
    say("[linattn 64-bit offsets]")
    B, H, N, D = 1, 2, 70, 64
    step = 2 ** 31 + 64
    d = inputs(13, B, H, H, N, D, D, "bf16")
    buf = torch.empty(step + N * D, dtype=torch.bfloat16, device="cuda")
    ref = lc.linear_attention(d["q"], d["k"], d["v"], d["ld"], state=d["state"])
    far = buf.as_strided((B, H, N, D), (0, step, D, 1))
    far.copy_(d["k"])
    got = lc.linear_attention(d["q"], far, d["v"], d["ld"], state=d["state"])
    assert bool((ref[0] == got[0]).all()) and bool((ref[1] == got[1]).all())
    out = lc.linear_attention(d["q"], d["k"], d["v"], d["ld"], state=d["state"], out=far)[0]
    assert bool((out == ref[0]).all())
    tok = torch.empty(40 * (N - 1) * 2 ** 20 + 4096, dtype=torch.bfloat16, device="cuda")
    far = tok.as_strided((B, H, N, D), (0, D, 40 * 2 ** 20, 1))
    far.copy_(d["v"])
    got = lc.linear_attention(d["q"], d["k"], far, d["ld"], state=d["state"])
    assert bool((ref[0] == got[0]).all())


def test_state_in_place_pieces_and_single_tokens_agree(lc):
    """A prompt in one call, in pieces whose state is moved on in place, and token by token."""
    say("[linattn pieces]")
    B, H, G, N, D = 2, 4, 2, 150, 64
    d = inputs(14, B, H, G, N, D, D, "f32")
    ry, rS = ref_fwd(d)
    S = d["state"].clone()
    for a, b in ((0, 1), (1, 70), (70, 134), (134, 150)):
        y, out = lc.linear_attention(d["q"][:, :, a:b], d["k"][:, :, a:b], d["v"][:, :, a:b], d["ld"], state=S, state_out=S)
        assert out.data_ptr() == S.data_ptr()
        assert rel(y, ry[:, :, a:b]) <= TOL["f32"]
    assert rel(S, rS) <= TOL_F32
    S = d["state"].clone()
    for t in range(N):
        y = lc.linear_attention_step(d["q"][:, :, t], d["k"][:, :, t], d["v"][:, :, t], d["ld"], S)
        assert rel(y, ry[:, :, t]) <= TOL["f32"], t
    assert rel(S, rS) <= TOL_F32


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("B,H,G,Dk,Dv", [(1, 1, 1, 8, 8), (3, 4, 2, 64, 64), (2, 6, 1, 128, 128), (1, 2, 2, 256, 256),
                                         (5, 3, 3, 40, 104), (70, 4, 4, 128, 64), (2, 2, 2, 136, 24)])
def test_single_tokens(lc, dtype, B, H, G, Dk, Dv):
    say(f"[linattn step] {dtype} {B, H, G, Dk, Dv}")
    d = inputs(300 + B, B, H, G, 1, Dk, Dv, dtype)
    ry, rS = ref_fwd(d)
    y = lc.linear_attention_step(d["q"][:, :, 0], d["k"][:, :, 0], d["v"][:, :, 0], d["ld"], d["state"])
    ey, eS = rel(y, ry[:, :, 0]), rel(d["state"], rS)
    say(f"   y {ey:.2e}  state {eS:.2e}")
    # the token form rounds nothing but its result
    assert ey <= TOL[dtype] and eS <= TOL_F32


def test_slots_choose_states_and_leave_the_others(lc):
    import torch
    say("[linattn slots]")
    d = inputs(15, 4, 4, 2, 1, 64, 64, "bf16")
    rng = np.random.default_rng(16)
    pool = host(rng, (6, 4, 64, 64), "f32").cuda()
    before = pool.clone()
    slots = torch.tensor([3, -1, 0, 99], dtype=torch.int32, device="cuda")
    y = lc.linear_attention_step(d["q"][:, :, 0], d["k"][:, :, 0], d["v"][:, :, 0], d["ld"], pool, slots=slots)
    d["state"] = before[[3, 1, 0, 2]]
    ry, rS = ref_fwd(d)
    for row, slot in ((0, 3), (2, 0)):
        assert rel(y[row], ry[row, :, 0]) <= TOL["bf16"] and rel(pool[slot], rS[row]) <= TOL_F32
    assert float(y[1].abs().max()) == 0 and float(y[3].abs().max()) == 0
    for slot in (1, 2, 4, 5):
        assert bool((pool[slot] == before[slot]).all())


def test_gradients_against_differences(lc):
    """The result is linear in q, in (k), in (v) and in the state, one at a time, so a difference of two
    forward calls is the directional derivative.  (The decay's gradient is set against differences of
    the float64 recurrence in test_mixer_oracle.py: over a step small enough for its curvature the
    rounding of fp32 results is larger than the difference.)"""
    say("[linattn differences]")
    d = inputs(17, 2, 4, 2, 130, 64, 48, "f32", lengths=(130, 77))
    g = lc.linear_attention_bwd(d["dy"], d["q"], d["k"], d["v"], d["ld"], state=d["state"], dstate=d["dstate"],
                                lengths=d["lengths"])

    def loss(**kw):
        e = dict(d, **kw)
        y, S = lc.linear_attention(e["q"], e["k"], e["v"], e["ld"], state=e["state"], lengths=e["lengths"])
        return float((y.double() * d["dy"].double()).sum() + (S.double() * d["dstate"].double()).sum())

    rng = np.random.default_rng(18)
    for name, grad in (("q", g.dq), ("k", g.dk), ("v", g.dv), ("state", g.dstate)):
        delta = host(rng, tuple(d[name].shape), "f32").cuda()
        want = loss(**{name: d[name] + delta}) - loss(**{name: d[name] - delta})
        got = 2 * float((grad.double() * delta.double()).sum())
        # the terms' sizes, not their sum, carry the rounding
        size = float((grad.double() * delta.double()).abs().sum())
        say(f"   {name}: {got:.6g} against {want:.6g}")
        assert abs(got - want) <= 1e-5 * size


def test_repeats_bit_for_bit_and_on_another_stream(lc):
    import torch
    say("[linattn repeat]")
    d = inputs(19, 2, 4, 2, 900, 128, 64, "bf16", lengths=(900, 555))
    runs = []
    side = torch.cuda.Stream()
    for s in (None, None, side):
        if s is not None:
            s.wait_stream(torch.cuda.current_stream())
        y, S = lc.linear_attention(d["q"], d["k"], d["v"], d["ld"], state=d["state"], lengths=d["lengths"], stream=s)
        g = lc.linear_attention_bwd(d["dy"], d["q"], d["k"], d["v"], d["ld"], state=d["state"], dstate=d["dstate"],
                                    lengths=d["lengths"], need_dlog_decay=True, stream=s)
        torch.cuda.synchronize()
        runs.append((y, S) + tuple(g))
    for other in runs[1:]:
        for a, b in zip(runs[0], other):
            assert bool((a == b).all())


def test_in_a_captured_graph(lc):
    """Forward, gradients and a token recorded once and replayed on changed inputs, with eager work
    between the replays."""
    import torch
    say("[linattn graph]")
    d = inputs(20, 2, 4, 2, 300, 64, 64, "bf16", lengths=(300, 100))
    tok = d["state"].clone()

    def go():
        y, S = lc.linear_attention(d["q"], d["k"], d["v"], d["ld"], state=d["state"], lengths=d["lengths"])
        g = lc.linear_attention_bwd(d["dy"], d["q"], d["k"], d["v"], d["ld"], state=d["state"], dstate=d["dstate"],
                                    lengths=d["lengths"], need_dlog_decay=True)
        z = lc.linear_attention_step(d["q"][:, :, 5], d["k"][:, :, 5], d["v"][:, :, 5], d["ld"], tok)
        return (y, S) + tuple(g) + (z,)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        go()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = go()
    for i in range(3):
        for name in ("q", "k", "v", "dy"):
            d[name].copy_(host(np.random.default_rng(40 + i), tuple(d[name].shape), "bf16").cuda())
        start = tok.clone()
        graph.replay()
        torch.cuda.synchronize()
        kept, moved = [t.clone() for t in out], tok.clone()
        tok.copy_(start)
        for a, b in zip(kept, go()):
            assert bool((a == b).all()), i
        assert bool((moved == tok).all())
        torch.cuda.synchronize()


def test_empty_calls(lc):
    import torch
    say("[linattn empty]")
    d = inputs(21, 2, 2, 2, 3, 16, 16, "bf16")
    e = lambda t, n: t[:, :, :n].contiguous()  # noqa: E731
    y, S = lc.linear_attention(e(d["q"], 0), e(d["k"], 0), e(d["v"], 0), d["ld"], state=d["state"])
    assert y.shape == (2, 2, 0, 16) and bool((S == d["state"]).all())
    y, S = lc.linear_attention(e(d["q"], 0), e(d["k"], 0), e(d["v"], 0), d["ld"])
    assert float(S.abs().max()) == 0
    g = lc.linear_attention_bwd(e(d["dy"], 0), e(d["q"], 0), e(d["k"], 0), e(d["v"], 0), d["ld"], state=d["state"],
                                dstate=d["dstate"], need_dlog_decay=True)
    assert bool((g.dstate == d["dstate"]).all()) and float(g.dlog_decay.abs().max()) == 0
    y, S = lc.linear_attention(d["q"][:0], d["k"][:0], d["v"][:0], d["ld"])
    assert y.shape == (0, 2, 3, 16) and S.shape == (0, 2, 16, 16)
    assert torch.cuda.synchronize() is None
