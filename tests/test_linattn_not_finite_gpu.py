"""Linear attention with values that are not finite: an infinity or a NaN at one token reaches what the definition lets it
reach -- its own and later tokens, for v its own column, for q its own token -- and nothing else changes."""
import numpy as np
import pytest

from tests.mixer_util import TOL, host, say

pytestmark = pytest.mark.gpu

BAD = {"inf": float("inf"), "-inf": float("-inf"), "nan": float("nan")}


@pytest.fixture(scope="module")
def lc():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from fft_long_convolution_amd import lconv
    lconv.load()
    return lconv


def make(seed, B, H, N, Dk, Dv, dtype):
    import torch
    rng = np.random.default_rng(seed)
    d = {n: host(rng, (B, H, N, D), dtype).cuda() for n, D in (("q", Dk), ("k", Dk), ("v", Dv), ("dy", Dv))}
    d["ld"] = torch.tensor(np.float32(-np.logspace(-3, 0, H)), device="cuda")
    d["state"], d["dstate"] = host(rng, (B, H, Dk, Dv), "f32").cuda(), host(rng, (B, H, Dk, Dv), "f32").cuda()
    return d


def run(lc, d):
    y, S = lc.linear_attention(d["q"], d["k"], d["v"], d["ld"], state=d["state"])
    g = lc.linear_attention_bwd(d["dy"], d["q"], d["k"], d["v"], d["ld"], state=d["state"], dstate=d["dstate"])
    return {"y": y, "S": S, "dq": g.dq, "dk": g.dk, "dv": g.dv, "dS": g.dstate}


def check(name, got, clean, reached, dtype):
    """`reached` (of the row's shape): not finite there; elsewhere as without the bad value.  (Elsewhere fp16's power of two
    for a neighbour's operands may be another one: to the type's rounding, not to the bit.)"""
    import torch
    got, clean = got.float(), clean.float()
    assert not bool(torch.isfinite(got[reached]).any()), f"{name}: a place that the value reaches is finite"
    rest = ~reached
    assert bool(torch.isfinite(got[rest]).all()), f"{name}: {int((~torch.isfinite(got) & rest).sum())} places out of its reach are not finite"
    e = float((got[rest] - clean[rest]).norm() / clean[rest].norm().clamp_min(1e-30))
    assert e <= TOL[dtype], (name, e)
    return e


SHAPES = [(1, 2, 70, 64, 72), (1, 1, 33, 128, 128), (25, 16, 170, 128, 128), (1, 2, 400, 40, 200), (1, 2, 1300, 64, 64), (9, 16, 200, 96, 96),
          (1, 2, 65, 256, 256)]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(map(str, s)))
def test_reach_of_v_and_its_like(lc, dtype, shape):
    """v in the forward, and the operands in v's place in the gradients' three roles: k for dq, q for dk, dy for dv."""
    import torch
    B, H, N, Dk, Dv = shape
    say(f"[linattn not finite] {dtype} {shape}")
    d = make(800 + N, B, H, N, Dk, Dv, dtype)
    clean = run(lc, d)
    rng = np.random.default_rng(801)
    tokens = sorted({0, 1, 15, 16, 17, 31, 32, N // 2, N - 2, N - 1})
    for i, t in enumerate(tokens):
        value = BAD[["inf", "nan", "-inf"][i % 3]]
        b, h = int(rng.integers(B)), int(rng.integers(H))
        before, after = torch.arange(N, device="cuda") <= t, torch.arange(N, device="cuda") >= t
        none = lambda n, D: torch.zeros(B, H, n, D, dtype=torch.bool, device="cuda")  # noqa: E731
        for name, D in (("v", Dv), ("dy", Dv), ("q", Dk), ("k", Dk)):
            c = int(rng.integers(D))
            x = d[name].clone()
            x[b, h, t, c] = value
            e = dict(d, **{name: x})
            got = run(lc, e)
            if name == "v":
                r = none(N, Dv)
                r[b, h, after, c] = True
                check("y", got["y"], clean["y"], r, dtype)
                r = none(Dk, Dv)
                r[b, h, :, c] = True
                check("S", got["S"], clean["S"], r, dtype)
            elif name == "dy":                       # dv_t = sum over i >= t of (q_i . k_t) dy_i
                r = none(N, Dv)
                r[b, h, before, c] = True
                check("dv", got["dv"], clean["dv"], r, dtype)
            elif name == "q":                        # dk_t = sum over i >= t of (v_t . dy_i) q_i
                r = none(N, Dk)
                r[b, h, before, c] = True
                check("dk", got["dk"], clean["dk"], r, dtype)
                r = none(N, Dv)
                r[b, h, t, :] = True                 # and one row of y
                check("y", got["y"], clean["y"], r, dtype)
            else:                                    # dq_i = sum over j <= i of (dy_i . v_j) k_j; y from the token on
                r = none(N, Dk)
                r[b, h, after, c] = True
                check("dq", got["dq"], clean["dq"], r, dtype)
                r = none(N, Dv)
                r[b, h, after, :] = True
                check("y", got["y"], clean["y"], r, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("value", ["inf", "nan"])
def test_reach_of_a_state_that_enters(lc, dtype, value):
    """An infinity or a NaN in one place of a state: its column of y and of the state that leaves, no other."""
    import torch
    say(f"[linattn state not finite] {dtype} {value}")
    for shape in ((2, 2, 70, 64, 72), (25, 16, 170, 128, 128), (1, 2, 1300, 64, 64)):
        B, H, N, Dk, Dv = shape
        d = make(820, B, H, N, Dk, Dv, dtype)
        clean = run(lc, d)
        x = d["state"].clone()
        x[B - 1, 1, 5, 37] = BAD[value]
        got = run(lc, dict(d, state=x))
        r = torch.zeros(B, H, N, Dv, dtype=torch.bool, device="cuda")
        r[B - 1, 1, :, 37] = True
        check("y", got["y"], clean["y"], r, dtype)
        r = torch.zeros(B, H, Dk, Dv, dtype=torch.bool, device="cuda")
        r[B - 1, 1, 5, 37] = True
        out = got["S"].clone()
        assert not bool(torch.isfinite(out[B - 1, 1, 5, 37]))
        keep = torch.ones(Dv, dtype=torch.bool, device="cuda")
        keep[37] = False
        e = float((out[..., keep] - clean["S"][..., keep]).norm() / clean["S"][..., keep].norm())
        assert bool(torch.isfinite(out[..., keep]).all()) and e <= TOL["f32"]
