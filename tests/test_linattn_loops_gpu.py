"""Linear attention at 192 columns, whole rows in the pipelined chunk loop: the first and last batch row against the float64
recurrence and, whole, against a second run bit for bit (a stage read before its loads are in would differ from run to run)."""
import pytest

from oracle import mixer
from tests.mixer_util import TOL, TOL_F32, rel_rows, say, wide
from tests.test_linattn_gpu import inputs, lc, ref_fwd  # noqa: F401

pytestmark = pytest.mark.gpu


# (types, B, H, G, N, Dk, Dv)
LOOPS = [
    ("f32", 9, 16, 16, 200, 192, 192),
    ("f32 f16 bf16", 16, 16, 8, 330, 192, 160),
]


@pytest.mark.parametrize("dtype,case", [(t, c) for c in LOOPS for t in c[0].split()], ids=lambda x: x if isinstance(x, str) else "-".join(map(str, x[1:])))
def test_loops(lc, dtype, case):  # noqa: F811
    _, B, H, G, N, Dk, Dv = case
    say(f"[linattn loops] {dtype} {case[1:]}")
    check(lc, dtype, B, H, G, N, Dk, Dv)


def check(lc, dtype, B, H, G, N, Dk, Dv):  # noqa: F811
    d = inputs(900 + N, B, H, G, N, Dk, Dv, dtype, "bnhd", True, None)

    def run():
        y, S = lc.linear_attention(d["q"], d["k"], d["v"], d["ld"], state=d["state"])
        return (y, S) + tuple(lc.linear_attention_bwd(d["dy"], d["q"], d["k"], d["v"], d["ld"], state=d["state"], dstate=d["dstate"]))[:4]

    got, again = run(), run()
    for name, a, b in zip("y S dq dk dv dS".split(), got, again):
        assert bool((a == b).all()), name
    for b in (0, B - 1):
        e = {n: (t if n in ("ld", "scale") or t is None else t[b:b + 1]) for n, t in d.items()}
        ry, rS = ref_fwd(e)
        r = mixer.linattn_bwd(wide(e["dy"]), wide(e["q"]), wide(e["k"]), wide(e["v"]), wide(e["ld"]), e["scale"], wide(e["state"]),
                              wide(e["dstate"]))
        errs = [rel_rows(t[b:b + 1], x) for t, x in zip((got[0],) + got[2:5], (ry,) + r[:3])]
        states = [rel_rows(got[1][b:b + 1], rS), rel_rows(got[5][b:b + 1], r[3])]
        say(f"   row {b}: y dq dk dv " + " ".join(f"{v:.2e}" for v in errs) + " states " + " ".join(f"{v:.2e}" for v in states))
        assert max(errs) <= TOL[dtype] and max(states) <= TOL_F32
