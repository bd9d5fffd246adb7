"""How far a value that is not finite goes in the gradients of the gated recurrence, operand by operand: x and the input gate through
the states to later tokens, dy and dstate through their gradients to earlier ones, z to both; never to another channel or row."""
import numpy as np
import pytest

from tests.mixer_util import host, say
from tests.test_gated_scan_forms_gpu import MORE
from tests.test_gated_scan_gpu import HOW, cuda, inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lc():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from fft_long_convolution_amd import lconv
    lconv.load()
    return lconv


def reached(what, t, N, mix):
    """The tokens of dx, dz, dinput_gate and whether drate and dstate, of the channel that has it at token t."""
    upto, since, own = np.arange(N) <= t, np.arange(N) >= t, np.arange(N) == t
    none, later = np.zeros(N, bool), np.arange(N) > t
    plain = mix == "plain"                       # m = 1 whatever a is
    return {"x": (none, later if plain else since, own, True, False),
            "input_gate": (own, later if plain else since, own, True, False),
            "z": (upto & ~own if plain else upto, np.ones(N, bool), upto & ~own if plain else upto, True, True),
            "dy": (upto, upto, upto, True, True)}[what]


@pytest.mark.parametrize("how", HOW + MORE, ids=lambda h: "-".join(map(str, h)))
def test_reach(lc, how):
    import torch
    gate, mix, gated = how
    rng = np.random.default_rng(1500)
    for B, N, C in ((2, 150, 6), (1, 700, 70)):              # whole rows, segments
        say(f"[scan not finite] {how} {(B, N, C)}")
        x, z, i, rate = inputs(rng, B, N, C, "bf16", gate, gated)
        clean = dict(x=x, z=z, input_gate=i, dy=host(rng, (B, N, C), "bf16"))
        clean = {k: None if v is None else v.cuda() for k, v in clean.items()}
        gr, = cuda(rate)
        ds = host(rng, (B, C), "f32").cuda()

        def run(o):
            f = lc.gated_scan(o["x"], o["z"], gate, mix, o["input_gate"], gr, need_marks=True)
            return f, lc.gated_scan_bwd(o["dy"], o["x"], o["z"], f.marks, gate, mix, o["input_gate"], gr, dstate=ds)

        _, want = run(clean)
        for what in ("x", "z", "input_gate", "dy"):
            if clean[what] is None:
                continue
            for bad in (float("nan"),) if what in ("z", "input_gate") else (float("nan"), float("inf")):
                b, t, c = B - 1, int(rng.integers(0, N)), int(rng.integers(0, C))
                say(f"   {bad} in {what}{[b, t, c]}")
                o = {k: None if v is None else v.clone() for k, v in clean.items()}
                o[what][b, t, c] = bad
                f, got = run(o)
                if what != "dy":
                    hit = np.zeros((B, N, C), bool)
                    hit[b, t:, c] = True
                    assert np.array_equal(~f.y.isfinite().cpu().numpy(), hit)
                dx, dz, di, drate, dstate = reached(what, t, N, mix)
                for name, g, w, tokens in (("dx", got.dx, want.dx, dx), ("dz", got.dz, want.dz, dz), ("di", got.dinput_gate, want.dinput_gate, di)):
                    if g is None:
                        continue
                    hit = np.zeros((B, N, C), bool)
                    hit[b, :, c] = tokens
                    assert np.array_equal(~g.isfinite().cpu().numpy(), hit), name
                    rest = torch.ones((B, N, C), dtype=torch.bool, device="cuda")
                    rest[b, :, c] = False
                    assert bool((g[rest] == w[rest]).all()), name
                for name, g, w, there, at in (("drate", got.drate, want.drate, drate, (c,)), ("dstate", got.dstate, want.dstate, dstate, (b, c))):
                    if g is None:
                        continue
                    hit = torch.zeros(g.shape, dtype=torch.bool, device="cuda")
                    hit[at] = there
                    assert bool((~g.isfinite() == hit).all()), name
                    hit[at] = True
                    assert bool((g[~hit] == w[~hit]).all()), name
