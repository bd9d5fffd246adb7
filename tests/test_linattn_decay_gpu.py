"""A state that is carried over tokens which add nothing to it (k, v, q and dy zero: masked by multiplication), for decays
from fast to none, whole rows and rows in segments: states and their gradients keep fp32's accuracy relative to what is
left of them, head by head."""
import numpy as np
import pytest

from oracle import mixer
from tests.mixer_util import TOL_F32, host, rel_rows, say, wide

pytestmark = pytest.mark.gpu

# decays of a token: the state's factor over a chunk of 32 from 1 to 1e-14
DECAYS = [0.0, -1e-7, -1e-4, -0.01, -0.05, -0.1, -0.2, -0.3, -0.4, -0.5, -0.7, -1.0]


@pytest.fixture(scope="module")
def lc():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from fft_long_convolution_amd import lconv
    lconv.load()
    return lconv


def quiet(seed, B, H, N, Dk, Dv, dtype, loud):
    """Inputs that are zero but for the tokens of `loud`."""
    import torch
    rng = np.random.default_rng(seed)
    keep = torch.zeros(N, 1)
    keep[loud] = 1.0
    d = {n: (host(rng, (B, H, N, D), dtype) * keep.to(host(rng, (1,), dtype).dtype)).cuda()
         for n, D in (("q", Dk), ("k", Dk), ("v", Dv), ("dy", Dv))}
    d["ld"] = torch.tensor(DECAYS[:H] if H == len(DECAYS) else DECAYS[-H:], device="cuda")
    d["state"], d["dstate"] = host(rng, (B, H, Dk, Dv), "f32").cuda(), host(rng, (B, H, Dk, Dv), "f32").cuda()
    return d


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("B,N,Dk,Dv,loud", [
    (2, 32, 64, 64, []), (2, 70, 64, 64, []), (1, 70, 128, 128, [0, 1, 2]), (2, 64, 96, 72, [63]), (1, 67, 256, 200, [1]),
    (12, 70, 128, 128, [0])])
def test_silent_tokens_keep_the_state(lc, dtype, B, N, Dk, Dv, loud):
    say(f"[linattn silent] {dtype} {B, N, Dk, Dv, loud}")
    d = quiet(600 + N, B, len(DECAYS), N, Dk, Dv, dtype, loud)
    check(lc, d, N)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("N,H,Dk,Dv,loud", [(700, 12, 64, 64, [0, 300]), (1500, 8, 128, 128, [1490])])
def test_silent_tokens_over_segments(lc, dtype, N, H, Dk, Dv, loud):
    """Rows long enough to be split; the fastest decays would leave nothing that fp32 holds."""
    import torch
    say(f"[linattn silent segments] {dtype} {N, H, Dk, Dv, loud}")
    d = quiet(610 + N, 1, H, N, Dk, Dv, dtype, loud)
    d["ld"] = torch.tensor(np.float32(-np.logspace(-5, np.log10(60.0 / N), H)), device="cuda")
    check(lc, d, N)


def check(lc, d, N):
    _, S = lc.linear_attention(d["q"], d["k"], d["v"], d["ld"], scale=1.0, state=d["state"])
    args = [wide(d[n]) for n in ("q", "k", "v", "ld")]
    _, rS = mixer.linattn(*args, 1.0, wide(d["state"]))
    g = lc.linear_attention_bwd(d["dy"], d["q"], d["k"], d["v"], d["ld"], scale=1.0, state=d["state"], dstate=d["dstate"],
                                need_dlog_decay=True)
    r = mixer.linattn_bwd(wide(d["dy"]), *args, 1.0, wide(d["state"]), wide(d["dstate"]))
    eS, eD = rel_rows(S, rS), rel_rows(g.dstate, r[3])
    say(f"   state {eS:.2e}  dstate {eD:.2e} (tol {TOL_F32:.1e})")
    assert eS <= TOL_F32 and eD <= TOL_F32
    if not d["k"].any():
        # no token at all: dlog_decay = N gamma^N <state, dstate>, against the root of the sum of its terms' squares
        terms = N * np.exp(N * wide(d["ld"]))[:, None] * np.moveaxis(wide(d["state"]) * wide(d["dstate"]), 0, 1).reshape(len(d["ld"]), -1)
        off = np.abs(wide(g.dlog_decay) - terms.sum(1)) / np.sqrt((terms ** 2).sum(1))
        say(f"   dlog_decay {off.max():.2e}")
        assert off.max() <= TOL_F32


def test_thousands_of_single_tokens_keep_slow_decays(lc):
    """The token form's factor is used once a token: rounded to fp32 it would drift by half a unit each, over a memory of
    ten thousand tokens far beyond fp32's accuracy."""
    import torch
    say("[linattn token drift]")
    rng = np.random.default_rng(620)
    H, N, Dk, Dv = 12, 3000, 32, 32
    q, k, v = (host(rng, (1, H, N, D), "f32").cuda() for D in (Dk, Dk, Dv))
    ld = torch.tensor(np.float32(-np.logspace(-5, -1.5, H)), device="cuda")
    S = host(rng, (1, H, Dk, Dv), "f32", 50.0).cuda()          # the size that the sums grow to
    _, ref = mixer.linattn(wide(q), wide(k), wide(v), wide(ld), 1.0, wide(S))
    for t in range(N):
        lc.linear_attention_step(q[:, :, t], k[:, :, t], v[:, :, t], ld, S, scale=1.0)
    e = [rel_rows(S[:, h:h + 1], ref[:, h:h + 1]) for h in range(H)]
    say("   " + " ".join(f"{x:.1e}" for x in e))
    assert max(e) <= TOL_F32
