"""The gradient of linear attention's decay against the size of its own terms.

With T_t = gamma (T_{t-1} + S_{t-1}) it is the sum over tokens, rows and columns of scale q_d T_t[d, n] dy_n, and of T_L dstate: terms
of either sign, whose roundings add like a random walk, so an error is measured against the root of the sum of their squares.
bf16 data: S, T and the weighted v are multiplied in two bf16 parts, 2^-17 of each operand; four such factors allowed, 2^-15.
One rounding to bf16 instead (2^-9 at most, 2^-10.3 in the root mean square) is far outside.  fp16 and fp32 data: fp32 products,
64 half-units as for the other fp32 results."""
import numpy as np
import pytest

from oracle import mixer
from tests.mixer_util import TOL_F32, host, say, wide

TOL = {"bf16": 2.0 ** -15, "f16": TOL_F32, "f32": TOL_F32}


def tangent(q, k, v, dy, ld, scale, state, dstate, lengths, keep=lambda x: x):
    """(dlog_decay, root of the sum of its terms' squares) per head; keep: what T goes through as an operand."""
    B, H, N, Dk = q.shape
    G = k.shape[1]
    total, squares = np.zeros(H), np.zeros(H)
    for b in range(B):
        for h in range(H):
            g, gamma = h // (H // G), np.exp(ld[h])
            S, T = state[b, h].copy(), np.zeros(state.shape[2:])
            for t in range(min(max(int(lengths[b]), 0), N) if lengths is not None else N):
                T = gamma * (T + S)
                S = gamma * S + np.outer(k[b, g, t], v[b, g, t])
                total[h] += scale * (q[b, h, t] @ keep(T) @ dy[b, h, t])
                squares[h] += scale ** 2 * (q[b, h, t] ** 2 @ T ** 2 @ dy[b, h, t] ** 2)
            total[h] += np.sum(T * dstate[b, h])
            squares[h] += np.sum((T * dstate[b, h]) ** 2)
    return total, np.sqrt(squares)


def inputs(seed, B, H, G, N, Dk, Dv, dtype):
    import torch
    rng = np.random.default_rng(seed)
    d = {n: host(rng, (B, h, N, D), dtype) for n, h, D in (("q", H, Dk), ("k", G, Dk), ("v", G, Dv), ("dy", H, Dv))}
    d["ld"] = torch.tensor(-2.0 ** -np.linspace(1, 10, H) if H > 1 else [-0.02], dtype=torch.float32)
    d["state"], d["dstate"] = host(rng, (B, H, Dk, Dv), "f32"), host(rng, (B, H, Dk, Dv), "f32")
    return d


def reference(d, lengths, keep=lambda x: x):
    Dk = d["q"].shape[-1]
    return tangent(wide(d["q"]), wide(d["k"]), wide(d["v"]), wide(d["dy"]), wide(d["ld"]), Dk ** -0.5, wide(d["state"]), wide(d["dstate"]),
                   lengths, keep)


def test_the_tangent_is_the_oracle_and_one_rounding_shows():
    d = inputs(1, 2, 4, 2, 60, 24, 32, "bf16")
    want, size = reference(d, [60, 31])
    args = [wide(d[n]) for n in ("dy", "q", "k", "v", "ld")]
    dl = mixer.linattn_bwd(*args, 24 ** -0.5, wide(d["state"]), wide(d["dstate"]), np.array([60, 31]))[4]
    np.testing.assert_allclose(want, dl, rtol=1e-9)

    def bf16(x):                                               # one rounding of an operand, planted
        import torch
        return torch.from_numpy(x).to(torch.bfloat16).double().numpy()

    off = np.abs(reference(d, [60, 31], bf16)[0] - want) / size
    assert np.linalg.norm(off) > 4 * TOL["bf16"], off


CASES = [(1, 1, 1, 1, 8, 8, None), (2, 4, 2, 33, 64, 40, None), (1, 3, 3, 300, 128, 128, None), (2, 4, 1, 257, 96, 72, (257, 100)),
         (1, 2, 2, 200, 256, 136, None), (3, 2, 2, 150, 24, 200, (0, 1, 150)), (1, 2, 1, 1100, 64, 64, None)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c[:6])))
def test_dlog_decay(dtype, case):
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from fft_long_convolution_amd import lconv
    B, H, G, N, Dk, Dv, lengths = case
    say(f"[linattn dlog] {dtype} {case}")
    d = inputs(40 + N, B, H, G, N, Dk, Dv, dtype)
    c = {n: t.cuda() for n, t in d.items()}
    ln = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
    got = wide(lconv.linear_attention_bwd(c["dy"], c["q"], c["k"], c["v"], c["ld"], state=c["state"], dstate=c["dstate"], lengths=ln,
                                          need_dlog_decay=True).dlog_decay)
    want, size = reference(d, lengths)
    off = np.abs(got - want) / size
    say("   " + " ".join(f"{x:.1e}" for x in off) + f" (tol {TOL[dtype]:.1e})")
    assert off.max() <= TOL[dtype]
