"""Linear attention and its gradients in float64 numpy by chunks of 64 tokens, for rows too long or too many for the token by
token oracle (pinned against it in test_linattn_cover.py)."""
import numpy as np

CHUNK = 64


def _row(Q, K, V, lg, S, last_decays):
    """One head: O_t = S_t^T Q_t with S_t = gamma S_{t-1} + K_t V_t^T; with last_decays false the state that enters is not
    decayed ahead of the first token but behind it (the gradients' direction).  Returns (O, the state that leaves)."""
    n, r = len(Q), 0 if last_decays else 1
    O = np.zeros((n, V.shape[1]))  # noqa: E741
    for a in range(0, n, CHUNK):
        q, k, v = Q[a:a + CHUNK], K[a:a + CHUNK], V[a:a + CHUNK]
        t = np.arange(len(q))
        gap = t[:, None] - t[None, :]
        w = np.where(gap >= 0, np.exp(lg * np.maximum(gap, 0)), 0.0)
        O[a:a + CHUNK] = (q @ k.T * w) @ v + np.exp(lg * (t + 1 - r))[:, None] * (q @ S)
        S = np.exp(lg * len(q)) * S + (k * np.exp(lg * (len(q) - 1 - t + r))[:, None]).T @ v
    return O, S


def linattn_all(d, scale):
    """(y, S, dq, dk, dv, dstate) of numpy inputs q, k, v, dy, ld, state, dstate, lengths (or None)."""
    q, k, v, dy, ld = (d[n] for n in ("q", "k", "v", "dy", "ld"))
    B, H, N, Dk = q.shape
    G, Dv = k.shape[1], v.shape[-1]
    y, dq, dk, dv = np.zeros(dy.shape), np.zeros(q.shape), np.zeros(k.shape), np.zeros(v.shape)
    S, dS = np.zeros((B, H, Dk, Dv)), np.zeros((B, H, Dk, Dv))
    for b in range(B):
        n = N if d["lengths"] is None else min(max(int(d["lengths"][b]), 0), N)
        for h in range(H):
            g, lg = h // (H // G), ld[h]
            S0 = np.zeros((Dk, Dv)) if d["state"] is None else d["state"][b, h]
            G0 = np.zeros((Dk, Dv)) if d["dstate"] is None else d["dstate"][b, h]
            Q, K, V, Y = q[b, h, :n], k[b, g, :n], v[b, g, :n], dy[b, h, :n]
            o, S[b, h] = _row(Q, K, V, lg, S0, True)
            y[b, h, :n] = scale * o
            dq[b, h, :n] = scale * _row(Y, V, K, lg, S0.T, True)[0]
            back = slice(None, None, -1)
            dk[b, g, :n] += _row(V[back], scale * Y[back], Q[back], lg, G0.T, False)[0][back]
            o, dS[b, h] = _row(K[back], scale * Q[back], Y[back], lg, G0, False)
            dv[b, g, :n] += o[back]
    return y, S, dq, dk, dv, dS
