"""float64 oracles of linear attention, rotary positions and layer norm (numpy, from the definitions).

TEST INFRASTRUCTURE ONLY.  Arrays are float64 (already rounded to the storage type by the caller).
"""
from __future__ import annotations

import numpy as np


def linattn(q, k, v, log_decay, scale, state=None, lengths=None):
    """(y, state): the recurrence S = gamma S + k v^T, y = scale S^T q, token by token."""
    B, H, N, Dk = q.shape
    G, Dv = k.shape[1], v.shape[-1]
    y = np.zeros((B, H, N, Dv))
    S = np.zeros((B, H, Dk, Dv)) if state is None else state.copy()
    for b in range(B):
        n = N if lengths is None else min(max(int(lengths[b]), 0), N)
        for h in range(H):
            g, gamma = h // (H // G), np.exp(log_decay[h])
            for t in range(n):
                S[b, h] = gamma * S[b, h] + np.outer(k[b, g, t], v[b, g, t])
                y[b, h, t] = scale * (q[b, h, t] @ S[b, h])
    return y, S


def linattn_bwd(dy, q, k, v, log_decay, scale, state=None, dstate=None, lengths=None):
    """(dq, dk, dv, dstate_in, dlog_decay) by the recurrences of the states and their gradients."""
    B, H, N, Dk = q.shape
    G, Dv = k.shape[1], v.shape[-1]
    dq, dk, dv = np.zeros(q.shape), np.zeros(k.shape), np.zeros(v.shape)
    ds, dl = np.zeros((B, H, Dk, Dv)), np.zeros(H)
    for b in range(B):
        n = N if lengths is None else min(max(int(lengths[b]), 0), N)
        for h in range(H):
            g, gamma = h // (H // G), np.exp(log_decay[h])
            S = [np.zeros((Dk, Dv)) if state is None else state[b, h]]
            for t in range(n):
                S.append(gamma * S[-1] + np.outer(k[b, g, t], v[b, g, t]))
                dq[b, h, t] = scale * (S[-1] @ dy[b, h, t])
            D = np.zeros((Dk, Dv)) if dstate is None else dstate[b, h].copy()
            for t in range(n - 1, -1, -1):
                D += scale * np.outer(q[b, h, t], dy[b, h, t])      # dL/dS_t
                dk[b, g, t] += D @ v[b, g, t]
                dv[b, g, t] += D.T @ k[b, g, t]
                dl[h] += gamma * np.sum(D * S[t])
                D = gamma * D
            ds[b, h] = D
    return dq, dk, dv, ds, dl


def rotary(x, positions, inv_freq, interleaved=False, inverse=False, magnitude=1.0):
    """x [B, H, N, D], positions [B, N]: every pair turned as a complex number."""
    rot = 2 * len(inv_freq)
    a = positions[:, None, :, None] * inv_freq
    turn = magnitude * np.exp((-1j if inverse else 1j) * a)
    y = x.copy()
    lo, hi = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    z = (x[..., lo] + 1j * x[..., hi]) * turn
    y[..., lo], y[..., hi] = z.real, z.imag
    return y


def layer_norm(x, weight, bias, eps):
    mean = x.mean(-1)
    rstd = 1.0 / np.sqrt(((x - mean[..., None]) ** 2).mean(-1) + eps)
    return (x - mean[..., None]) * rstd[..., None] * weight + bias, mean, rstd


def layer_norm_bwd(dy, x, weight, mean, rstd):
    xhat = (x - mean[..., None]) * rstd[..., None]
    h = dy * weight
    dx = rstd[..., None] * (h - h.mean(-1, keepdims=True) - xhat * (h * xhat).mean(-1, keepdims=True))
    rows = tuple(range(x.ndim - 1))
    return dx, (dy * xhat).sum(rows), dy.sum(rows)
