"""float64 oracles of the gated linear recurrence, q/k norms with rotary positions, and the short convolution (numpy, from the
definitions).

TEST INFRASTRUCTURE ONLY.  Arrays are float64 (already rounded to the storage type by the caller).
"""
from __future__ import annotations

import numpy as np

from oracle import mixer


def _sigmoid(x):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-x))


def _row_lengths(lengths, B, N):
    return [N if lengths is None else min(max(int(lengths[b]), 0), N) for b in range(B)]


def decay(z, gate, rate=None):
    """(a, 1 - a, log a)."""
    with np.errstate(over="ignore"):
        la = z if gate == "log" else -np.logaddexp(0.0, -z) if gate == "sigmoid" else -rate * _sigmoid(z)
    return np.exp(la), -np.expm1(la), la


def mix_of(la, mix):
    """(m, dm / dlog a)."""
    if mix == "plain":
        return np.ones_like(la), np.zeros_like(la)
    if mix == "convex":
        return -np.expm1(la), -np.exp(la)
    m = np.sqrt(-np.expm1(2.0 * la))
    with np.errstate(divide="ignore", invalid="ignore"):
        return m, np.where(m > 0, -np.exp(2.0 * la) / m, 0.0)


def gated_scan(x, z, gate, mix, input_gate=None, rate=None, state=None, lengths=None):
    """(y, state): h = a h + m s x, token by token."""
    B, N, C = x.shape
    n = np.array(_row_lengths(lengths, B, N))[:, None]
    h = np.zeros((B, C)) if state is None else state.copy()
    y = np.zeros(x.shape)
    s = 1.0 if input_gate is None else _sigmoid(input_gate)
    u = s * x
    for t in range(N):
        a, _, la = decay(z[:, t], gate, rate)
        new = a * h + mix_of(la, mix)[0] * u[:, t]
        h = np.where(t < n, new, h)
        y[:, t] = np.where(t < n, new, 0.0)
    return y, h


def gated_scan_bwd(dy, x, z, gate, mix, input_gate=None, rate=None, state=None, dstate=None, lengths=None, size=False):
    """(dx, dz, dinput_gate, drate, dstate_in) by the chain rule.  size: every term by its magnitude instead (inputs given by
    theirs), what roundings are measured against."""
    B, N, C = x.shape
    n = np.array(_row_lengths(lengths, B, N))[:, None]
    s = np.ones(x.shape) if input_gate is None else _sigmoid(input_gate)
    sign = 1.0 if size else -1.0
    before, h = [], np.zeros((B, C)) if state is None else state.copy()
    for t in range(N):
        a, _, la = decay(z[:, t], gate, rate)
        before.append(h)
        h = np.where(t < n, a * h + mix_of(la, mix)[0] * s[:, t] * x[:, t], h)
    G = np.zeros((B, C)) if dstate is None else dstate.copy()
    dx, dz, di, drate = np.zeros(x.shape), np.zeros(x.shape), np.zeros(x.shape), np.zeros(C)
    for t in range(N - 1, -1, -1):
        a, d, la = decay(z[:, t], gate, rate)
        m, dm = mix_of(la, mix)
        on = t < n
        now = G + dy[:, t]
        dx[:, t] = np.where(on, now * m * s[:, t], 0.0)
        di[:, t] = np.where(on, now * m * x[:, t] * s[:, t] * (1.0 - s[:, t]), 0.0)
        dl = a * now * before[t] - sign * now * s[:, t] * x[:, t] * dm if size else \
            a * now * before[t] + now * s[:, t] * x[:, t] * dm
        if gate == "sigmoid":
            dl = dl * d
        elif gate == "rate":
            p = _sigmoid(z[:, t])
            drate += np.where(on, sign * dl * p, 0.0).sum(0)
            dl = sign * dl * rate * p * _sigmoid(-z[:, t])
        dz[:, t] = np.where(on, dl, 0.0)
        G = np.where(on, a * now, G)
    return dx, dz, (None if input_gate is None else di), (drate if gate == "rate" else None), G


def _centre(x, centred):
    return x - x.mean(-1, keepdims=True) if centred else x


def qk_norm_rotary(x, weight, positions, inv_freq, eps, centred=False, interleaved=False, magnitude=1.0):
    """x [B, H, N, D]: each head's row over its root mean square (of the centred row), times the weight, turned."""
    u = _centre(x, centred)
    y = u / np.sqrt((u * u).mean(-1, keepdims=True) + eps) * weight
    return mixer.rotary(y, positions, inv_freq, interleaved, False, magnitude) if len(inv_freq) else y


def qk_norm_rotary_bwd(dy, x, weight, positions, inv_freq, eps, centred=False, interleaved=False, magnitude=1.0):
    """(dx, dweight)."""
    if len(inv_freq):
        dy = mixer.rotary(dy, positions, inv_freq, interleaved, True, magnitude)
    u = _centre(x, centred)
    r = 1.0 / np.sqrt((u * u).mean(-1, keepdims=True) + eps)
    h = dy * weight
    dx = r * (h - u * r * r * (h * u).mean(-1, keepdims=True))
    return _centre(dx, centred), (dy * u * r).sum((0, 1, 2))


def short_conv(x, weight, bias=None, silu=False, state=None, lengths=None):
    """(y, state): p_t = bias + sum_j weight[:, j] x_{t-K+1+j} over the row's own tokens and the K - 1 before them."""
    B, N, C = x.shape
    K = weight.shape[1]
    y, last = np.zeros(x.shape), np.zeros((B, K - 1, C))
    for b, n in enumerate(_row_lengths(lengths, B, N)):
        row = np.concatenate((np.zeros((K - 1, C)) if state is None else state[b], x[b, :n]))
        p = np.zeros((n, C)) + (0.0 if bias is None else bias)
        for j in range(K):
            p += weight[:, j] * row[j:j + n]
        y[b, :n] = p * _sigmoid(p) if silu else p
        last[b] = row[n:]
    return y, last


def short_conv_bwd(dy, x, weight, bias=None, silu=False, state=None, dstate=None, lengths=None):
    """(dx, dweight, dbias, dstate_in)."""
    B, N, C = x.shape
    K = weight.shape[1]
    dx, dw, db, ds = np.zeros(x.shape), np.zeros(weight.shape), np.zeros(C), np.zeros((B, K - 1, C))
    for b, n in enumerate(_row_lengths(lengths, B, N)):
        row = np.concatenate((np.zeros((K - 1, C)) if state is None else state[b], x[b, :n]))
        p = np.zeros((n, C)) + (0.0 if bias is None else bias)
        for j in range(K):
            p += weight[:, j] * row[j:j + n]
        s = _sigmoid(p)
        dp = dy[b, :n] * (s + p * s * (1.0 - s) if silu else 1.0)
        g = np.zeros((n + K - 1, C))
        if dstate is not None:
            g[n:] += dstate[b]
        for j in range(K):
            g[j:j + n] += weight[:, j] * dp
            dw[:, j] += (dp * row[j:j + n]).sum(0)
        db += dp.sum(0)
        dx[b, :n], ds[b] = g[K - 1:], g[:K - 1]
    return dx, dw, db, ds
