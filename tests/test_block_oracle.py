"""The float64 oracles of the recurrent block's operators against closed forms, brute force and differences (CPU)."""
import numpy as np
import pytest

from oracle import block

# central differences with steps of 1e-6 on values of order one: truncation 1e-12, cancellation 1e-10
DIFF = 1e-7


def slope_along(f, args, name, rng):
    """(d/de f(args + e v), v) by central differences along a random direction of one argument."""
    v = rng.standard_normal(args[name].shape)
    at = lambda e: f(**{**args, name: args[name] + e * v})  # noqa: E731
    return (at(1e-6) - at(-1e-6)) / 2e-6, v


def test_scan_closed_forms():
    x = np.ones((1, 5, 1))
    y, h = block.gated_scan(x, np.full((1, 5, 1), np.log(0.5)), "log", "plain")
    assert np.allclose(y[0, :, 0], [1, 1.5, 1.75, 1.875, 1.9375], rtol=1e-15) and h[0, 0] == y[0, 4, 0]
    y, _ = block.gated_scan(x, np.zeros((1, 5, 1)), "sigmoid", "convex")        # towards one, half of the way each time
    assert np.allclose(y[0, :, 0], 1 - 0.5 ** np.arange(1, 6), rtol=1e-15)
    y, _ = block.gated_scan(x, np.full((1, 5, 1), -np.inf), "log", "norm", input_gate=np.zeros((1, 5, 1)))
    assert np.allclose(y, 0.5)                                                  # no memory
    y, h = block.gated_scan(x, np.zeros((1, 5, 1)), "rate", "plain", rate=np.array([np.log(4.0)]), state=np.array([[8.0]]),
                            lengths=[2])
    assert np.allclose(y[0, :, 0], [5, 3.5, 0, 0, 0]) and np.allclose(h, 3.5)


@pytest.mark.parametrize("gate", ["log", "sigmoid", "rate"])
@pytest.mark.parametrize("mix", ["plain", "convex", "norm"])
def test_scan_gradients_against_differences(gate, mix):
    rng = np.random.default_rng(5)
    B, N, C = 3, 7, 4
    z = rng.standard_normal((B, N, C))
    a = dict(x=rng.standard_normal((B, N, C)), z=-np.exp(z) if gate == "log" else z, input_gate=rng.standard_normal((B, N, C)),
             state=rng.standard_normal((B, C)))
    if gate == "rate":
        a["rate"] = rng.random(C) + 0.1
    n, dy, ds = [7, 0, 3], rng.standard_normal((B, N, C)), rng.standard_normal((B, C))

    def loss(**k):
        y, h = block.gated_scan(gate=gate, mix=mix, lengths=n, **k)
        return (y * dy).sum() + (h * ds).sum()

    g = block.gated_scan_bwd(dy, gate=gate, mix=mix, dstate=ds, lengths=n, **a)
    for name, grad in zip(("x", "z", "input_gate", "rate", "state"), g):
        if grad is None:
            continue
        want, v = slope_along(loss, a, name, rng)
        assert abs(want - (grad * v).sum()) <= DIFF * np.abs(grad * v).sum(), name
    # magnitudes bound the values
    size = block.gated_scan_bwd(np.abs(dy), np.abs(a["x"]), a["z"], gate, mix, a["input_gate"], a.get("rate"), np.abs(a["state"]),
                                np.abs(ds), n, size=True)
    for v, w in zip(g, size):
        assert v is None or np.all(np.abs(v) <= w * (1 + 1e-12))


@pytest.mark.parametrize("centred", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot", [0, 6, 8])
def test_qk_norm_rotary(centred, interleaved, rot):
    rng = np.random.default_rng(6)
    B, H, N, D = 2, 3, 4, 8
    a = dict(x=rng.standard_normal((B, H, N, D)), weight=1 + 0.1 * rng.standard_normal(D))
    pos, f = rng.integers(0, 50, (B, N)).astype(float), 10.0 ** -np.arange(rot // 2)
    how = dict(positions=pos, inv_freq=f, eps=1e-3, centred=centred, interleaved=interleaved, magnitude=1.5)
    y = block.qk_norm_rotary(**a, **how)
    # by hand, one row
    x = a["x"][1, 2, 3] - (a["x"][1, 2, 3].mean() if centred else 0.0)
    v = x / np.sqrt((x ** 2).sum() / D + 1e-3) * a["weight"]
    for p in range(rot // 2):
        i, j = (2 * p, 2 * p + 1) if interleaved else (p, p + rot // 2)
        c, s = 1.5 * np.cos(pos[1, 3] * f[p]), 1.5 * np.sin(pos[1, 3] * f[p])
        v[i], v[j] = v[i] * c - v[j] * s, v[j] * c + v[i] * s
    assert np.allclose(v, y[1, 2, 3], rtol=1e-12, atol=1e-12)
    dy = rng.standard_normal(y.shape)
    g = block.qk_norm_rotary_bwd(dy, **a, **how)
    for name, grad in zip(("x", "weight"), g):
        want, d = slope_along(lambda **k: (block.qk_norm_rotary(**k, **how) * dy).sum(), a, name, rng)
        assert abs(want - (grad * d).sum()) <= DIFF * np.abs(grad * d).sum()


@pytest.mark.parametrize("K", [1, 2, 5])
@pytest.mark.parametrize("silu", [False, True])
def test_short_conv(K, silu):
    rng = np.random.default_rng(7)
    B, N, C = 3, 6, 2
    a = dict(x=rng.standard_normal((B, N, C)), weight=rng.standard_normal((C, K)), bias=rng.standard_normal(C),
             state=rng.standard_normal((B, K - 1, C)))
    n = [6, 0, 2]
    y, last = block.short_conv(silu=silu, lengths=n, **a)
    for b in range(B):                      # by hand
        seen = [a["state"][b, j] for j in range(K - 1)]
        for t in range(n[b]):
            seen.append(a["x"][b, t])
            p = a["bias"] + sum(a["weight"][:, j] * seen[len(seen) - K + j] for j in range(K))
            assert np.allclose(y[b, t], p / (1 + np.exp(-p)) if silu else p)
        assert np.all(y[b, n[b]:] == 0) and np.all(last[b] == np.array(seen[len(seen) - (K - 1):]).reshape(K - 1, C))
    dy, ds = rng.standard_normal(y.shape), rng.standard_normal(last.shape)

    def loss(**k):
        p, q = block.short_conv(silu=silu, lengths=n, **k)
        return (p * dy).sum() + (q * ds).sum()

    g = block.short_conv_bwd(dy, dstate=ds, silu=silu, lengths=n, **a)
    for name, grad in zip(("x", "weight", "bias", "state"), g):
        want, d = slope_along(loss, a, name, rng)
        assert abs(want - (grad * d).sum()) <= DIFF * max(np.abs(grad * d).sum(), 1e-3)
