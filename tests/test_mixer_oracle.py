"""The float64 oracles of linear attention, rotary positions and layer norm, pinned by closed forms and
by differences (CPU)."""
import numpy as np

from fft_long_convolution_amd import lconv
from oracle import mixer


def case(seed, B=2, H=4, G=2, N=9, Dk=3, Dv=5):
    r = np.random.default_rng(seed)
    n = r.standard_normal
    return dict(q=n((B, H, N, Dk)), k=n((B, G, N, Dk)), v=n((B, G, N, Dv)), log_decay=-np.exp(n(H)), scale=0.7,
                state=n((B, H, Dk, Dv)), lengths=np.array([N, 4]))


def test_linattn_is_the_masked_matrix_form():
    d = case(1)
    y, S = mixer.linattn(**d)
    for b in range(2):
        n = d["lengths"][b]
        for h in range(4):
            t = np.arange(n)
            gap = t[:, None] - t[None, :]
            w = np.where(gap >= 0, np.exp(d["log_decay"][h] * np.maximum(gap, 0)), 0.0)
            q, k, v = d["q"][b, h, :n], d["k"][b, h // 2, :n], d["v"][b, h // 2, :n]
            first = np.exp(d["log_decay"][h] * (t + 1))[:, None] * (q @ d["state"][b, h])
            np.testing.assert_allclose(y[b, h, :n], 0.7 * ((q @ k.T * w) @ v + first), rtol=1e-11, atol=1e-12)
            tail = np.exp(d["log_decay"][h] * (n - 1 - t))
            np.testing.assert_allclose(S[b, h], np.exp(d["log_decay"][h] * n) * d["state"][b, h] + (k * tail[:, None]).T @ v,
                                       rtol=1e-11, atol=1e-12)
            assert not y[b, h, n:].any()


def test_linattn_without_decay_is_a_running_sum_and_without_memory_the_token_alone():
    d = case(2)
    d.update(state=None, lengths=None, log_decay=np.zeros(4))
    y, S = mixer.linattn(**d)
    kv = np.cumsum(d["k"][:, [0, 0, 1, 1], :, :, None] * d["v"][:, [0, 0, 1, 1], :, None, :], axis=2)
    np.testing.assert_allclose(y, 0.7 * np.einsum("bhnd,bhnde->bhne", d["q"], kv), rtol=1e-11)
    np.testing.assert_allclose(S, kv[:, :, -1], rtol=1e-12)
    d["log_decay"] = np.full(4, -np.inf)
    y, _ = mixer.linattn(**d)
    qk = np.einsum("bhnd,bhnd->bhn", d["q"], d["k"][:, [0, 0, 1, 1]])
    np.testing.assert_allclose(y, 0.7 * qk[..., None] * d["v"][:, [0, 0, 1, 1]], rtol=1e-11)


def test_linattn_gradients_are_differences():
    d = case(3)
    r = np.random.default_rng(4)
    dy, dS = r.standard_normal((2, 4, 9, 5)), r.standard_normal((2, 4, 3, 5))

    def loss(**kw):
        y, S = mixer.linattn(**dict(d, **kw))
        return np.sum(dy * y) + np.sum(dS * S)

    g = mixer.linattn_bwd(dy, dstate=dS, **d)
    for name, grad in zip(("q", "k", "v", "state", "log_decay"), g):
        for _ in range(3):
            e = r.standard_normal(d[name].shape)
            eps = 1e-5
            want = (loss(**{name: d[name] + eps * e}) - loss(**{name: d[name] - eps * e})) / (2 * eps)
            assert abs(np.sum(grad * e) - want) <= 1e-8 * max(1.0, np.sum(np.abs(grad * e)))


def test_a_planted_mistake_in_the_gradient_shows():
    """The decay left out of the state's gradient once moves dk far beyond the GPU tests' tolerances."""
    d = case(5)
    r = np.random.default_rng(6)
    dy = r.standard_normal((2, 4, 9, 5))
    right = mixer.linattn_bwd(dy, **d)[1]
    wrong = mixer.linattn_bwd(dy, **dict(d, log_decay=d["log_decay"] * np.array([1, 1, 1, 0.9])))[1]
    assert np.linalg.norm(right - wrong) / np.linalg.norm(right) > 1e-2


def test_rotary_turns_and_keeps_lengths():
    r = np.random.default_rng(7)
    x = r.standard_normal((2, 3, 4, 10))
    pos = r.integers(0, 100, (2, 4))
    f = np.array([1.0, 0.3, 0.01])
    for inter in (False, True):
        y = mixer.rotary(x, pos, f, inter)
        lo, hi = ((0, 1) if inter else (0, 3))
        a = pos[:, None, :] * f[0]
        np.testing.assert_allclose(y[..., lo], x[..., lo] * np.cos(a) - x[..., hi] * np.sin(a), rtol=1e-12)
        np.testing.assert_allclose(y[..., hi], x[..., hi] * np.cos(a) + x[..., lo] * np.sin(a), rtol=1e-12)
        np.testing.assert_allclose((y ** 2).sum(-1), (x ** 2).sum(-1), rtol=1e-12)
        np.testing.assert_allclose(mixer.rotary(y, pos, f, inter, inverse=True), x, rtol=1e-11, atol=1e-12)
        # scores depend on the distance of the positions alone
        z = r.standard_normal((2, 3, 4, 10))
        s = (mixer.rotary(x, pos, f, inter) * mixer.rotary(z, pos + 5, f, inter)).sum(-1)
        t = (mixer.rotary(x, pos + 40, f, inter) * mixer.rotary(z, pos + 45, f, inter)).sum(-1)
        np.testing.assert_allclose(s, t, rtol=1e-10, atol=1e-10)


def test_rotary_frequencies():
    f = lambda *a, **k: lconv.rotary_frequencies(*a, device="cpu", **k)  # noqa: E731
    plain, m = f(64)
    np.testing.assert_allclose(plain.numpy(), 10000.0 ** (-np.arange(32) / 32), rtol=1e-6)
    assert m == 1.0 and plain.shape == (32,)
    np.testing.assert_allclose(f(64, scaling="linear", factor=4.0)[0].numpy(), plain.numpy() / 4, rtol=1e-6)
    b, _ = f(64, scaling="base", factor=4.0)
    assert b[0] == plain[0]
    np.testing.assert_allclose(float(b[-1]), float(plain[-1]) / 4, rtol=1e-5)
    p, m = f(64, scaling="by_parts", factor=4.0, original=4096)
    ratio = (plain / p).numpy()
    assert np.all(np.diff(ratio) >= -1e-6) and abs(ratio[0] - 1) < 1e-6 and abs(ratio[-1] - 4) < 1e-5
    turns = 4096 * plain.numpy() / (2 * np.pi)
    assert np.all(np.abs(ratio[turns > 40] - 1) < 1e-6) and np.all(np.abs(ratio[turns < 0.8] - 4) < 1e-5)
    assert abs(m - (1 + 0.1 * np.log(4.0))) < 1e-12


def test_layer_norm_and_its_gradient_by_differences():
    r = np.random.default_rng(8)
    x, dy, w, b = r.standard_normal((4, 7)), r.standard_normal((4, 7)), r.standard_normal(7), r.standard_normal(7)
    y, mean, rstd = mixer.layer_norm(x, np.ones(7), np.zeros(7), 0.0)
    np.testing.assert_allclose(y.mean(-1), 0, atol=1e-12)
    np.testing.assert_allclose(y.var(-1), 1, rtol=1e-12)
    _, mean, rstd = mixer.layer_norm(x, w, b, 1e-3)
    g = mixer.layer_norm_bwd(dy, x, w, mean, rstd)
    loss = lambda x, w, b: np.sum(dy * mixer.layer_norm(x, w, b, 1e-3)[0])  # noqa: E731
    for i, grad in enumerate(g):
        e = r.standard_normal((x, w, b)[i].shape)
        at = [[a + s * 1e-6 * e if j == i else a for j, a in enumerate((x, w, b))] for s in (1, -1)]
        want = (loss(*at[0]) - loss(*at[1])) / 2e-6
        assert abs(np.sum(grad * e) - want) <= 1e-7 * np.sum(np.abs(grad * e))
