"""Layer norm on views with evenly spaced rows: which layouts the wrapper takes (CPU), and that they give the dense copy's
results (GPU)."""
import pytest

torch = pytest.importorskip("torch")

from fft_long_convolution_amd import lconv  # noqa: E402
from tests.mixer_util import host, say  # noqa: E402


def views(t):
    """(name, view, row stride) of t [4, 6, 40]."""
    return [("dense", t, 40), ("last dimension", t[..., :32], 40), ("one token of every sequence", t[:, 2:3], 240), ("one token", t[:, 2], 240),
            ("one row", t[1:2, 3:4, 8:24], 16), ("every second sequence's one token", t[::2, 5:6], 480), ("tokens of one sequence", t[2:3, 1:5, :32], 40),
            ("nothing", t[:0, :, :8], 8)]


def test_rows_of_views():
    t = torch.zeros(4, 6, 40)
    for name, v, step in views(t):
        rows, C, got = lconv._rows("x", v, v.shape, v.dtype)
        assert (rows, C) == (v[..., 0].numel(), v.shape[-1]), name
        assert rows <= 1 or got == step, name
    for v in (t[:, :5], t[:, ::2][:, :, :32][:3, :2].transpose(0, 1), t.transpose(1, 2), t[..., ::2], t[:, :1].expand(4, 6, 40)):
        with pytest.raises(ValueError, match="evenly spaced"):
            lconv._rows("x", v, v.shape, v.dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_views_give_the_dense_copys_results(dtype):
    import numpy as np
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    say(f"[norm layouts] {dtype}")
    rng = np.random.default_rng(570)
    t, g = host(rng, (4, 6, 40), dtype).cuda(), host(rng, (4, 6, 40), dtype).cuda()
    for (name, x, _), (_, dy, _) in zip(views(t), views(g)):
        w, b = host(rng, (x.shape[-1],), dtype).cuda(), host(rng, (x.shape[-1],), dtype).cuda()
        y, mean, rstd = lconv.layer_norm(x, w, b)
        y2, mean2, rstd2 = lconv.layer_norm(x.contiguous(), w, b)
        got = (y, mean, rstd) + lconv.layer_norm_bwd(dy, x, w, mean, rstd)
        want = (y2, mean2, rstd2) + lconv.layer_norm_bwd(dy.contiguous(), x.contiguous(), w, mean2, rstd2)
        for a, c in zip(got, want):
            assert a.shape == c.shape and bool((a == c).all()), name
        kept = t.clone()
        inside = views(kept)[[v[0] for v in views(t)].index(name)][1]
        lconv.layer_norm(inside, w, b, out=inside)                # in place, and nothing else is touched
        assert bool((inside == y).all())
        inside.copy_(x)
        assert bool((kept == t).all()), name
