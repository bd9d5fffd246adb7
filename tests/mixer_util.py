"""Helpers of the mixer operators' GPU tests: seeded inputs in the storage types, error measures and
the tolerances."""
import numpy as np

from tests.gpu_util import say  # noqa: F401

# Half a unit in the last place, relative to a power of two.
ULP = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}

# Relative L2 error of many values stored in the dtype.  16-bit: rounding is off by at most 2^-8 for
# bf16's 8 bits and by less than 2^-9 in the root mean square; one operand of each matrix product --
# scores or state -- is rounded once more, so two such roundings add, with a third as headroom.  fp32:
# sums of at most 4096 products, 64 half-units where roundings add like a random walk (sqrt(4096)).
TOL = {"f32": 64 * 2.0 ** -24, "f16": 3 * 2.0 ** -12, "bf16": 3 * 2.0 ** -9}
# fp32 results (states, statistics, weight gradients) of any input type.
TOL_F32 = 64 * 2.0 ** -24


def tdtype(dtype):
    import torch
    return {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[dtype]


def host(rng, shape, dtype, scale=1.0):
    """A CPU tensor of the storage type."""
    import torch
    return torch.from_numpy(rng.standard_normal(shape, dtype=np.float32) * np.float32(scale)).to(tdtype(dtype))


def wide(t):
    return None if t is None else t.detach().cpu().double().numpy()


def rel(got, ref):
    """Relative L2 error over everything; nan and inf in the result fail."""
    got = wide(got) if not isinstance(got, np.ndarray) else got
    assert got.shape == ref.shape, (got.shape, ref.shape)
    if not np.all(np.isfinite(got)):
        return float("inf")
    n = np.linalg.norm(ref)
    return float(np.linalg.norm(got - ref) / n) if n else float(np.linalg.norm(got))


def rel_rows(got, ref):
    """The largest relative L2 error of a (b, h) row."""
    got = wide(got)
    return max(rel(got[b, h], ref[b, h]) for b in range(ref.shape[0]) for h in range(ref.shape[1]))


def off_by(got, ref, dtype, size):
    """The largest error of an element beyond the rounding to its type (half a unit of the result's own
    binade), as a fraction of `size`, the magnitude of the terms that made it: the fp32 arithmetic's
    share."""
    got = wide(got)
    assert got.shape == ref.shape and np.all(np.isfinite(got))
    least = {"f32": -126, "f16": -14, "bf16": -126}[dtype]
    binade = np.maximum(np.floor(np.log2(np.maximum(np.abs(ref), 1e-300))), least)
    over = np.abs(got - ref) - ULP[dtype] * 2.0 ** binade
    return float(np.max(over / np.maximum(size, 1e-30), initial=0.0))
