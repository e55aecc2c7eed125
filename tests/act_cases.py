"""Inputs and comparisons shared by the activation-checkpoint tests."""

import numpy as np

from oracle import rounding

# A rounding to 16 bits is off by half a step: eps / 2 relative, or half the
# smallest subnormal.
HALF = {"f16": (2.0 ** -11, 2.0 ** -25), "bf16": (2.0 ** -8, 2.0 ** -134)}
# Hardware exp2 and reciprocal may flush what lies below the fp32 normal range.
TINY = 2.0 ** -120


def activation(rng, rows, cols, dtype, std=1.0):
    x = rng.standard_normal((rows, cols)) * std
    x *= np.where(rng.random(cols) < 1 / 64, 8.0, 1.0)
    return rounding.narrow(x.astype(np.float32), dtype).reshape(rows, cols)


def wide(bits, dtype):
    return rounding.widen(bits, dtype).astype(np.float64)


def close16(got_bits, want, err, dtype, what):
    """A 16-bit result within its rounding and the float32 evaluation's bound of the float64 value."""
    got = wide(got_bits, dtype)
    rel, sub = HALF[dtype]
    bound = rel * (np.abs(want) + err) + sub + err + TINY
    # beyond the largest finite value the result may be infinite
    big = 65504.0 if dtype == "f16" else 3.38e38
    ok = (np.abs(got - want) <= bound) | ((np.abs(want) + bound >= big) & ~(np.abs(got) < big * 0.99))
    if not ok.all():
        i = np.unravel_index(np.argmax(np.where(ok, 0, np.abs(got - want) / bound)), got.shape)
        raise AssertionError(f"{what} at {i}: {got[i]!r}, exact {want[i]!r}, bound {bound[i] if bound.ndim else bound!r}")


def close32(got, want, err, what):
    got = np.asarray(got, np.float64)
    bound = err + 2.0 ** -24 * np.abs(want)
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), f"{what}: {got[bad][:3]} vs {want[bad][:3]} (bound {bound[bad][:3]})"
