"""Bounds that the activation kernels' comments state, recomputed (CPU).

The fp32 constants are read from the kernels' source, so that what is checked is what is built.
"""

import os
import re

import numpy as np
import pytest
from scipy import special

from oracle import act

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "zero_sharded_mixed_flat_amd", "csrc")


def _tail_polynomial():
    """(0.32, coefficients from t^7 down to t^0) as written in act.hip."""
    with open(os.path.join(CSRC, "act.hip")) as f:
        text = f.read()
    body = text[text.index("float normal_tail(float a) {"):text.index("return t * p;")]
    rate = float(re.search(r"fmaf\((0\.\d+)f, a, 1\.0f\)", body).group(1))
    coef = [float.fromhex(c) for c in re.findall(r"-?0x1\.[0-9a-f]+p[-+]\d+", body)]
    assert len(coef) == 8
    return np.float32(rate), [np.float32(c) for c in coef]


# a = 0 to 60 in steps of 2^-13: every value is an fp32 one.
A = np.arange(0, 60 * 8192 + 1) / 8192.0


def test_normal_tail_polynomial():
    rate, coef = _tail_polynomial()
    assert [float(c) for c in coef] == [float(np.float32(c)) for c in coef]
    want = special.erfcx(A / np.sqrt(2.0)) / 2                  # exp(a^2/2) P(-a)
    t = 1.0 / (1.0 + float(rate) * A)
    p = np.zeros_like(t)
    for c in coef:
        p = p * t + float(c)
    assert np.abs(p * t / want - 1).max() < 5.0e-7
    # in fp32, fused multiply-adds as one rounding each
    fma = lambda x, y, z: (x.astype(np.float64) * np.float64(y) + np.float64(z)).astype(np.float32)
    a = A.astype(np.float32)
    t = (np.float32(1) / fma(a, rate, 1.0)).astype(np.float32)
    p = np.full_like(t, coef[0])
    for c in coef[1:]:
        p = fma(p, t, c)
    assert np.abs((t * p).astype(np.float32) / want - 1).max() < 8e-7


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("bits,margin", [(11, 2.0 ** -19), (8, 2.0 ** -16)])
def test_quotients_stay_away_from_rounding_boundaries(fmt, bits, margin):
    # x / scale with scale = A / qmax, A and x of `bits` significant bits: relative distance of qmax x / A from every
    # midpoint of two codes that it is not on, in exact integers.
    sig = np.arange(1 << (bits - 1), 1 << bits, dtype=np.int64)
    x, a = np.meshgrid(sig, sig, indexing="ij")
    qmax = 127 if fmt == "int8" else 448
    values = np.arange(128.0) if fmt == "int8" else act.e4m3_values()
    mids = ((values[1:] + values[:-1]) / 2 * 1024).astype(np.int64)           # exact in units of 2^-10
    least = 1.0
    for shift in range(22 if fmt == "e4m3" else 10):
        num, den = qmax * x << 10, a << shift                                 # the quotient in units of 2^-10
        inside = num <= (qmax << 10) * den
        near = np.searchsorted(mids, num / den)
        for j in (np.maximum(near - 1, 0), np.minimum(near, len(mids) - 1)):
            off = np.abs(num - mids[j] * den)
            least = min(least, (off / num)[inside & (off > 0)].min())
    assert margin <= least < 16 * margin
