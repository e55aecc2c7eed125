"""GPU parity of the gated activation in its far left tail, where exp(-z) leaves the
fp32 range but the activation itself does not.

f(g) is evaluated in fp32: below the normal range it is a multiple of 2^-149, off by
half of that (2^-150) besides the oracle's bound, and the products with up and dh
carry that on.  Nothing else is allowed for, in contrast to a tail flushed to zero.

The oracle's bound counts one rounding of the exponential's argument z; the tanh form's
z has six more (two constants, the square, the sum and two products), each moving the
exponential by |z| 2^-24: its bound of 2 |z| 2^-24 and more is taken fourfold.
"""

import numpy as np
import pytest
import torch

from act_cases import HALF, wide
from oracle import act, rounding
from test_gpu_act import FN, Mat, _ckpt, _note, abi  # noqa: F401

pytestmark = pytest.mark.gpu

# First and last gate: from where the logistic function or the density (times its
# factors) is still far above 2^-126 to where the activation is 0 in fp32.
RANGE = {"silu": (-70.0, -112.0), "gelu_tanh": (-9.0, -11.5), "gelu": (-12.0, -15.0)}


WIDER = {"silu": 1.0, "gelu": 1.0, "gelu_tanh": 4.0}


def _near(got_bits, want, err, what):
    got = wide(got_bits, "bf16")
    rel, sub = HALF["bf16"]
    bound = rel * (np.abs(want) + err) + sub + err
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.size}, first {got[bad][0]!r} for {want[bad][0]!r}"


@pytest.mark.parametrize("fn", sorted(FN))
@pytest.mark.parametrize("up", [None, 1.0, 2.0 ** 30, -(2.0 ** 100)])
def test_far_tail(abi, fn, up):
    _note(f"tail {fn} up {up}")
    hi, lo = RANGE[fn]
    bits = np.unique(rounding.narrow(np.linspace(lo, hi, 400).astype(np.float32), "bf16"))
    rows, cols = len(bits), 8                        # a value per row: a block of its own, restored exactly
    x = np.repeat(bits[:, None], cols, 1)
    u = None if up is None else rounding.narrow(np.full((rows, cols), up, np.float32), "bf16").reshape(rows, cols)
    dh = rounding.narrow(np.full((rows, cols), -1.5, np.float32), "bf16").reshape(rows, cols)
    m, h, again = Mat(rows, cols, "bf16", x), Mat(rows, cols, "bf16"), Mat(rows, cols, "bf16")
    mu = None if up is None else Mat(rows, cols, "bf16", u)
    d, dg = Mat(rows, cols, "bf16", dh), Mat(rows, cols, "bf16")
    du = None if up is None else Mat(rows, cols, "bf16")
    t = lambda v: None if v is None else v.t
    gc, gs = _ckpt(abi, rows, cols)
    uc, us = (None, None) if up is None else _ckpt(abi, rows, cols)
    abi.zero_act_glu_forward(m.t, cols, t(mu), cols, "bf16", rows, cols, FN[fn], 1, h.t, cols, gc, gs, uc, us)
    abi.zero_act_glu_backward(gc, gs, uc, us, 1, rows, cols, FN[fn], d.t, cols, "bf16", dg.t, cols, t(du), cols, again.t,
                              cols)
    torch.cuda.synchronize()
    back = act.restore(*act.save(x, "bf16", "int8"), "bf16", "int8")
    assert np.array_equal(back, x)
    g = wide(x, "bf16")
    u64 = None if up is None else wide(act.restore(*act.save(u, "bf16", "int8"), "bf16", "int8"), "bf16")
    assert up is None or (u64 == up).all()
    scale = 1.0 if up is None else abs(up)
    k, least = WIDER[fn], 2.0 ** -150
    v, e = act.glu_forward(g, u64, fn)
    _near(h.bits(), v, k * e + (scale + 1) * least, "h")
    (a, ae), b, (r, re) = act.glu_backward(g, u64, wide(dh, "bf16"), fn)
    _near(dg.bits(), a, k * ae + (1.5 * scale + 1) * least, "dgate")
    _near(again.bits(), r, k * re + (scale + 1) * least, "recomputed h")
    if up is not None:
        _near(du.bits(), b[0], k * b[1] + 2.5 * least, "dup")


@pytest.mark.parametrize("fn", sorted(FN))
def test_the_ordinary_range_meets_the_tail(abi, fn):
    # Every bf16 gate value between the ordinary range and the tail: no step where they meet.
    hi, lo = RANGE[fn]
    first, last = rounding.narrow(np.array([hi / 4, lo], np.float32), "bf16")
    bits = np.arange(int(first), int(last) + 1, dtype=np.uint16)
    x = np.repeat(bits[:, None], 8, 1)
    m, h = Mat(len(bits), 8, "bf16", x), Mat(len(bits), 8, "bf16")
    gc, gs = _ckpt(abi, len(bits), 8)
    abi.zero_act_glu_forward(m.t, 8, None, 0, "bf16", len(bits), 8, FN[fn], 1, h.t, 8, gc, gs, None, None)
    torch.cuda.synchronize()
    v, e = act.glu_forward(wide(x, "bf16"), None, fn)
    _near(h.bits(), v, WIDER[fn] * e + 2.0 ** -150, "h")
