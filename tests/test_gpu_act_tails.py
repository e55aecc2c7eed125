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


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("fn", sorted(FN))
def test_blocks_that_mix_tail_and_ordinary_values(abi, fn, fmt):
    # Octs with and without tail values, blocks whose largest magnitude is a positive value, a value just at the
    # tail's border, and one with a NaN, whose other values keep their own activation.
    rng = np.random.default_rng(5)
    rows, cols = 24, 530
    hi, lo = RANGE[fn]
    x = np.where(rng.random((rows, cols)) < 0.1, rng.uniform(lo, hi / 2, (rows, cols)), rng.standard_normal((rows, cols)))
    x[3] = np.abs(x[3])
    x[4] = hi * 0.98
    x[5, ::8] = -lo
    bits = rounding.narrow(x.astype(np.float32), "bf16").reshape(rows, cols)
    bits[7, 100] = 0xFFC0                            # a NaN with its sign set
    bits[8, 300] = 0xFF80                            # minus infinity
    u = rounding.narrow((rng.standard_normal((rows, cols)) * 2.0 ** 60).astype(np.float32), "bf16").reshape(rows, cols)
    fm = {"int8": 1, "e4m3": 2}[fmt]
    m, mu, h = Mat(rows, cols, "bf16", bits), Mat(rows, cols, "bf16", u), Mat(rows, cols, "bf16", pad=3)
    (gc, gs), (uc, us) = _ckpt(abi, rows, cols), _ckpt(abi, rows, cols)
    abi.zero_act_glu_forward(m.t, cols, mu.t, cols, "bf16", rows, cols, FN[fn], fm, h.t, h.stride, gc, gs, uc, us)
    dh = rounding.narrow(rng.standard_normal((rows, cols)).astype(np.float32), "bf16").reshape(rows, cols)
    d, dg, du = Mat(rows, cols, "bf16", dh), Mat(rows, cols, "bf16"), Mat(rows, cols, "bf16")
    abi.zero_act_glu_backward(gc, gs, uc, us, fm, rows, cols, FN[fn], d.t, cols, "bf16", dg.t, cols, du.t, cols)
    torch.cuda.synchronize()
    k, least = WIDER[fn], 2.0 ** -150
    bad = np.zeros((rows, cols), bool)
    bad[7, 100] = bad[8, 300] = True
    g, uu = wide(np.where(bad, 0, bits).astype(np.uint16), "bf16"), wide(u, "bf16")
    v, e = act.glu_forward(g, uu, fn)
    got = h.bits()
    assert np.isnan(wide(got, "bf16")[bad]).all()
    _near(got[~bad], v[~bad], (k * e + (np.abs(uu) + 1) * least)[~bad], "h")
    rg = wide(act.restore(*act.save(bits, "bf16", fmt), "bf16", fmt), "bf16")
    ru = wide(act.restore(*act.save(u, "bf16", fmt), "bf16", fmt), "bf16")
    nan = np.isnan(rg)
    assert nan[7, :256].all() and nan[8, 256:512].all() and nan.sum() == 512
    d64 = wide(dh, "bf16")
    (a, ae), (b, be), _ = act.glu_backward(np.where(nan, 0, rg), ru, d64, fn)
    for out, want, err, what in ((dg, a, k * ae + (np.abs(d64 * ru) + 1) * least, "dgate"),
                                 (du, b, k * be + (np.abs(d64) + 1) * least, "dup")):
        assert np.isnan(wide(out.bits(), "bf16")[nan]).all()
        _near(out.bits()[~nan], want[~nan], err[~nan], what)
    assert h.guards_intact()
