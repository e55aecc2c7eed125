"""8-bit activation checkpoints and the operators that write and read them.

Test infrastructure: see the package docstring.

Pages: a checkpointed activation is stored in the forward pass and read again
in the backward pass, and may be partitioned over ranks (CMU 11-868 Lecture 18
notes §4.1, §4.2).  The pages store it in 16 bits; 8 bits with one scale per 256
values is the format they give for parameters (§4.5), applied here along the
rows of an activation matrix.

The decisions (scale, code, restored 16-bit value) are float32 IEEE operations
written out in numpy, compared bit for bit.  Everything computed from them
(activation, norm, gradients) is in float64, with next to each value a bound on
what a float32 evaluation may be off by before its last rounding: the `_err`
arrays, in the units of the value, for U = 2^-24 per operation.
"""

import math

import numpy as np
from scipy import special

from .rounding import is_finite16, narrow, widen

BLOCK = 256
QMAX = {"int8": np.float32(127.0), "e4m3": np.float32(448.0)}
U = 2.0 ** -24


def e4m3_values():
    """The 127 non-negative finite values of 4 exponent bits (bias 7) and 3 mantissa bits, by code."""
    vals = []
    for code in range(127):
        e, m = code >> 3, code & 7
        vals.append(math.ldexp(m, -9) if e == 0 else math.ldexp(8 + m, e - 10))
    return np.array(vals)


_E4M3 = e4m3_values()
_E4M3_MID = (_E4M3[1:] + _E4M3[:-1]) / 2          # exact in float64


def e4m3_encode(q):
    """float32 values, |q| <= 448 after clamping -> code bytes (nearest, ties to the even code)."""
    a = np.minimum(np.abs(q.astype(np.float64)), 448.0)
    lo = np.searchsorted(_E4M3_MID, a, side="left")       # a <= mid[lo]
    tie = (lo < len(_E4M3_MID)) & (a == _E4M3_MID[np.minimum(lo, len(_E4M3_MID) - 1)])
    code = np.where(tie & (lo % 2 == 1), lo + 1, lo).astype(np.uint8)
    return np.where(np.signbit(q), code | 0x80, code).astype(np.uint8)


def e4m3_decode(code):
    v = _E4M3[np.minimum(code & 0x7F, 126)].astype(np.float32)
    return np.where(code & 0x80, -v, v).astype(np.float32)


def save(bits16, dtype, fmt):
    """[rows, cols] patterns -> (code bytes [rows, cols], scales [rows, blocks])."""
    rows, cols = bits16.shape
    nb = -(-cols // BLOCK)
    codes = np.zeros((rows, cols), np.uint8)
    scales = np.zeros((rows, nb), np.float32)
    for b in range(nb):
        part = bits16[:, b * BLOCK:(b + 1) * BLOCK]
        x = widen(part, dtype)
        finite = is_finite16(part, dtype).all(axis=1)
        amax = np.where(finite, np.abs(np.where(is_finite16(part, dtype), x, 0)).max(axis=1), 0).astype(np.float32)
        s = (amax / QMAX[fmt]).astype(np.float32)
        live = (s > 0)[:, None]
        with np.errstate(invalid="ignore", over="ignore"):
            q = np.where(live, x / np.where(live, s[:, None], np.float32(1)), np.float32(0)).astype(np.float32)
        q = np.where(finite[:, None], q, np.float32(0))
        q = np.clip(q, -QMAX[fmt], QMAX[fmt])
        c = np.rint(q).astype(np.int8).view(np.uint8) if fmt == "int8" else e4m3_encode(q)
        codes[:, b * BLOCK:(b + 1) * BLOCK] = np.where(live & finite[:, None], c, 0)
        scales[:, b] = np.where(finite, s, np.float32(np.nan))
    return codes, scales


def restore(codes, scales, dtype, fmt):
    """-> 16-bit patterns: round16(float32(code * scale))."""
    v = codes.view(np.int8).astype(np.float32) if fmt == "int8" else e4m3_decode(codes)
    s = np.repeat(scales, BLOCK, axis=1)[:, :codes.shape[1]]
    with np.errstate(invalid="ignore"):
        return narrow((v * s).astype(np.float32), dtype)


def act(g, fn):
    """f(g), f'(g) in float64 and what float32 may be off by: (f, f_err, df, df_err).

    An exponential of argument z carries |z| + 1 roundings of its argument (the
    product with log2 e and the constant itself), plus a few ulps for the
    exponential, the reciprocal and the operations after it: 16 in all.  The
    normal tail's polynomial is good to 8e-7, 14 U.
    """
    g = np.asarray(g, np.float64)
    if fn == "gelu":
        cdf = special.ndtr(g)
        pdf = np.exp(-g * g / 2) / math.sqrt(2 * math.pi)
        k = (g * g + 32) * 2 * U
        return g * cdf, k * np.abs(g * cdf), cdf + g * pdf, k * (cdf + np.abs(g * pdf))
    if fn == "silu":
        z, zp = g, np.ones_like(g)
    else:
        z = math.sqrt(8 / math.pi) * (g + 0.044715 * g ** 3)
        zp = math.sqrt(8 / math.pi) * (1 + 3 * 0.044715 * g * g)
    s, c = special.expit(z), special.expit(-z)
    k = (np.minimum(np.abs(z), 128) + 16) * 2 * U
    return g * s, k * np.abs(g * s), s * (1 + g * c * zp), k * s * (1 + np.abs(g * c * zp))


def glu_forward(gate, up, fn):
    """float64 inputs -> (h, err); up may be None."""
    f, fe, _, _ = act(gate, fn)
    if up is None:
        return f, fe
    return f * up, fe * np.abs(up) + U * np.abs(f * up)


def glu_backward(g, u, dh, fn):
    """Restored g, u (or None) -> ((dgate, err), (dup, err) or None, (h, err))."""
    f, fe, df, dfe = act(g, fn)
    uu = np.ones_like(g) if u is None else u
    a = dh * uu * df
    dgate = (a, np.abs(dh * uu) * dfe + 3 * U * np.abs(a))
    h = (f * uu, fe * np.abs(uu) + U * np.abs(f * uu))
    return dgate, (None if u is None else (dh * f, np.abs(dh) * fe + U * np.abs(dh * f))), h


# Longest chain of float32 additions of a row sum: 32 elements per lane, 6 steps
# across a wave, 16 waves, and the handful of operations before and after.
ROW_DEPTH = 64


def residual(x, branch, alpha, dtype):
    """16-bit patterns -> the residual stream's patterns: float32 product, float32 sum, one rounding to 16 bits."""
    p = (np.float32(alpha) * widen(branch, dtype)).astype(np.float32)
    return narrow((widen(x, dtype) + p).astype(np.float32), dtype)


def norm_forward(r, weight, bias, kind, eps):
    """float64 r [rows, cols] -> (y, err), (rstd, err), (mean, err)."""
    mean = r.mean(axis=1, keepdims=True) if kind == "layer" else np.zeros((r.shape[0], 1))
    d = r - mean
    rstd = 1 / np.sqrt((d * d).mean(axis=1, keepdims=True) + float(np.float32(eps)))
    size = np.abs(r).mean(axis=1, keepdims=True)
    mean_err = ROW_DEPTH * U * size if kind == "layer" else np.zeros_like(mean)
    # the variance moves by its own roundings, by 2 d U(|r| + |mean|) per element and by the mean's error
    rstd_err = rstd * (ROW_DEPTH * U + (rstd ** 2) * (np.abs(d) * (2 * U * (np.abs(r) + np.abs(mean)) + 2 * mean_err)
                                                      ).mean(axis=1, keepdims=True))
    w = 1.0 if weight is None else weight
    n = d * rstd
    n_err = rstd * (mean_err + U * (np.abs(r) + np.abs(mean))) + np.abs(d) * rstd_err + U * np.abs(n)
    y = n * w
    y_err = np.abs(w) * n_err + U * np.abs(y)
    if bias is not None:
        y = y + bias
        y_err = y_err + U * np.abs(y)
    return (y, y_err), (rstd[:, 0], rstd_err[:, 0]), (mean[:, 0], mean_err[:, 0])


def norm_backward(r, mean, rstd, weight, dy, dres, kind, row_chain):
    """Restored r and the float32 statistics as given -> (dr, err), (dweight, err), (dbias, err).

    row_chain: the longest chain of additions in the sums over rows.
    """
    mean = np.zeros((r.shape[0], 1)) if kind == "rms" else mean[:, None]
    rstd = rstd[:, None]
    n = (r - mean) * rstd
    n_err = 2 * U * rstd * (np.abs(r) + np.abs(mean))
    d = dy * (1.0 if weight is None else weight)
    avg = lambda v: v.mean(axis=1, keepdims=True)
    mn = avg(d * n)
    mn_err = ROW_DEPTH * U * avg(np.abs(d * n)) + avg(np.abs(d) * n_err)
    md = avg(d) if kind == "layer" else 0.0
    md_err = ROW_DEPTH * U * avg(np.abs(d)) if kind == "layer" else 0.0
    core = d - n * mn - md
    err = rstd * (md_err + np.abs(n) * mn_err + n_err * np.abs(mn)
                  + 4 * U * (np.abs(d) + np.abs(n * mn) + np.abs(md)))
    dr = rstd * core + dres
    err = err + 2 * U * (np.abs(rstd * core) + np.abs(dr))
    dw = (dy * n).sum(axis=0)
    dw_err = (np.abs(dy) * (row_chain * U * np.abs(n) + n_err)).sum(axis=0)
    return (dr, err), (dw, dw_err), (dy.sum(axis=0), row_chain * U * np.abs(dy).sum(axis=0))


def weight_grad(dy, x):
    """dW = dy^T x and the bias sums, with the bound of a float32 sum in any order (2 U per addition: a matrix
    instruction's internal additions may truncate)."""
    t = dy.shape[0]
    dw, db = dy.T @ x, dy.sum(axis=0)
    return (dw, 2 * U * t * (np.abs(dy).T @ np.abs(x))), (db, 2 * U * t * np.abs(dy).sum(axis=0))
