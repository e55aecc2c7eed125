"""GPU parity of the 8-bit activation checkpoint, the gated activation and the
residual norm against the oracle.

Codes, scales and restored values are float32 decisions and are compared bit
for bit; computed results lie within one 16-bit rounding plus the bound that
the oracle derives for a float32 evaluation.
"""

import numpy as np
import pytest
import torch

from act_cases import activation, close16, close32, wide
from oracle import act, quant, rounding

pytestmark = pytest.mark.gpu

TORCH16 = {"f16": torch.float16, "bf16": torch.bfloat16}
FMT = {"int8": 1, "e4m3": 2}
FN = {"silu": 1, "gelu": 2, "gelu_tanh": 3}
KIND = {"rms": 1, "layer": 2}


@pytest.fixture(scope="module")
def abi():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from zero_sharded_mixed_flat_amd import abi as _abi
    return _abi


def _note(msg):
    print(msg, flush=True)


class Mat:
    """A [rows, cols] device matrix inside a larger buffer (row pad, element offset) filled with a guard pattern."""

    def __init__(self, rows, cols, dtype, bits=None, pad=0, off=0):
        self.rows, self.cols, self.stride, self.dtype = rows, cols, cols + pad, dtype
        self.buf = torch.full((off + rows * self.stride + 8,), 0x5A5A, dtype=torch.int16, device="cuda")
        self.view = self.buf[off:off + rows * self.stride].view(TORCH16[dtype]).view(rows, self.stride)
        self.t = self.view[:, :cols]
        self.off = off
        if bits is not None:
            self.t.copy_(torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).cuda().view(TORCH16[dtype]))

    def bits(self):
        return self.t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)

    def guards_intact(self):
        b = self.buf.cpu().numpy()
        body = b[self.off:self.off + self.rows * self.stride].reshape(self.rows, self.stride)
        return (b[:self.off] == 0x5A5A).all() and (b[self.off + self.rows * self.stride:] == 0x5A5A).all() and \
            (body[:, self.cols:] == 0x5A5A).all()


def _ckpt(abi, rows, cols):
    return (torch.full((abi.zero_act_code_bytes(rows, cols) + 16,), 0x77, dtype=torch.uint8, device="cuda"),
            torch.full((abi.zero_act_scale_count(rows, cols) + 1,), -5.0, device="cuda"))


def _host_ckpt(codes, scales, rows, cols):
    pitch, nb = (cols + 15) // 16 * 16, -(-cols // 256)
    c = codes.cpu().numpy()
    s = scales.cpu().numpy()
    assert (c[rows * pitch:] == 0x77).all() and s[rows * nb] == -5.0        # nothing past the end
    c = c[:rows * pitch].reshape(rows, pitch)
    assert not c[:, cols:].any()                                            # pad bytes are 0
    return c[:, :cols].copy(), s[:rows * nb].reshape(rows, nb)


def _dev_ckpt(codes, scales):
    rows, cols = codes.shape
    buf = np.zeros((rows, (cols + 15) // 16 * 16), np.uint8)
    buf[:, :cols] = codes
    return torch.from_numpy(buf).cuda(), torch.from_numpy(scales.copy()).cuda()


def _same_ckpt(got, want, what):
    (gc, gs), (wc, ws) = got, want
    assert np.array_equal(gs, ws, equal_nan=True), f"{what} scales"
    assert np.array_equal(gc, wc), f"{what} codes: {np.argwhere(gc != wc)[:5]}"


SHAPES = [(1, 1), (1, 1600), (3, 7), (2, 255), (5, 256), (4, 257), (33, 4801), (257, 1000)]


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("pad,off", [(0, 0), (5, 3)])
def test_save_restore(abi, fmt, dtype, rows, cols, pad, off):
    _note(f"save {fmt} {dtype} {rows}x{cols} pad {pad} off {off}")
    x = activation(np.random.default_rng(rows * 7 + cols), rows, cols, dtype)
    m, y = Mat(rows, cols, dtype, x, pad, off), Mat(rows, cols, dtype, None, pad, off)
    codes, scales = _ckpt(abi, rows, cols)
    abi.zero_act_save(m.t, m.stride, dtype, rows, cols, FMT[fmt], codes, scales)
    abi.zero_act_restore(codes, scales, FMT[fmt], rows, cols, y.t, y.stride, dtype)
    torch.cuda.synchronize()
    want = act.save(x, dtype, fmt)
    _same_ckpt(_host_ckpt(codes, scales, rows, cols), want, "saved")
    assert np.array_equal(y.bits(), act.restore(*want, dtype, fmt))
    assert y.guards_intact() and m.guards_intact()


def test_restore_into_the_other_type(abi):
    x = activation(np.random.default_rng(5), 9, 700, "bf16")
    codes, scales = act.save(x, "bf16", "e4m3")
    y = Mat(9, 700, "f16")
    abi.zero_act_restore(*_dev_ckpt(codes, scales), 2, 9, 700, y.t, y.stride, "f16")
    torch.cuda.synchronize()
    assert np.array_equal(y.bits(), act.restore(codes, scales, "f16", "e4m3"))


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_codes_for_every_pair_of_magnitudes(abi, fmt):
    # Every fp16 significand as the block maximum against every fp16 significand over 13 binades (INT8) or 20
    # (E4M3): the multiplied and corrected quotient must take the IEEE division's decisions.
    qmax = 127.0 if fmt == "int8" else 448.0
    binades = 13 if fmt == "int8" else 20
    sig = np.arange(1024, dtype=np.int64)
    # values with biased exponents 25 - k.. below the maximum's 25; fp16 patterns
    xs = np.concatenate([((25 - k) << 10 | sig).astype(np.uint16) for k in range(1, binades)])
    xs = np.concatenate([xs, np.arange(25 << 10, 26 << 10).astype(np.uint16)])
    xs = np.resize(xs, -(-xs.size // 255) * 255).reshape(-1, 255)
    per = xs.shape[0]
    for a0 in range(0, 1024, 128):
        top = torch.arange(a0, a0 + 128, dtype=torch.int32) + (25 << 10)
        rows = torch.from_numpy(xs.astype(np.int32)).cuda().repeat(128, 1)
        amax = top.cuda().repeat_interleave(per)[:, None]
        body = torch.minimum(rows, amax.expand_as(rows))     # magnitudes above the maximum become the maximum
        m = torch.cat([body, amax], 1).to(torch.int16).contiguous()
        m[:, ::2] |= -32768                                   # alternate signs
        n = m.shape[0]
        _note(f"pairs {fmt} from {a0}: {n} blocks")
        codes = torch.empty(n, 256, dtype=torch.uint8, device="cuda")
        scales = torch.empty(n, device="cuda")
        x = m.view(torch.float16)
        abi.zero_act_save(x, 256, "f16", n, 256, FMT[fmt], codes, scales)
        v = x.float()
        s = v.abs().amax(1) / torch.tensor(qmax, device="cuda")
        q = v / s[:, None]
        q = q.clamp(-qmax, qmax)
        want = q.round().to(torch.int8).view(torch.uint8) if fmt == "int8" else q.to(torch.float8_e4m3fn).view(torch.uint8)
        assert torch.equal(scales, s)
        assert torch.equal(codes, want), f"{int((codes != want).sum())} codes differ"


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_far_ranges_of_bf16(abi, fmt):
    # Blocks from the smallest subnormals to the largest finite values, zeros, infinities and NaN.
    rng = np.random.default_rng(11)
    tops = np.concatenate([[1, 2, 3, 0x7F, 0x80, 0x81], np.arange(0x0100, 0x7F80, 0x173), [0x7F7F, 0x0000]])
    x = np.zeros((len(tops) + 2, 300), np.uint16)
    for i, t in enumerate(tops):
        x[i] = rng.integers(0, t + 1, 300) | (rng.integers(0, 2, 300) << 15)
        x[i, 17] = t
    x[-2, 40] = 0x7F80
    x[-1, 299] = 0xFFC1
    m = Mat(*x.shape, "bf16", x)
    codes, scales = _ckpt(abi, *x.shape)
    abi.zero_act_save(m.t, m.stride, "bf16", *x.shape, FMT[fmt], codes, scales)
    y = Mat(*x.shape, "bf16")
    abi.zero_act_restore(codes, scales, FMT[fmt], *x.shape, y.t, y.stride, "bf16")
    torch.cuda.synchronize()
    want = act.save(x, "bf16", fmt)
    _same_ckpt(_host_ckpt(codes, scales, *x.shape), want, "far")
    back, ref = y.bits(), act.restore(*want, "bf16", fmt)
    nan = np.isnan(rounding.widen(ref, "bf16"))
    assert np.array_equal(np.isnan(rounding.widen(back, "bf16")), nan) and np.array_equal(back[~nan], ref[~nan])
    assert nan[-2, :256].all() and not nan[-2, 256:].any() and nan[-1, 256:].all() and not nan[-1, :256].any()


def test_int8_is_the_flat_quantisers(abi):
    x = activation(np.random.default_rng(2), 12, 768, "bf16")
    d = Mat(12, 768, "bf16", x)
    codes, scales = _ckpt(abi, 12, 768)
    abi.zero_act_save(d.t, d.stride, "bf16", 12, 768, 1, codes, scales)
    c2 = torch.empty(12 * 768, dtype=torch.uint8, device="cuda")
    s2 = torch.empty(36, device="cuda")
    abi.zero_quantize_blocks(d.t.contiguous(), "bf16", 12 * 768, 8, c2, s2)
    torch.cuda.synchronize()
    assert torch.equal(codes[:12 * 768], c2) and torch.equal(scales[:36], s2)


def test_a_very_long_row_and_very_many_short_ones(abi):
    n = 100_000_007
    x = torch.randn(n, device="cuda").to(torch.bfloat16)
    codes = torch.empty(abi.zero_act_code_bytes(1, n), dtype=torch.uint8, device="cuda")
    scales = torch.empty(abi.zero_act_scale_count(1, n), device="cuda")
    abi.zero_act_save(x, n, "bf16", 1, n, 1, codes, scales)
    c2 = torch.empty(n, dtype=torch.uint8, device="cuda")
    s2 = torch.empty_like(scales)
    abi.zero_quantize_blocks(x, "bf16", n, 8, c2, s2)
    torch.cuda.synchronize()
    assert torch.equal(codes[:n], c2) and not codes[n:].any() and torch.equal(scales, s2)
    rows = 3_000_001
    codes = torch.empty(rows, 16, dtype=torch.uint8, device="cuda")
    scales = torch.empty(rows, device="cuda")
    y = torch.empty(rows, dtype=torch.bfloat16, device="cuda")
    abi.zero_act_save(x, 1, "bf16", rows, 1, 1, codes, scales)
    abi.zero_act_restore(codes, scales, 1, rows, 1, y, 1, "bf16")
    torch.cuda.synchronize()
    v = x[:rows].float()
    assert torch.equal(scales, v.abs() / torch.tensor(127.0, device="cuda"))
    assert torch.equal(codes[:, 0].view(torch.int8).float(), 127 * torch.sign(v)) and not codes[:, 1:].any()
    assert torch.equal(y, (127 * torch.sign(v) * scales).to(torch.bfloat16))


def test_rows_of_a_checkpoint_are_a_checkpoint(abi):
    # A rank holding rows 20..60 of a partitioned checkpoint restores them from pointers alone.
    x = activation(np.random.default_rng(8), 64, 530, "f16")
    codes, scales = act.save(x, "f16", "int8")
    dc, ds = _dev_ckpt(codes, scales)
    y = Mat(40, 530, "f16")
    abi.zero_act_restore(dc[20:60], ds[20:60], 1, 40, 530, y.t, y.stride, "f16")
    torch.cuda.synchronize()
    assert np.array_equal(y.bits(), act.restore(codes, scales, "f16", "int8")[20:60])


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("fn", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("gated", [True, False])
@pytest.mark.parametrize("rows,cols", [(1, 5), (3, 1600), (37, 261), (130, 1024)])
def test_glu(abi, fmt, dtype, fn, gated, rows, cols):
    _note(f"glu {fmt} {dtype} {fn} gated {gated} {rows}x{cols}")
    rng = np.random.default_rng(rows + cols)
    parts = 2 if gated else 1
    x = activation(rng, rows, parts * cols, dtype, 2.0)
    x[0, :min(cols, 5)] = rounding.narrow(np.array([0.0, -0.0, 12.0, -12.0, 1e-6], np.float32), dtype)[:min(cols, 5)]
    both = Mat(rows, parts * cols, dtype, x, pad=3, off=1)                 # gate and up interleave
    gate, up = both.t[:, :cols], both.t[:, cols:] if gated else None
    h = Mat(rows, cols, dtype)
    gc, gs = _ckpt(abi, rows, cols)
    uc, us = _ckpt(abi, rows, cols) if gated else (None, None)
    abi.zero_act_glu_forward(gate, both.stride, up, both.stride, dtype, rows, cols, FN[fn], FMT[fmt], h.t, h.stride,
                             gc, gs, uc, us)
    torch.cuda.synchronize()
    g64, u64 = wide(x[:, :cols], dtype), wide(x[:, cols:], dtype) if gated else None
    close16(h.bits(), *act.glu_forward(g64, u64, fn), dtype, "h")
    want = act.save(x[:, :cols], dtype, fmt)
    _same_ckpt(_host_ckpt(gc, gs, rows, cols), want, "gate")
    if gated:
        wu = act.save(x[:, cols:], dtype, fmt)
        _same_ckpt(_host_ckpt(uc, us, rows, cols), wu, "up")
    dh = activation(rng, rows, cols, dtype, 0.02)
    d = Mat(rows, cols, dtype, dh, pad=1)
    dx = Mat(rows, parts * cols, dtype, None, pad=5, off=3)
    again = Mat(rows, cols, dtype, None, pad=2)
    dgate, dup = dx.t[:, :cols], dx.t[:, cols:] if gated else None
    abi.zero_act_glu_backward(gc, gs, uc, us, FMT[fmt], rows, cols, FN[fn], d.t, d.stride, dtype, dgate, dx.stride, dup,
                              dx.stride, again.t, again.stride)
    torch.cuda.synchronize()
    rg = wide(act.restore(*want, dtype, fmt), dtype)
    ru = wide(act.restore(*wu, dtype, fmt), dtype) if gated else None
    a, b, c = act.glu_backward(rg, ru, wide(dh, dtype), fn)
    out = dx.bits()
    close16(out[:, :cols], *a, dtype, "dgate")
    if gated:
        close16(out[:, cols:], *b, dtype, "dup")
    close16(again.bits(), *c, dtype, "recomputed h")
    assert dx.guards_intact() and again.guards_intact() and h.guards_intact()


@pytest.mark.parametrize("fn", ["silu", "gelu", "gelu_tanh"])
def test_glu_at_the_ends_of_the_range(abi, fn):
    # bf16 values up to the largest finite ones, and non-finite ones, which the backward pass must show.
    vals = np.array([0x7F7F, 0xFF7F, 0x42B0, 0xC2B0, 0x4170, 0xC170, 0x0001, 0x8001, 0x0080, 0x3F80], np.uint16)
    for v in vals:
        x = np.full((1, 8), v, np.uint16)
        m, h = Mat(1, 8, "bf16", x), Mat(1, 8, "bf16")
        gc, gs = _ckpt(abi, 1, 8)
        abi.zero_act_glu_forward(m.t, 8, None, 0, "bf16", 1, 8, FN[fn], 1, h.t, 8, gc, gs, None, None)
        one = Mat(1, 8, "bf16", np.full((1, 8), 0x3F80, np.uint16))
        dg = Mat(1, 8, "bf16")
        abi.zero_act_glu_backward(gc, gs, None, None, 1, 1, 8, FN[fn], one.t, 8, "bf16", dg.t, 8, None, 0)
        torch.cuda.synchronize()
        with np.errstate(over="ignore", invalid="ignore"):
            g = wide(x, "bf16")
            back = wide(act.restore(*act.save(x, "bf16", "int8"), "bf16", "int8"), "bf16")
            f, fe, _, _ = act.act(np.clip(g, -1e3, None), fn)
            f = np.where(g < -1e3, 0.0, np.where(g > 1e3, g, f))
            fe = np.where(np.abs(g) > 1e3, 0.0, fe)
            _, _, df, dfe = act.act(np.clip(back, -1e3, 1e3), fn)
        close16(h.bits(), f, fe, "bf16", f"f({v:#x})")
        close16(dg.bits(), df, dfe, "bf16", f"f'({v:#x})")
    for bad in (0x7F80, 0x7FC0):
        x = np.full((2, 260), 0x3F80, np.uint16)
        x[1, 3] = bad
        m, h = Mat(2, 260, "bf16", x), Mat(2, 260, "bf16")
        gc, gs = _ckpt(abi, 2, 260)
        abi.zero_act_glu_forward(m.t, 260, None, 0, "bf16", 2, 260, FN[fn], 1, h.t, 260, gc, gs, None, None)
        one = Mat(2, 260, "bf16", np.full((2, 260), 0x3F80, np.uint16))
        dg = Mat(2, 260, "bf16")
        abi.zero_act_glu_backward(gc, gs, None, None, 1, 2, 260, FN[fn], one.t, 260, "bf16", dg.t, 260, None, 0)
        torch.cuda.synchronize()
        nan = np.isnan(wide(dg.bits(), "bf16"))
        assert nan[1, :256].all() and not nan[0].any() and not nan[1, 256:].any()


NORM_SHAPES = [(1, 1), (3, 16384), (1, 16), (5, 1600), (3, 511), (9, 2049), (4, 4097), (2, 12289), (1030, 37)]


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("dtype,fmt", [("f16", "int8"), ("bf16", "e4m3"), ("bf16", "int8"), ("f16", "e4m3")])
@pytest.mark.parametrize("rows,cols", NORM_SHAPES)
def test_norm(abi, kind, dtype, fmt, rows, cols):
    _note(f"norm {kind} {dtype} {fmt} {rows}x{cols}")
    rng = np.random.default_rng(rows * 31 + cols)
    full = (rows + cols) % 2 == 1                    # weight, bias, branch and dres given; or only what must be
    x = activation(rng, rows, cols, dtype)
    br = activation(rng, rows, cols, dtype, 0.5) if full else None
    w = rounding.narrow((1 + 0.2 * rng.standard_normal(cols)).astype(np.float32), dtype) if full else None
    b = rounding.narrow((0.1 * rng.standard_normal(cols)).astype(np.float32), dtype) if full else None
    vec = lambda v: None if v is None else Mat(1, cols, dtype, v[None], off=1)
    dw_, db_ = vec(w), vec(b)
    t = lambda m: None if m is None else m.t
    mx = Mat(rows, cols, dtype, x, pad=3, off=1)
    mb = Mat(rows, cols, dtype, br, pad=2) if full else None
    mr = Mat(rows, cols, dtype, None, pad=1) if full else None
    my = Mat(rows, cols, dtype, None, pad=7, off=5)
    codes, scales = _ckpt(abi, rows, cols)
    mean = torch.zeros(rows, device="cuda") if kind == "layer" else None
    rstd = torch.zeros(rows, device="cuda")
    alpha, eps = 0.7071, 1e-5
    stride = lambda m: 0 if m is None else m.stride
    abi.zero_act_norm_forward(mx.t, mx.stride, t(mb), stride(mb), alpha, t(dw_), t(db_), dtype, rows, cols, KIND[kind],
                              eps, FMT[fmt], t(mr), stride(mr), my.t, my.stride, codes, scales, mean, rstd)
    torch.cuda.synchronize()
    r = act.residual(x, br, alpha, dtype).reshape(rows, cols) if full else x
    if full:
        assert np.array_equal(mr.bits(), r) and mr.guards_intact()
    w64 = None if w is None else wide(w, dtype)
    y, rs, mn = act.norm_forward(wide(r, dtype), w64, None if b is None else wide(b, dtype), kind, eps)
    close16(my.bits(), *y, dtype, "y")
    close32(rstd.cpu().numpy(), *rs, "rstd")
    if kind == "layer":
        close32(mean.cpu().numpy(), *mn, "mean")
    want = act.save(r, dtype, fmt)
    _same_ckpt(_host_ckpt(codes, scales, rows, cols), want, "residual")
    assert my.guards_intact()

    dy, dr = activation(rng, rows, cols, dtype, 0.02), activation(rng, rows, cols, dtype, 0.02) if full else None
    md, mdr = Mat(rows, cols, dtype, dy, pad=5), Mat(rows, cols, dtype, dr, off=1) if full else None
    dx, dbr = Mat(rows, cols, dtype, None, pad=1, off=3), Mat(rows, cols, dtype) if full else None
    old = activation(rng, 2, cols, dtype, 0.1)
    gw, gb = Mat(1, cols, dtype, old[:1], off=1), Mat(1, cols, dtype, old[1:], off=3)
    ws = torch.empty(abi.zero_act_norm_workspace_bytes(rows, cols), dtype=torch.uint8, device="cuda")
    abi.zero_act_norm_backward(codes, scales, FMT[fmt], mean, rstd, t(dw_), rows, cols, KIND[kind], md.t, md.stride,
                               t(mdr), stride(mdr), alpha, dtype, dx.t, dx.stride, t(dbr), stride(dbr), full, gw.t, gb.t,
                               ws)
    torch.cuda.synchronize()
    d64 = lambda v: v.cpu().numpy().astype(np.float64)
    # a thread's rows, the block's waves, the partials of one way and the fold's tree
    chain = -(-rows // 1024) + 4 + 16 + 8
    a, dw, db = act.norm_backward(wide(act.restore(*want, dtype, fmt), dtype), None if mean is None else d64(mean),
                                  d64(rstd), w64, wide(dy, dtype), wide(dr, dtype) if full else 0.0, kind, chain)
    close16(dx.bits(), *a, dtype, "dx")
    if full:
        al = float(np.float32(alpha))
        close16(dbr.bits(), al * a[0], al * a[1] + 2.0 ** -24 * np.abs(al * a[0]), dtype, "dbranch")
    add = wide(old, dtype) if full else np.zeros((2, cols))
    for got, (v, e), o, what in ((gw, dw, add[0], "dweight"), (gb, db, add[1], "dbias")):
        close16(got.bits()[0], v + o, e + 2.0 ** -24 * np.abs(v + o), dtype, what)
        assert got.guards_intact()
    assert dx.guards_intact()


# A block of the backward pass does several rows: at each number of threads per row, aligned and not.
@pytest.mark.parametrize("kind,dtype,fmt", [("rms", "bf16", "int8"), ("layer", "f16", "e4m3")])
@pytest.mark.parametrize("rows,cols", [(4500, 300), (1500, 601), (600, 2104), (530, 5001), (520, 9000)])
def test_norm_many_rows(abi, kind, dtype, fmt, rows, cols):
    test_norm(abi, kind, dtype, fmt, rows, cols)


def test_norm_wants_only_some_gradients(abi):
    rows, cols = 700, 1031
    rng = np.random.default_rng(2)
    x, dy = activation(rng, rows, cols, "bf16"), activation(rng, rows, cols, "bf16", 0.1)
    codes, scales = _dev_ckpt(*act.save(x, "bf16", "int8"))
    rstd = torch.rand(rows, device="cuda") + 0.5
    md = Mat(rows, cols, "bf16", dy)
    ws = torch.empty(abi.zero_act_norm_workspace_bytes(rows, cols), dtype=torch.uint8, device="cuda")
    out = {}
    for w, b in ((True, True), (True, False), (False, True), (False, False)):
        ws.fill_(0xFF)
        dx, gw, gb = Mat(rows, cols, "bf16"), Mat(1, cols, "bf16"), Mat(1, cols, "bf16")
        abi.zero_act_norm_backward(codes, scales, 1, None, rstd, None, rows, cols, 1, md.t, cols, None, 0, 1.0, "bf16",
                                   dx.t, cols, None, 0, False, gw.t if w else None, gb.t if b else None, ws)
        torch.cuda.synchronize()
        out[w, b] = dx.bits(), gw.bits(), gb.bits()
    ref = out[True, True]
    for (w, b), got in out.items():
        assert np.array_equal(got[0], ref[0])
        assert np.array_equal(got[1], ref[1]) if w else (got[1] == 0x5A5A).all()
        assert np.array_equal(got[2], ref[2]) if b else (got[2] == 0x5A5A).all()


@pytest.mark.parametrize("w,b", [(True, False), (False, True)])
def test_norm_with_weight_or_bias_alone(abi, w, b):
    rows, cols = 6, 777
    rng = np.random.default_rng(4)
    x, vec = activation(rng, rows, cols, "f16"), activation(rng, 1, cols, "f16")
    mx, my, mv = Mat(rows, cols, "f16", x), Mat(rows, cols, "f16"), Mat(1, cols, "f16", vec, off=1)
    codes, scales = _ckpt(abi, rows, cols)
    mean, rstd = torch.zeros(rows, device="cuda"), torch.zeros(rows, device="cuda")
    abi.zero_act_norm_forward(mx.t, cols, None, 0, 0.0, mv.t if w else None, mv.t if b else None, "f16", rows, cols, 2,
                              1e-5, 1, None, 0, my.t, cols, codes, scales, mean, rstd)
    torch.cuda.synchronize()
    v = wide(vec, "f16")
    y, _, _ = act.norm_forward(wide(x, "f16"), v if w else None, v if b else None, "layer", 1e-5)
    close16(my.bits(), *y, "f16", "y")


def test_norm_in_place(abi):
    # the residual stream and its gradient updated in place give the same bits as out of place
    rows, cols = 21, 3000
    rng = np.random.default_rng(1)
    x, br = activation(rng, rows, cols, "bf16"), activation(rng, rows, cols, "bf16", 0.5)
    outs = []
    for inplace in (False, True):
        mx, mb, my = Mat(rows, cols, "bf16", x), Mat(rows, cols, "bf16", br), Mat(rows, cols, "bf16")
        mr = mx if inplace else Mat(rows, cols, "bf16")
        codes, scales = _ckpt(abi, rows, cols)
        rstd = torch.zeros(rows, device="cuda")
        abi.zero_act_norm_forward(mx.t, cols, mb.t, cols, 1.0, None, None, "bf16", rows, cols, 1, 1e-6, 2, mr.t, cols,
                                  my.t, cols, codes, scales, None, rstd)
        md, mdr = Mat(rows, cols, "bf16", br), Mat(rows, cols, "bf16", x)
        dx = mdr if inplace else Mat(rows, cols, "bf16")
        abi.zero_act_norm_backward(codes, scales, 2, None, rstd, None, rows, cols, 1, md.t, cols, mdr.t, cols, 1.0,
                                   "bf16", dx.t, cols, None, 0, False, None, None, None, workspace_bytes=0)
        torch.cuda.synchronize()
        outs.append((mr.bits(), my.bits(), dx.bits()))
    for p, q in zip(*outs):
        assert np.array_equal(p, q)


def test_norm_gradient_against_differences(abi):
    # Exactly representable checkpoints (integers with a block maximum of 127), so the analytic gradient is that
    # of the forward pass; central differences of the oracle's forward pass in float64.
    rng = np.random.default_rng(6)
    rows, cols = 3, 40
    r = rng.integers(-60, 61, (rows, cols)).astype(np.float32)
    r[:, 0] = 127
    bits = rounding.narrow(r, "f16").reshape(rows, cols)
    w = rounding.narrow((1 + 0.1 * rng.standard_normal(cols)).astype(np.float32), "f16")
    dy = activation(rng, rows, cols, "f16")
    mx, my, mw = Mat(rows, cols, "f16", bits), Mat(rows, cols, "f16"), Mat(1, cols, "f16", w[None])
    codes, scales = _ckpt(abi, rows, cols)
    mean, rstd = torch.zeros(rows, device="cuda"), torch.zeros(rows, device="cuda")
    abi.zero_act_norm_forward(mx.t, cols, None, 0, 0.0, mw.t, None, "f16", rows, cols, 2, 1e-5, 1, None, 0, my.t, cols,
                              codes, scales, mean, rstd)
    md, dx = Mat(rows, cols, "f16", dy), Mat(rows, cols, "f16")
    abi.zero_act_norm_backward(codes, scales, 1, mean, rstd, mw.t, rows, cols, 2, md.t, cols, None, 0, 1.0, "f16", dx.t,
                               cols, None, 0, False, None, None, None, workspace_bytes=0)
    torch.cuda.synchronize()
    w64, dy64, r64 = wide(w, "f16"), wide(dy, "f16"), r.astype(np.float64)
    loss = lambda v: (act.norm_forward(v, w64, None, "layer", 1e-5)[0][0] * dy64).sum()
    num = np.zeros_like(r64)
    h = 1e-3
    for i in range(rows):
        for j in range(cols):
            e = np.zeros_like(r64)
            e[i, j] = h
            num[i, j] = (loss(r64 + e) - loss(r64 - e)) / (2 * h)
    # truncation h^2/6 |f'''| with r of size 60 and variance 60^2 is below 1e-9; differences' rounding 1e-12 / h
    (_, err), _, _ = act.norm_backward(r64, mean.cpu().numpy().astype(np.float64), rstd.cpu().numpy().astype(np.float64),
                                       w64, dy64, 0.0, "layer", 1)
    close16(dx.bits(), num, err + 1e-8, "f16", "dx against differences")


def test_empty_calls(abi):
    abi.zero_act_save(0, 5, "f16", 0, 5, 1, 0, 0)
    abi.zero_act_restore(0, 0, 1, 5, 0, 0, 0, "f16")
    abi.zero_act_glu_forward(0, 9, None, 0, "f16", 0, 9, 1, 1, 0, 9, 0, 0, None, None)
    g = Mat(2, 300, "bf16", np.full((2, 300), 0x3F80, np.uint16))
    for accumulate, want in ((False, 0), (True, 0x3F80)):
        abi.zero_act_norm_backward(0, 0, 1, None, 0, None, 0, 300, 1, 0, 300, None, 0, 1.0, "bf16", 0, 300, None, 0,
                                   accumulate, g.t[0], g.t[1], None, workspace_bytes=0)
        torch.cuda.synchronize()
        assert (g.bits() == want).all()
        g.t.fill_(1.0)


@pytest.mark.parametrize("rows,cols", [(2_097_160, 520), (8_388_613, 24)])
def test_norm_of_more_rows_than_one_launch(abi, rows, cols):
    # 2^21 blocks are a launch; the rows around the seam and the last ones equal the same rows alone.
    x = torch.randn(rows, cols, device="cuda").to(torch.bfloat16)
    br = torch.randn(cols, device="cuda").to(torch.bfloat16).expand(rows, cols).contiguous()

    def run(sl):
        xs, bs = x[sl].clone(), br[sl].contiguous()
        n = xs.shape[0]
        y, (codes, scales) = torch.empty_like(xs), _ckpt(abi, n, cols)
        mean, rstd = torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
        abi.zero_act_norm_forward(xs, cols, bs, cols, 1.0, None, None, "bf16", n, cols, 2, 1e-5, 1, xs, cols, y, cols,
                                  codes, scales, mean, rstd)
        torch.cuda.synchronize()
        return (xs, y, codes[:n * ((cols + 15) // 16 * 16)].view(n, -1), scales[:n * -(-cols // 256)].view(n, -1), mean,
                rstd)

    whole = run(slice(0, rows))
    seam = (1 << 21) * (1 if cols > 512 else 4)
    for sl in (slice(seam - 6, min(seam + 6, rows)), slice(rows - 3, rows), slice(0, 5)):
        for a, b in zip(whole, run(sl)):
            assert torch.equal(a[sl], b)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_offsets_past_32_bits(abi, fmt):
    # 2.2e9 elements, 4.4 GB of 16-bit values, 2.2 GB of codes: the last rows equal the same rows saved alone.
    rows, cols = 137_000, 16_128
    _note(f"large {fmt}")
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
    x[:4].normal_()
    x[4:-8] = 1.0
    x[-8:].normal_()
    codes = torch.empty(abi.zero_act_code_bytes(rows, cols), dtype=torch.uint8, device="cuda")
    scales = torch.empty(abi.zero_act_scale_count(rows, cols), device="cuda")
    abi.zero_act_save(x, cols, "bf16", rows, cols, FMT[fmt], codes, scales)
    y = torch.empty_like(x)
    abi.zero_act_restore(codes, scales, FMT[fmt], rows, cols, y, cols, "bf16")
    torch.cuda.synchronize()
    for sl in (slice(0, 4), slice(rows - 8, rows)):
        part = x[sl].contiguous()
        bits = part.view(torch.int16).cpu().numpy().view(np.uint16)
        want = act.restore(*act.save(bits, "bf16", fmt), "bf16", fmt)
        assert np.array_equal(y[sl].contiguous().view(torch.int16).cpu().numpy().view(np.uint16), want)
    mid = y[4:-8]
    assert bool((mid == 1.0).all())
