"""The weight gradient's forms (tile size, input restored first or while staged, split over
the tokens) with earlier gradients to add to, output gradients in wider or misaligned
matrices, and workspaces of any content; and views of more than two dimensions.

Integer inputs make every sum exact in any order.
"""

import numpy as np
import pytest
import torch

from act_cases import activation, close16, wide
from oracle import act, rounding
from test_gpu_act import FMT, FN, TORCH16, Mat, _dev_ckpt, _note, abi  # noqa: F401

pytestmark = pytest.mark.gpu

FORMS = [
    (200, 4100, 4104),     # 256 x 256 tiles, decoded while staged
    (700, 4100, 4101),     # ... restored first
    (4801, 1030, 2056),    # 128 x 128 tiles, restored first, split over the tokens
    (4801, 1030, 700),     # ... decoded while staged
    (40_000, 120, 9),      # one tile, many splits
    (130, 70_000, 5),      # large enough for 256 x 256 tiles, rows too close for their loads
]


def _integer_case(abi, rows, inner, outer, dtype, fmt, pad, off):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(rows + inner)
    half = TORCH16[dtype]
    x = torch.randint(-9, 10, (rows, inner), generator=gen, device="cuda").to(half)
    x[:, ::256] = 127 if fmt == "int8" else 448
    codes = torch.empty(rows, (inner + 15) // 16 * 16, dtype=torch.uint8, device="cuda")
    scales = torch.empty(rows, -(-inner // 256), device="cuda")
    abi.zero_act_save(x, inner, dtype, rows, inner, FMT[fmt], codes, scales)
    assert bool((scales == 1).all())
    dy = Mat(rows, outer, dtype, pad=pad, off=off)
    # what lies between the rows must not count, whatever it is
    dy.buf.view(half).fill_(float("nan"))
    dy.t.copy_(torch.randint(-1, 2, (rows, outer), generator=gen, device="cuda").to(half))
    old_w = torch.randint(-99, 100, (outer, inner), generator=gen, device="cuda").to(half)
    old_b = torch.randint(-99, 100, (outer,), generator=gen, device="cuda").to(half)
    d = dy.t.double()
    return codes, scales, dy, old_w, old_b, d.t().contiguous() @ x.double(), d.sum(0)


@pytest.mark.parametrize("pad,off", [(0, 0), (3, 1), (24, 5)])
@pytest.mark.parametrize("dtype,fmt", [("bf16", "int8"), ("f16", "e4m3")])
@pytest.mark.parametrize("rows,inner,outer", FORMS)
def test_accumulation_and_strides_are_exact(abi, dtype, fmt, rows, inner, outer, pad, off):
    _note(f"weight_grad {dtype} {fmt} {rows} {inner} {outer} pad {pad} off {off}")
    half = TORCH16[dtype]
    codes, scales, dy, old_w, old_b, want_w, want_b = _integer_case(abi, rows, inner, outer, dtype, fmt, pad, off)
    assert float(want_w.abs().max()) + 99 < 2 ** 24
    ws = torch.empty(max(abi.zero_act_weight_grad_workspace_bytes(rows, inner, outer), 16), dtype=torch.uint8,
                     device="cuda").fill_(0xFF)
    for accumulate, bias in ((True, True), (True, False), (False, True)):
        mw, mb = Mat(outer, inner, dtype, off=1), Mat(1, outer, dtype, off=3)
        mw.t.copy_(old_w)
        mb.t.copy_(old_b[None])
        abi.zero_act_weight_grad(dy.t, dy.stride, dtype, codes, scales, FMT[fmt], rows, inner, outer, accumulate,
                                 mw.view.view(-1), mb.view.view(-1) if bias else None, ws)
        torch.cuda.synchronize()
        w = want_w + old_w.double() if accumulate else want_w
        b = (want_b + old_b.double() if accumulate else want_b) if bias else old_b.double()
        assert torch.equal(mw.t, w.float().to(half)) and torch.equal(mb.t[0], b.float().to(half)), (accumulate, bias)
        assert mw.guards_intact() and mb.guards_intact()


# All-zero, all-one and infinite contents, in a workspace of just the size and in one of a longer batch.
FILLS = [(0x00, 0), (0xFF, 0), (0x7F, 1 << 20), (0x80, 1 << 20)]


@pytest.mark.parametrize("rows,inner,outer", [(3000, 200, 150), (700, 4100, 4101), (4801, 1030, 2056)])
def test_the_workspaces_content_does_not_matter(abi, rows, inner, outer):
    rng = np.random.default_rng(9)
    x, dy = activation(rng, rows, inner, "bf16"), activation(rng, rows, outer, "bf16", 0.02)
    codes, scales = _dev_ckpt(*act.save(x, "bf16", "e4m3"))
    d = Mat(rows, outer, "bf16", dy)
    need = abi.zero_act_weight_grad_workspace_bytes(rows, inner, outer)
    assert need > 0
    first = None
    for fill, more in FILLS:
        ws = torch.full((need + more,), fill, dtype=torch.uint8, device="cuda")
        dw, db = Mat(outer, inner, "bf16"), Mat(1, outer, "bf16")
        abi.zero_act_weight_grad(d.t, d.stride, "bf16", codes, scales, 2, rows, inner, outer, False, dw.view.view(-1),
                                 db.view.view(-1), ws)
        torch.cuda.synchronize()
        got = dw.bits(), db.bits()
        assert (ws[need:] == fill).all()
        first = first or got
        assert np.array_equal(got[0], first[0]) and np.array_equal(got[1], first[1]), hex(fill)


@pytest.mark.parametrize("rows,cols", [(1500, 300), (4203, 601), (333, 5001)])
def test_the_norms_workspaces_content_does_not_matter(abi, rows, cols):
    rng = np.random.default_rng(3)
    x, dy = activation(rng, rows, cols, "f16"), activation(rng, rows, cols, "f16", 0.02)
    codes, scales = _dev_ckpt(*act.save(x, "f16", "int8"))
    rstd = torch.rand(rows, device="cuda") + 0.5
    mean = torch.rand(rows, device="cuda") - 0.5
    d = Mat(rows, cols, "f16", dy)
    need = abi.zero_act_norm_workspace_bytes(rows, cols)
    first = None
    for fill, more in FILLS:
        ws = torch.full((need + more,), fill, dtype=torch.uint8, device="cuda")
        dx, gw, gb = Mat(rows, cols, "f16"), Mat(1, cols, "f16"), Mat(1, cols, "f16")
        abi.zero_act_norm_backward(codes, scales, 1, mean, rstd, None, rows, cols, 2, d.t, cols, None, 0, 1.0, "f16", dx.t,
                                   cols, None, 0, False, gw.t, gb.t, ws)
        torch.cuda.synchronize()
        got = dx.bits(), gw.bits(), gb.bits()
        assert (ws[need:] == fill).all()
        first = first or got
        assert all(np.array_equal(p, q) for p, q in zip(got, first)), hex(fill)


def test_views_of_batches_and_heads(abi):
    # [batch, sequence, columns] and [tokens, heads, size] views, in and out, against the matrices they are.
    B, S, H, D = 3, 50, 6, 40
    rows, cols = B * S, H * D
    wide = torch.randn(rows, 3 * cols, device="cuda").to(torch.bfloat16)
    flat = wide[:, cols:2 * cols]
    out = {}
    for name, x in (("matrix", flat), ("heads", flat.view(rows, H, D)),
                    ("batch", wide.view(B, S, 3 * cols)[:, :, cols:2 * cols])):
        codes = torch.empty(rows, cols, dtype=torch.uint8, device="cuda")
        scales = torch.empty(rows, 1, device="cuda")
        abi.zero_act_save(x, 3 * cols, "bf16", rows, cols, 1, codes, scales)
        y = torch.zeros(rows, 3 * cols, dtype=torch.bfloat16, device="cuda")
        v = {"matrix": y[:, :cols], "heads": y[:, :cols].view(rows, H, D),
             "batch": y.view(B, S, 3 * cols)[:, :, :cols]}[name]
        abi.zero_act_restore(codes, scales, 1, rows, cols, v, 3 * cols, "bf16")
        torch.cuda.synchronize()
        assert not y[:, cols:].any()
        out[name] = codes, scales, y
    for name in ("heads", "batch"):
        assert all(torch.equal(p, q) for p, q in zip(out[name], out["matrix"])), name
    codes, scales, y = out["matrix"]
    with pytest.raises(ValueError, match="apart"):           # [sequence, batch, columns]: another order
        abi.zero_act_save(flat.contiguous().view(B, S, cols).transpose(0, 1), cols, "bf16", rows, cols, 1, codes, scales)
    with pytest.raises(ValueError, match="torch.float16 values"):
        abi.zero_act_save(flat.half(), cols, "bf16", rows, cols, 1, codes, scales)
    with pytest.raises(ValueError, match="torch.float64 values"):
        abi.zero_act_restore(codes, scales.double(), 1, rows, cols, y, 3 * cols, "bf16")


@pytest.mark.parametrize("fn", ["silu", "gelu", "gelu_tanh"])
def test_glu_gradients_against_differences(abi, fn):
    # Gates and ups that the checkpoint holds exactly (multiples of 1/32 with a block maximum of 127/32), so the
    # gradient is that of the forward pass; central differences of the oracle's forward pass in float64.
    rng = np.random.default_rng(8)
    rows, cols, step = 5, 60, 2.0 ** -5
    g, u = (rng.integers(-126, 127, (rows, cols)) * step for _ in range(2))
    g[:, 0] = u[:, 0] = 127 * step
    bits = lambda v: rounding.narrow(v.astype(np.float32), "f16").reshape(rows, cols)
    dh = activation(rng, rows, cols, "f16")
    mg, mu, md = Mat(rows, cols, "f16", bits(g)), Mat(rows, cols, "f16", bits(u)), Mat(rows, cols, "f16", dh)
    h, dg, du = Mat(rows, cols, "f16"), Mat(rows, cols, "f16"), Mat(rows, cols, "f16")
    (gc, gs), (uc, us) = [(torch.empty(rows, 64, dtype=torch.uint8, device="cuda"), torch.empty(rows, 1, device="cuda"))
                          for _ in range(2)]
    abi.zero_act_glu_forward(mg.t, cols, mu.t, cols, "f16", rows, cols, FN[fn], 1, h.t, cols, gc, gs, uc, us)
    abi.zero_act_glu_backward(gc, gs, uc, us, 1, rows, cols, FN[fn], md.t, cols, "f16", dg.t, cols, du.t, cols)
    torch.cuda.synchronize()
    assert bool((gs == step).all()) and bool((us == step).all())
    d64, e = wide(dh, "f16"), 1e-4
    f = lambda a, b: act.glu_forward(a, b, fn)[0] * d64          # element by element: differences of all at once
    (_, ge), (_, ue), _ = act.glu_backward(g, u, d64, fn)
    # truncation: e^2 / 6 |f'''| |u dh|, |f'''| below 1 for all three, |u| <= 4, |dh| < 64; rounding: a few ulps of
    # |h dh| over e
    slack = e * e / 6 * 4 * 64 + 2.0 ** -50 * 16 * 64 / e
    close16(dg.bits(), (f(g + e, u) - f(g - e, u)) / (2 * e), ge + slack, "f16", "dgate")
    close16(du.bits(), (f(g, u + e) - f(g, u - e)) / (2 * e), ue + slack, "f16", "dup")


def test_weight_gradient_against_differences(abi):
    # The loss sum(dy (x W^T + b)) is linear in W and b: differences of any width are its gradient.
    rng = np.random.default_rng(4)
    rows, inner, outer = 9, 20, 7
    x = rng.integers(-60, 61, (rows, inner)).astype(np.float64)
    x[:, 0] = 127
    xb = rounding.narrow(x.astype(np.float32), "bf16").reshape(rows, inner)
    dy = activation(rng, rows, outer, "bf16")
    codes, scales = _dev_ckpt(*act.save(xb, "bf16", "int8"))
    md, mw, mb = Mat(rows, outer, "bf16", dy), Mat(outer, inner, "bf16"), Mat(1, outer, "bf16")
    abi.zero_act_weight_grad(md.t, outer, "bf16", codes, scales, 1, rows, inner, outer, False, mw.t, mb.t, None,
                             workspace_bytes=0)
    torch.cuda.synchronize()
    d64, w, b = wide(dy, "bf16"), rng.standard_normal((outer, inner)), rng.standard_normal(outer)
    loss = lambda w, b: (d64 * (x @ w.T + b)).sum()
    num, numb = np.zeros_like(w), np.zeros_like(b)
    for o in range(outer):
        for i in range(inner):
            p = np.zeros_like(w)
            p[o, i] = 1.0
            num[o, i] = (loss(w + p, b) - loss(w - p, b)) / 2
        q = np.zeros_like(b)
        q[o] = 1.0
        numb[o] = (loss(w, b + q) - loss(w, b - q)) / 2
    (_, we), (_, be) = act.weight_grad(d64, x)
    # float64 losses of sums of 9 * 7 * 20 products of up to 127 * 8 * 4
    slack = 2.0 ** -52 * 9 * 7 * 20 * 127 * 8 * 4
    close16(mw.bits(), num, we + slack, "bf16", "dweight")
    close16(mb.bits()[0], numb, be + slack, "bf16", "dbias")
