"""The norm's backward pass with more partial sums than one pass of their fold takes
(over 256), and offsets past 2^31 elements in the norm and the gated activation.

Integer inputs make every sum over rows exact in any order, so a row that is dropped,
doubled or folded into another column shows.
"""

import numpy as np
import pytest
import torch

from act_cases import close16, wide
from oracle import act, rounding
from test_gpu_act import FMT, FN, KIND, TORCH16, Mat, _note, abi  # noqa: F401

pytestmark = pytest.mark.gpu

# Blocks of 4 wave rows, of 256 and of 512 threads: 826, 841 and 421 partial sums (chunks of 5 passes each, the last
# one short), 1024 and 512 in full, and the last sizes below where the larger grids begin.
SHAPES = [(16501, 300), (4203, 601), (2101, 2104), (16384, 64), (4096, 2048), (2048, 2049), (4095, 601), (2047, 4096)]


def _integers(gen, rows, cols, fmt, dtype):
    """Integers whose checkpoint has scale 1 (codes, scales) and their values."""
    v = torch.randint(-9, 10, (rows, cols), generator=gen, device="cuda")
    v[:, ::256] = 127 if fmt == "int8" else 448
    return v.to(TORCH16[dtype])


def _saved(abi, x, fmt, dtype):
    rows, cols = x.shape
    codes = torch.empty(rows, (cols + 15) // 16 * 16, dtype=torch.uint8, device="cuda")
    scales = torch.empty(rows, -(-cols // 256), device="cuda")
    abi.zero_act_save(x, cols, dtype, rows, cols, FMT[fmt], codes, scales)
    assert bool((scales == 1).all())
    return codes, scales


@pytest.mark.parametrize("kind,dtype,fmt", [("rms", "bf16", "int8"), ("layer", "f16", "e4m3")])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_many_partial_sums(abi, kind, dtype, fmt, rows, cols):
    _note(f"norm backward {kind} {dtype} {fmt} {rows}x{cols}")
    gen = torch.Generator(device="cuda")
    gen.manual_seed(rows + cols)
    half = TORCH16[dtype]
    codes, scales = _saved(abi, _integers(gen, rows, cols, fmt, dtype), fmt, dtype)
    r = codes[:, :cols].view(torch.int8).double() if fmt == "int8" else codes[:, :cols].view(torch.float8_e4m3fn).double()
    # n = (r - mean) rstd is exact: small integers and a power of two
    mean = torch.randint(-3, 4, (rows,), generator=gen, device="cuda").float() if kind == "layer" else None
    rstd = torch.full((rows,), 0.25, device="cuda")
    n = (r if mean is None else r - mean.double()[:, None]) * 0.25
    dy = torch.randint(-1, 2, (rows, cols), generator=gen, device="cuda").to(half)
    md, dx = Mat(rows, cols, dtype, pad=3, off=1), Mat(rows, cols, dtype, pad=1)
    md.t.copy_(dy)
    sums = (dy.double() * n).sum(0), dy.double().sum(0)
    old = [torch.randint(-99, 100, (cols,), generator=gen, device="cuda").to(half) for _ in range(2)]
    assert float((dy.double() * n).abs().sum(0).max()) * 4 < 2 ** 24          # in quarters
    ws = torch.empty(abi.zero_act_norm_workspace_bytes(rows, cols), dtype=torch.uint8, device="cuda")
    first = None
    for want_w, want_b, accumulate in ((1, 1, 0), (1, 0, 0), (0, 1, 0), (1, 1, 1), (0, 1, 1)):
        ws.fill_(0xFF)
        out = [Mat(1, cols, dtype, off=1), Mat(1, cols, dtype, off=3)]
        for m, o in zip(out, old):
            m.t.copy_(o[None])
        abi.zero_act_norm_backward(codes, scales, FMT[fmt], mean, rstd, None, rows, cols, KIND[kind], md.t, md.stride,
                                   None, 0, 1.0, dtype, dx.t, dx.stride, None, 0, bool(accumulate),
                                   out[0].t if want_w else None, out[1].t if want_b else None, ws)
        torch.cuda.synchronize()
        for k, (m, s, wanted) in enumerate(zip(out, sums, (want_w, want_b))):
            exact = s + old[k].double() if accumulate else s
            want = exact.float().to(half) if wanted else old[k]
            assert torch.equal(m.t[0], want), (k, want_w, want_b, accumulate, int((m.t[0] != want).sum()))
            assert m.guards_intact()
        bits = dx.bits()
        assert dx.guards_intact() and (first is None or np.array_equal(bits, first))
        first = bits
    a, _, _ = act.norm_backward(r.cpu().numpy(), None if mean is None else mean.cpu().numpy().astype(np.float64),
                                rstd.cpu().numpy().astype(np.float64), None, dy.double().cpu().numpy(), 0.0, kind, 1)
    close16(first, *a, dtype, "dx")


def test_norm_offsets_past_32_bits(abi):
    # 2.2e9 elements, 2.2 GB of codes: the last rows equal the same rows alone, forward and backward.
    rows, cols, last = 137_000, 16_128, 5
    _note("norm large")
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    half = torch.bfloat16
    x = torch.ones(rows, cols, dtype=half, device="cuda")
    x[-last:] = torch.randint(-9, 10, (last, cols), generator=gen, device="cuda").to(half)
    br = torch.ones(rows, cols, dtype=half, device="cuda")
    dy = torch.zeros(rows, cols, dtype=half, device="cuda")
    dy[-last:] = torch.randint(-2, 3, (last, cols), generator=gen, device="cuda").to(half)

    def run(x, br, dy):
        n = x.shape[0]
        e = lambda *s, dt=half: torch.empty(*s, dtype=dt, device="cuda")
        res, y, dx, db = e(n, cols), e(n, cols), e(n, cols), e(n, cols)
        codes, scales = e(n, cols, dt=torch.uint8), e(n, cols // 256, dt=torch.float32)
        mean, rstd = e(n, dt=torch.float32), e(n, dt=torch.float32)
        abi.zero_act_norm_forward(x, cols, br, cols, 0.5, None, None, "bf16", n, cols, 2, 1e-5, 1, res, cols, y, cols,
                                  codes, scales, mean, rstd)
        gb = e(cols)
        ws = e(abi.zero_act_norm_workspace_bytes(n, cols), dt=torch.uint8)
        abi.zero_act_norm_backward(codes, scales, 1, mean, rstd, None, n, cols, 2, dy, cols, None, 0, 0.5, "bf16", dx,
                                   cols, db, cols, False, None, gb, ws)
        torch.cuda.synchronize()
        return [t[-last:].clone() for t in (res, y, codes, scales, mean, rstd, dx, db)] + [gb]

    whole = run(x, br, dy)
    alone = run(x[-last:].clone(), br[-last:].clone(), dy[-last:].clone())
    for k, (a, b) in enumerate(zip(whole, alone)):
        assert torch.equal(a, b), k
    assert torch.equal(whole[-1], dy[-last:].float().sum(0).to(half))


def test_glu_offsets_past_32_bits(abi):
    # 1.1e9 elements of gate and up each in one matrix of 2.2e9, and as many again in its gradient.
    rows, cols, last = 137_000, 8_064, 5
    _note("glu large")
    half = torch.bfloat16
    x = torch.ones(rows, 2 * cols, dtype=half, device="cuda")
    dh = torch.ones(rows, cols, dtype=half, device="cuda")
    for t in (x, dh):
        t[-last:].normal_()

    def run(x, dh):
        n, w = x.shape
        w //= 2
        e = lambda *s, dt=half: torch.empty(*s, dtype=dt, device="cuda")
        h, dx, again = e(n, w), e(n, 2 * w), e(n, w)
        ck = [(e(n, w, dt=torch.uint8), e(n, -(-w // 256), dt=torch.float32)) for _ in range(2)]
        abi.zero_act_glu_forward(x, 2 * w, x[:, w:], 2 * w, "bf16", n, w, FN["silu"], 2, h, w, *ck[0], *ck[1])
        abi.zero_act_glu_backward(*ck[0], *ck[1], 2, n, w, FN["silu"], dh, w, "bf16", dx, 2 * w, dx[:, w:], 2 * w, again, w)
        torch.cuda.synchronize()
        return [t[-last:].clone() for t in (h, dx, again, *ck[0], *ck[1])]

    for k, (a, b) in enumerate(zip(run(x, dh), run(x[-last:].clone(), dh[-last:].clone()))):
        assert torch.equal(a, b), k
    del x, dh
    # an ungated one whose codes pass 2^31 bytes
    rows, cols = 137_000, 16_128
    x = torch.ones(rows, cols, dtype=half, device="cuda")
    x[-last:].normal_()

    def plain(x):
        n, w = x.shape
        e = lambda *s, dt=half: torch.empty(*s, dtype=dt, device="cuda")
        h, dx, codes, scales = e(n, w), e(n, w), e(n, w, dt=torch.uint8), e(n, w // 256, dt=torch.float32)
        abi.zero_act_glu_forward(x, w, None, 0, "bf16", n, w, FN["gelu"], 1, h, w, codes, scales, None, None)
        abi.zero_act_glu_backward(codes, scales, None, None, 1, n, w, FN["gelu"], x, w, "bf16", dx, w, None, 0)
        torch.cuda.synchronize()
        return [t[-last:].clone() for t in (h, dx, codes, scales)]

    for k, (a, b) in enumerate(zip(plain(x), plain(x[-last:].clone()))):
        assert torch.equal(a, b), k


@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_a_batch_without_rows(abi, kind):
    # Tensors without elements have no address; the parameter gradients are written (zero) or kept.
    e = lambda *s, dt=torch.bfloat16: torch.empty(*s, dtype=dt, device="cuda")
    cols, f32 = 300, torch.float32
    mean = e(0, dt=f32) if kind == "layer" else None
    codes, scales = e(0, dt=torch.uint8), e(0, dt=f32)
    abi.zero_act_norm_forward(e(0, cols), cols, e(0, cols), cols, 1.0, None, None, "bf16", 0, cols, KIND[kind], 1e-5, 1,
                              e(0, cols), cols, e(0, cols), cols, codes, scales, mean, e(0, dt=f32))
    for accumulate, want in ((True, 1.0), (False, 0.0)):
        dw, db = torch.ones(cols, dtype=torch.bfloat16, device="cuda"), torch.ones(cols, dtype=torch.bfloat16, device="cuda")
        abi.zero_act_norm_backward(codes, scales, 1, mean, e(0, dt=f32), None, 0, cols, KIND[kind], e(0, cols), cols,
                                   e(0, cols), cols, 1.0, "bf16", e(0, cols), cols, e(0, cols), cols, accumulate, dw, db,
                                   e(abi.zero_act_norm_workspace_bytes(0, cols), dt=torch.uint8))
        torch.cuda.synchronize()
        assert bool((dw == want).all()) and bool((db == want).all())
