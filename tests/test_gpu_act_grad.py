"""GPU parity of the weight gradient taken from an 8-bit activation checkpoint,
and the checkpoint operators run together with the sharded step."""

import numpy as np
import pytest
import torch

from act_cases import activation, close16, wide
from oracle import act, rounding
from test_gpu_act import FMT, Mat, _dev_ckpt, _note, abi  # noqa: F401

pytestmark = pytest.mark.gpu

TORCH16 = {"f16": torch.float16, "bf16": torch.bfloat16}


def _run(abi, dtype, fmt, x, dy, off=0, old=None, bias=True, pad=0):
    """dW (and db) on the device and the oracle's; old: (dW0, db0) patterns to accumulate onto."""
    rows, inner = x.shape
    outer = dy.shape[1]
    codes, scales = act.save(x, dtype, fmt)
    dc, ds = _dev_ckpt(codes, scales)
    md = Mat(rows, outer, dtype, dy, pad=pad, off=off)
    mw = Mat(outer, inner, dtype, None if old is None else old[0], off=off)
    mb = Mat(1, outer, dtype, None if old is None else old[1][None], off=off) if bias else None
    ws = torch.empty(max(abi.zero_act_weight_grad_workspace_bytes(rows, inner, outer), 16), dtype=torch.uint8,
                     device="cuda").fill_(0xFF)
    abi.zero_act_weight_grad(md.t, md.stride, dtype, dc, ds, FMT[fmt], rows, inner, outer, old is not None,
                             mw.view.view(-1), None if mb is None else mb.view.view(-1), ws)
    torch.cuda.synchronize()
    back = wide(act.restore(codes, scales, dtype, fmt), dtype)
    w, b = act.weight_grad(wide(dy, dtype), back)
    assert mw.guards_intact() and (mb is None or mb.guards_intact())
    return mw, mb, w, b


def _check(mw, mb, w, b, dtype, old=None):
    for m, (v, e), k in ((mw, w, 0), (mb, b, 1)):
        if m is None:
            continue
        o = 0.0 if old is None else wide(old[k], dtype)
        got = m.bits() if k == 0 else m.bits()[0]
        close16(got, v + o, e + 2.0 ** -24 * np.abs(v + o), dtype, ("dweight", "dbias")[k])


SIZES = [(1, 1, 1), (1, 300, 5), (2, 16, 40), (7, 129, 65), (33, 256, 257), (64, 128, 128), (100, 511, 130),
         (257, 260, 300), (600, 64, 1000), (1000, 1000, 48), (2500, 100, 90), (5000, 257, 33)]


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("rows,inner,outer", SIZES)
def test_weight_grad(abi, fmt, dtype, rows, inner, outer):
    _note(f"weight_grad {fmt} {dtype} {rows} {inner} {outer}")
    rng = np.random.default_rng(rows + 3 * inner + 7 * outer)
    x, dy = activation(rng, rows, inner, dtype), activation(rng, rows, outer, dtype, 0.02)
    _check(*_run(abi, dtype, fmt, x, dy), dtype)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("rows,inner,outer", [(3, 70, 9), (130, 300, 200), (3000, 130, 129)])
def test_accumulate_at_an_odd_offset(abi, dtype, rows, inner, outer):
    _note(f"weight_grad accumulate {dtype} {rows} {inner} {outer}")
    rng = np.random.default_rng(rows)
    x, dy = activation(rng, rows, inner, dtype), activation(rng, rows, outer, dtype, 0.02)
    old = activation(rng, outer, inner, dtype, 0.5), activation(rng, 1, outer, dtype, 0.5)[0]
    _check(*_run(abi, dtype, "int8", x, dy, off=3, old=old, pad=1), dtype, old)
    _check(*_run(abi, dtype, "int8", x, dy, off=1, old=old, bias=False), dtype, old)


def test_integers_are_exact(abi):
    # Sums of integer products below 2^24 are exact in fp32 in any order, so the result is the rounded integer:
    # any dropped, doubled or misplaced token, row or column shows.
    for rows, inner, outer in ((1, 515, 259), (129, 258, 514), (4097, 260, 130)):
        rng = np.random.default_rng(rows)
        x = rng.integers(-9, 10, (rows, inner)).astype(np.float32)
        x[:, ::256] = 127                               # scale 1: restored exactly
        dy = rng.integers(-3, 4, (rows, outer)).astype(np.float32)
        xb = rounding.narrow(x, "bf16").reshape(x.shape)
        db = rounding.narrow(dy, "bf16").reshape(dy.shape)
        mw, mb, _, _ = _run(abi, "bf16", "int8", xb, db)
        want = dy.astype(np.float64).T @ x.astype(np.float64)
        assert np.abs(want).max() < 2 ** 24
        assert np.array_equal(mw.bits(), rounding.narrow(want.astype(np.float32), "bf16").reshape(want.shape))
        assert np.array_equal(mb.bits()[0], rounding.narrow(dy.sum(0).astype(np.float32), "bf16"))


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("rows,inner,outer", [
    (200, 4100, 4104),     # 256 x 256 tiles, decoded while staged
    (700, 4100, 4101),     # ... restored first; rows of odd length
    (4801, 1030, 2056),    # 128 x 128 tiles, restored first, split over the tokens
    (130, 520, 70_000),    # one row of input tiles
    (40_000, 120, 9),      # one tile, many splits, fewer than a quarter of it used
    (130, 70_000, 5),      # large enough for 256 x 256 tiles, rows too close for their loads
])
def test_large_shapes_are_exact(abi, dtype, fmt, rows, inner, outer):
    # Integers as above (E4M3 holds those up to 16 with a block maximum of 448), checked in fp64 on the GPU.
    _note(f"weight_grad exact {dtype} {fmt} {rows} {inner} {outer}")
    gen = torch.Generator(device="cuda")
    gen.manual_seed(rows)
    half = TORCH16[dtype]
    x = torch.randint(-9, 10, (rows, inner), generator=gen, device="cuda").to(half)
    x[:, ::256] = 127 if fmt == "int8" else 448
    dy = torch.randint(-1, 2, (rows, outer), generator=gen, device="cuda").to(half)
    codes = torch.empty(rows, (inner + 15) // 16 * 16, dtype=torch.uint8, device="cuda")
    scales = torch.empty(rows, -(-inner // 256), device="cuda")
    abi.zero_act_save(x, inner, dtype, rows, inner, FMT[fmt], codes, scales)
    mw, mb = Mat(outer, inner, dtype, off=1), Mat(1, outer, dtype, off=3)
    ws = torch.empty(max(abi.zero_act_weight_grad_workspace_bytes(rows, inner, outer), 16), dtype=torch.uint8,
                     device="cuda").fill_(0xFF)
    abi.zero_act_weight_grad(dy, outer, dtype, codes, scales, FMT[fmt], rows, inner, outer, False, mw.view.view(-1),
                             mb.view.view(-1), ws)
    want = dy.double().t().contiguous() @ x.double()
    torch.cuda.synchronize()
    assert bool((scales == 1).all()) and float(want.abs().max()) < 2 ** 24
    assert torch.equal(mw.t, want.float().to(half)) and torch.equal(mb.t[0], dy.double().sum(0).float().to(half))
    assert mw.guards_intact() and mb.guards_intact()


def test_rows_far_apart(abi):
    # A stride past the 24 bits of the unchecked loads' offsets.
    rows, inner, outer, stride = 130, 40, 24, (1 << 24) + 8
    big = torch.zeros((rows - 1) * stride + outer, dtype=torch.bfloat16, device="cuda")
    dy = torch.randint(-3, 4, (rows, outer), device="cuda").to(torch.bfloat16)
    view = big.as_strided((rows, outer), (stride, 1))
    view.copy_(dy)
    codes = torch.randint(-127, 128, (rows, 48), dtype=torch.int8, device="cuda").view(torch.uint8)
    scales = torch.ones(rows, 1, device="cuda")
    dw = torch.empty(outer, inner, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(max(abi.zero_act_weight_grad_workspace_bytes(rows, inner, outer), 16), dtype=torch.uint8, device="cuda")
    abi.zero_act_weight_grad(view, stride, "bf16", codes, scales, 1, rows, inner, outer, False, dw, None, ws)
    want = dy.double().t().contiguous() @ codes.view(torch.int8)[:, :inner].double()
    torch.cuda.synchronize()
    assert torch.equal(dw, want.float().to(torch.bfloat16))


def test_narrow_gradients_of_many_tokens(abi):
    # Fewer output columns than an oct, rows closer than an oct: every load is checked.
    for outer in (1, 3, 7, 8, 9):
        rng = np.random.default_rng(outer)
        x, dy = activation(rng, 333, 300, "f16"), activation(rng, 333, outer, "f16", 0.1)
        _check(*_run(abi, "f16", "int8", x, dy), "f16")


def test_non_finite_values_reach_the_gradient(abi):
    rng = np.random.default_rng(3)
    x, dy = activation(rng, 300, 600, "bf16"), activation(rng, 300, 70, "bf16")
    x[123, 300] = 0x7F80
    mw, mb, _, _ = _run(abi, "bf16", "int8", x, dy)
    nan = np.isnan(wide(mw.bits(), "bf16"))
    assert nan[:, 256:512].all() and not nan[:, :256].any() and not nan[:, 512:].any()
    assert np.isfinite(wide(mb.bits(), "bf16")).all()
    x[123, 300] = 0
    dy[299, 11] = 0x7FC0
    mw, mb, _, _ = _run(abi, "bf16", "int8", x, dy)
    nan = np.isnan(wide(mw.bits(), "bf16"))
    assert nan[11].all() and not np.delete(nan, 11, 0).any()
    assert np.isnan(wide(mb.bits(), "bf16"))[0, 11] and np.isnan(wide(mb.bits(), "bf16")).sum() == 1


def test_subnormals_count(abi):
    # fp16 subnormals in the gradient and in the restored activation are multiplied, not flushed.
    dy = np.full((40, 64), 0x0001, np.uint16)                  # 2^-24
    x = np.full((40, 256), 0x0003, np.uint16)
    x[:, 0] = 0x6400                                           # 1024
    mw, _, _, _ = _run(abi, "f16", "int8", x, dy)
    got = wide(mw.bits(), "f16")
    assert np.array_equal(got[:, 0], np.full(64, 40 * 1024 * 2.0 ** -24))
    big = np.full((40, 64), 0x6400, np.uint16)
    tiny = np.full((40, 256), 0x007F, np.uint16)               # 127 * 2^-24: scale 2^-24, restored exactly
    mw, _, _, _ = _run(abi, "f16", "int8", tiny, big)
    assert np.array_equal(wide(mw.bits(), "f16"), np.full((64, 256), 40 * 1024 * 127 * 2.0 ** -24))
    # the same in bf16: 2^-133 times 2^100
    dy = np.full((40, 64), 0x0001, np.uint16)
    x = np.full((40, 256), 0x7180, np.uint16)                  # 2^100
    mw, _, _, _ = _run(abi, "bf16", "int8", x, dy)
    got = wide(mw.bits(), "bf16")
    assert np.all(np.abs(got / (40 * 2.0 ** -33) - 1) <= 2.0 ** -8), got[0, :3]


def test_no_rows_no_columns(abi):
    for accumulate, want in ((False, 0), (True, 0x3F80)):
        m = Mat(5, 7, "bf16", np.full((5, 7), 0x3F80, np.uint16))
        b = Mat(1, 5, "bf16", np.full((1, 5), 0x3F80, np.uint16))
        abi.zero_act_weight_grad(0, 5, "bf16", 0, 0, 1, 0, 7, 5, accumulate, m.view.view(-1), b.view.view(-1), None,
                                 workspace_bytes=0)
        torch.cuda.synchronize()
        assert (m.bits() == want).all() and (b.bits() == want).all()
    # no input columns: only the bias gradient is left
    for rows in (9, 256):
        dy = Mat(rows, 5, "bf16", np.full((rows, 5), 0x3F80, np.uint16))
        ws = torch.empty(max(abi.zero_act_weight_grad_workspace_bytes(rows, 0, 5), 16), dtype=torch.uint8, device="cuda")
        abi.zero_act_weight_grad(dy.t, 5, "bf16", 0, 0, 1, rows, 0, 5, False, 0, b.view.view(-1), ws)
        torch.cuda.synchronize()
        assert (wide(b.bits(), "bf16") == rows).all()
    abi.zero_act_weight_grad(0, 0, "bf16", 0, 0, 1, 9, 7, 0, False, 0, None, None, workspace_bytes=0)
    many = Mat(130, 70_001, "bf16", np.full((130, 70_001), 0x3F80, np.uint16))
    b = Mat(1, 70_001, "bf16")
    abi.zero_act_weight_grad(many.t, 70_001, "bf16", 0, 0, 1, 130, 0, 70_001, False, 0, b.view.view(-1), None,
                             workspace_bytes=0)
    torch.cuda.synchronize()
    assert (wide(b.bits(), "bf16") == 130).all() and b.guards_intact()


def test_repeatable_and_independent_of_the_workspaces_content(abi):
    rng = np.random.default_rng(9)
    x, dy = activation(rng, 3000, 200, "f16"), activation(rng, 3000, 150, "f16", 0.02)
    a = _run(abi, "f16", "e4m3", x, dy)
    b = _run(abi, "f16", "e4m3", x, dy)
    assert np.array_equal(a[0].bits(), b[0].bits()) and np.array_equal(a[1].bits(), b[1].bits())


def test_offsets_past_32_bits(abi):
    # 2.2e9 gradient values: the tokens that are not zero lie in the last 100 rows.
    rows, outer, inner = 275_000, 8000, 16
    dy = torch.zeros(rows, outer, dtype=torch.bfloat16, device="cuda")
    tail = torch.randint(-3, 4, (100, outer), device="cuda").to(torch.bfloat16)
    dy[-100:] = tail
    codes = torch.randint(-127, 128, (rows, inner), dtype=torch.int8, device="cuda").view(torch.uint8)
    scales = torch.ones(rows, 1, device="cuda")
    dw = torch.empty(outer, inner, dtype=torch.bfloat16, device="cuda")
    db = torch.empty(outer, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(max(abi.zero_act_weight_grad_workspace_bytes(rows, inner, outer), 16), dtype=torch.uint8, device="cuda")
    abi.zero_act_weight_grad(dy, outer, "bf16", codes, scales, 1, rows, inner, outer, False, dw, db, ws)
    want = tail.double().t().contiguous() @ codes[-100:].view(torch.int8).double()      # exact integers
    torch.cuda.synchronize()
    assert torch.equal(dw, want.float().to(torch.bfloat16)) and torch.equal(db, tail.float().sum(0).to(torch.bfloat16))


# ---------------------------------------------------------------------------
# Together
# ---------------------------------------------------------------------------

class Block:
    """One pre-norm gated MLP block trained from 8-bit checkpoints, its gradients in the rank's flat local gradient.

    forward: res = x + alpha branch; y = norm(res) w + b; [g | u] = y W1^T; h = silu(g) u; o = h W2^T
    backward from the checkpoints of res, y, g, u and h; then the sharded step's reduce, norm and AdamW.
    """

    T, H, F = 1100, 264, 520

    def __init__(self, abi, seed):
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)
        T, H, F = self.T, self.H, self.F
        self.abi = abi
        half = torch.bfloat16
        rnd = lambda *s, std=1.0: (torch.randn(*s, generator=gen, device="cuda") * std).to(half)
        self.sizes = [H, H, 2 * F * H, 2 * F, H * F]            # norm weight, norm bias, W1, b1, W2
        self.psi = sum(self.sizes)
        self.master = torch.randn(self.psi, generator=gen, device="cuda") * 0.05
        self.master[:H] = 1.0
        self.param = self.master.to(half)
        self.m, self.v = torch.zeros_like(self.master), torch.zeros_like(self.master)
        self.grad = torch.zeros(self.psi, dtype=half, device="cuda")
        self.peer = rnd(self.psi, std=1e-3)                     # the other rank's local gradient
        self.reduced = torch.zeros_like(self.grad)
        self.x, self.branch, self.do = rnd(T, H), rnd(T, H, std=0.5), rnd(T, H, std=0.01)
        e = lambda *s, dt=half: torch.empty(*s, dtype=dt, device="cuda")
        self.res, self.y, self.h, self.gu = e(T, H), e(T, H), e(T, F), e(T, 2 * F)
        self.dgu, self.dx, self.dbranch = e(T, 2 * F), e(T, H), e(T, H)
        ck = lambda c: (e(abi.zero_act_code_bytes(T, c), dt=torch.uint8), e(abi.zero_act_scale_count(T, c), dt=torch.float32))
        self.c_res, self.c_y, self.c_g, self.c_u, self.c_h = ck(H), ck(H), ck(F), ck(F), ck(F)
        self.mean, self.rstd = e(T, dt=torch.float32), e(T, dt=torch.float32)
        n = max(abi.zero_act_norm_workspace_bytes(T, H), abi.zero_act_weight_grad_workspace_bytes(T, H, 2 * F),
                abi.zero_act_weight_grad_workspace_bytes(T, F, H), 16)
        self.ws = e(n, dt=torch.uint8)
        self.step_ws = e(abi.zero_workspace_bytes(self.psi, 1), dt=torch.uint8)
        self.flag = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.norm = torch.zeros(1, dtype=torch.float64, device="cuda")
        self.coef = torch.zeros(1, device="cuda")
        self.hp = abi.adam_hparams(1e-3, 0.9, 0.95, 1e-8, 0.1, 1.0, 1)

    def parts(self, flat):
        return torch.split(flat, self.sizes)

    def step(self):
        a, T, H, F = self.abi, self.T, self.H, self.F
        w, b, w1, b1, w2 = self.parts(self.param)
        gw, gb, gw1, gb1, gw2 = self.parts(self.grad)
        w1, w2 = w1.view(2 * F, H), w2.view(H, F)
        a.zero_act_norm_forward(self.x, H, self.branch, H, 0.5, w, b, "bf16", T, H, 2, 1e-5, 1, self.res, H, self.y, H,
                                *self.c_res, self.mean, self.rstd)
        a.zero_act_save(self.y, H, "bf16", T, H, 1, *self.c_y)
        torch.addmm(b1, self.y, w1.t(), out=self.gu)
        a.zero_act_glu_forward(self.gu, 2 * F, self.gu[:, F:], 2 * F, "bf16", T, F, 1, 1, self.h, F, *self.c_g, *self.c_u)
        a.zero_act_save(self.h, F, "bf16", T, F, 2, *self.c_h)
        # backward
        dh = self.do @ w2
        a.zero_act_weight_grad(self.do, H, "bf16", *self.c_h, 2, T, F, H, False, gw2, None, self.ws)
        a.zero_act_glu_backward(*self.c_g, *self.c_u, 1, T, F, 1, dh, F, "bf16", self.dgu, 2 * F, self.dgu[:, F:], 2 * F)
        a.zero_act_weight_grad(self.dgu, 2 * F, "bf16", *self.c_y, 1, T, H, 2 * F, False, gw1, gb1, self.ws)
        dy = self.dgu @ w1
        a.zero_act_norm_backward(*self.c_res, 1, self.mean, self.rstd, w, T, H, 2, dy, H, self.do, H, 0.5, "bf16",
                                 self.dx, H, self.dbranch, H, False, gw, gb, self.ws)
        # the sharded step on the local gradient just written
        a.zero_reduce_shard([self.grad, self.peer], self.psi, "bf16", 1.0, self.reduced, self.step_ws, 0, self.flag)
        a.zero_grad_norm(None, self.psi, "bf16", 1.0, self.step_ws, 1, None, 0, 1.0, self.flag, self.norm, self.coef)
        a.zero_adam_step(self.master, self.m, self.v, self.reduced, "bf16", self.psi, self.hp, self.coef, self.flag,
                         self.param, "bf16")

    def state(self):
        return [t.clone() for t in (self.grad, self.reduced, self.master, self.m, self.v, self.param, self.dx,
                                    self.dbranch, self.res, self.y, self.h)]


def _same_bits(a, b):
    v = lambda t: t.view(torch.int32 if t.element_size() == 4 else torch.int16)
    return torch.equal(v(a), v(b))


def test_a_block_trains_from_its_checkpoints(abi):
    # Against autograd in fp64 on the unquantised block: the 8-bit checkpoints move a gradient by their own error
    # only.  INT8 of N(0,1) blocks of 256 (maximum near 3 sigma, or 8 sigma here at most) is off by at most half of
    # 8/127 per element, E4M3 by 2^-4 relative, independent from element to element; a relative L2 error of 5 % of each
    # gradient is more than the worst case of the norm of those errors for every tensor here (0.5 * 8/127 = 3.1 %
    # through one product, plus bf16 rounding of each of at most 5 intermediate tensors at 2^-8 = 0.4 %).
    blk = Block(abi, 5)
    w0 = blk.param.clone()
    blk.step()
    torch.cuda.synchronize()
    p = [t.detach().double().requires_grad_() for t in blk.parts(w0)]
    w, b, w1, b1, w2 = p
    x, br = blk.x.double().requires_grad_(), blk.branch.double().requires_grad_()
    res = x + 0.5 * br
    mu = res.mean(1, keepdim=True)
    y = (res - mu) / ((res - mu).square().mean(1, keepdim=True) + 1e-5).sqrt() * w + b
    gu = y @ w1.view(2 * blk.F, blk.H).t() + b1
    h = torch.nn.functional.silu(gu[:, :blk.F]) * gu[:, blk.F:]
    ((h @ w2.view(blk.H, blk.F).t() + res) * blk.do.double()).sum().backward()
    for got, want, what in zip(list(blk.parts(blk.grad)) + [blk.dx, blk.dbranch],
                               [t.grad for t in p] + [x.grad, br.grad],
                               ["norm weight", "norm bias", "W1", "b1", "W2", "dx", "dbranch"]):
        err = (got.double() - want).norm() / want.norm()
        assert err < 0.05, (what, float(err))
    assert int(blk.flag.item()) == 0 and not _same_bits(blk.param, w0)


def test_captured_steps_equal_eager_steps(abi):
    eager, graph = Block(abi, 9), Block(abi, 9)
    Block(abi, 1).step()                              # library and kernel start-up outside the capture
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        graph.step()
    for k in range(4):
        eager.step()
        g.replay()
        junk = torch.randn(1 << 18, device="cuda")
        assert torch.isfinite(junk.sum())
        torch.cuda.synchronize()
        for i, (p, q) in enumerate(zip(eager.state(), graph.state())):
            assert _same_bits(p, q), (k, i)


def test_two_streams_at_once_with_their_own_workspaces(abi):
    a, b, ref = Block(abi, 3), Block(abi, 4), [Block(abi, 3), Block(abi, 4)]
    for r in ref:
        r.step()
        r.step()
    torch.cuda.synchronize()
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(2):
        for blk, st in zip((a, b), s):
            with torch.cuda.stream(st):
                blk.step()
    torch.cuda.synchronize()
    for blk, r in zip((a, b), ref):
        for p, q in zip(blk.state(), r.state()):
            assert _same_bits(p, q)


def test_a_non_finite_activation_skips_the_step(abi):
    blk = Block(abi, 6)
    blk.branch[17, 3] = float("inf")
    w0 = blk.param.clone()
    blk.step()
    torch.cuda.synchronize()
    assert int(blk.flag.item()) & 1 and _same_bits(blk.param, w0) and not blk.m.any()
