"""Activation-checkpoint calls on matrices without elements (CPU: nothing is launched).

A tensor without elements has no address, so with no rows or no columns which
optional arguments are present cannot be told from their addresses.
"""

import pytest
import torch

from zero_sharded_mixed_flat_amd import abi

F32, U8 = torch.float32, torch.uint8
# Fake, never-dereferenced device addresses: buffers sized for the longest batch.
A = [0x1000000000 * (k + 1) for k in range(8)]


def _e(*shape, dtype=torch.bfloat16):
    t = torch.empty(*shape, dtype=dtype)
    assert t.numel() == 0 and t.data_ptr() == 0
    return t


SIZES = [(0, 300), (5, 0), (0, 0)]


def _vec(rows):
    return _e(0, dtype=F32) if rows == 0 else A[7]


@pytest.mark.parametrize("rows,cols", SIZES)
@pytest.mark.parametrize("kind", [1, 2])
def test_norm_forward(rows, cols, kind):
    mean = _vec(rows) if kind == 2 else None
    m = lambda: _e(rows, cols)
    codes, scales = _e(0, dtype=U8), _e(0, dtype=F32)
    abi.zero_act_norm_forward(m(), cols, m(), cols, 1.0, None, None, "bf16", rows, cols, kind, 1e-5, 1, m(), cols, m(),
                              cols, codes, scales, mean, _vec(rows), stream=0)
    # a batch's empty slices next to whole buffers
    abi.zero_act_norm_forward(m(), cols, m(), cols, 1.0, None, None, "bf16", rows, cols, kind, 1e-5, 1, A[0], cols, A[1],
                              cols, A[2], A[3], mean, A[4], stream=0)


@pytest.mark.parametrize("kind", [1, 2])
def test_norm_backward(kind):
    mean = _e(0, dtype=F32) if kind == 2 else None
    m = lambda: _e(0, 300)
    for dw, db in ((None, None), (A[0], A[1])):          # accumulating over no rows: nothing to write
        abi.zero_act_norm_backward(_e(0, dtype=U8), _e(0, dtype=F32), 1, mean, _e(0, dtype=F32), None, 0, 300, kind, m(),
                                   300, m(), 300, 0.5, "bf16", m(), 300, m(), 300, True, dw, db, None, stream=0)
    n = lambda: _e(5, 0)
    abi.zero_act_norm_backward(_e(0, dtype=U8), _e(0, dtype=F32), 1, A[2] if kind == 2 else None, A[3], None, 5, 0, kind,
                               n(), 0, None, 0, 1.0, "bf16", n(), 0, None, 0, False, None, None, None, stream=0)


@pytest.mark.parametrize("rows,cols", SIZES)
def test_glu(rows, cols):
    m = lambda: _e(rows, 2 * cols)
    bufs = [(A[0], A[1], A[2], A[3]), tuple(_e(0, dtype=t) for t in (U8, F32, U8, F32))]
    for gc, gs, uc, us in bufs:
        abi.zero_act_glu_forward(m()[:, :cols], 2 * cols, m()[:, cols:], 2 * cols, "bf16", rows, cols, 1, 1,
                                 _e(rows, cols), cols, gc, gs, uc, us, stream=0)
        abi.zero_act_glu_backward(gc, gs, uc, us, 1, rows, cols, 1, _e(rows, cols), cols, "bf16", m()[:, :cols], 2 * cols,
                                  m()[:, cols:], 2 * cols, stream=0)


def test_what_can_be_told_is_still_refused():
    with pytest.raises(abi.ZeroError):
        abi.zero_act_glu_forward(0, 9, 0, 9, "f16", 0, 9, 4, 1, 0, 9, 0, 0, 0, 0, stream=0)        # fn
    with pytest.raises(abi.ZeroError):
        abi.zero_act_norm_forward(0, 9, None, 0, 1.0, None, None, "f16", 0, 9, 1, 0.0, 1, None, 0, 0, 9, 0, 0, None, 0,
                                  stream=0)                                                       # eps
    with pytest.raises(abi.ZeroError):
        abi.zero_act_norm_backward(0, 0, 1, None, 0, None, 0, 9, 3, 0, 9, None, 0, 1.0, "f16", 0, 9, None, 0, False, None,
                                   None, None, stream=0)                                          # kind
