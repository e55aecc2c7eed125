"""Sizes and refusals of the activation-checkpoint calls (CPU: every call here
fails in validation or has nothing to do, before the HIP runtime is touched)."""

import random

import pytest
import torch

from zero_sharded_mixed_flat_amd import abi

E, L = abi.ZERO_EINVAL, abi.ZERO_EALIAS
# Fake, never-dereferenced device addresses far apart.
A = [0x1000000000 * (k + 1) for k in range(16)]
R, C = 4, 300
CODES, SCALES = R * 304, 4 * R * 2


def _args(defaults, kw):
    unknown = set(kw) - set(defaults)
    assert not unknown, unknown
    return {**defaults, **kw}


def _save(**kw):
    return abi.zero_act_save(**_args(dict(x=A[0], x_stride=C, dtype="bf16", rows=R, cols=C, format=1, codes=A[1],
                                          scales=A[2], stream=0), kw))


def _restore(**kw):
    return abi.zero_act_restore(**_args(dict(codes=A[1], scales=A[2], format=1, rows=R, cols=C, y=A[0], y_stride=C,
                                             dtype="bf16", stream=0), kw))


def _glu_f(**kw):
    return abi.zero_act_glu_forward(**_args(dict(
        gate=A[0], gate_stride=2 * C, up=A[0] + 2 * C, up_stride=2 * C, dtype="f16", rows=R, cols=C, fn=1, format=2,
        h=A[1], h_stride=C, gate_codes=A[2], gate_scales=A[3], up_codes=A[4], up_scales=A[5], stream=0), kw))


def _glu_b(**kw):
    return abi.zero_act_glu_backward(**_args(dict(
        gate_codes=A[2], gate_scales=A[3], up_codes=A[4], up_scales=A[5], format=2, rows=R, cols=C, fn=3, dh=A[0],
        dh_stride=C, dtype="f16", dgate=A[1], dgate_stride=2 * C, dup=A[1] + 2 * C, dup_stride=2 * C, h=A[6],
        h_stride=C, stream=0), kw))


def _norm_f(**kw):
    return abi.zero_act_norm_forward(**_args(dict(
        x=A[0], x_stride=C, branch=A[1], branch_stride=C, alpha=1.0, weight=A[2], bias=A[3], dtype="bf16", rows=R,
        cols=C, kind=2, eps=1e-5, format=1, res=A[4], res_stride=C, y=A[5], y_stride=C, codes=A[6], scales=A[7],
        mean=A[8], rstd=A[9], stream=0), kw))


def _norm_b(**kw):
    return abi.zero_act_norm_backward(**_args(dict(
        codes=A[0], scales=A[1], format=1, mean=A[2], rstd=A[3], weight=A[4], rows=R, cols=C, kind=2, dy=A[5],
        dy_stride=C, dres=A[6], dres_stride=C, alpha=0.5, dtype="bf16", dx=A[7], dx_stride=C, dbranch=A[8],
        dbranch_stride=C, accumulate=False, dweight=A[9], dbias=A[10], workspace=A[11], stream=0,
        workspace_bytes=abi.zero_act_norm_workspace_bytes(R, C)), kw))


def _wgrad(**kw):
    return abi.zero_act_weight_grad(**_args(dict(
        dy=A[0], dy_stride=77, dtype="bf16", codes=A[1], scales=A[2], format=1, rows=5000, in_cols=C, out_cols=77,
        accumulate=True, dweight=A[3], dbias=A[4], workspace=A[5], stream=0,
        workspace_bytes=abi.zero_act_weight_grad_workspace_bytes(5000, C, 77)), kw))


COMMON = [(dict(rows=-1), E), (dict(dtype=0), E), (dict(format=0), E), (dict(format=3), E),
          (dict(rows=1 << 27), E)]
COLS = [(dict(cols=-1), E), (dict(cols=(1 << 30) + 1), E)]

CASES = [(fn, kw, code) for fn in (_save, _restore, _glu_f, _glu_b, _norm_f, _norm_b) for kw, code in COMMON + COLS]
CASES += [(_wgrad, kw, code) for kw, code in COMMON]
CASES += [(_save, kw, code) for kw, code in [
    (dict(x=0), E), (dict(x=A[0] + 1), E), (dict(x_stride=C - 1), E), (dict(x_stride=1 << 62), E), (dict(codes=0), E),
    (dict(codes=A[1] + 8), E), (dict(scales=0), E), (dict(scales=A[2] + 2), E),
    (dict(codes=A[0] + 2 * R * C - 16), L), (dict(scales=A[0]), L), (dict(scales=A[1] + CODES - 4), L)]]
CASES += [(_restore, kw, code) for kw, code in [
    (dict(y=0), E), (dict(y=A[0] + 1), E), (dict(y_stride=C - 1), E), (dict(codes=A[1] + 4), E), (dict(scales=0), E),
    (dict(y=A[1] + CODES - 2), L), (dict(y=A[2] - 2 * R * C + 2), L)]]
CASES += [(_glu_f, kw, code) for kw, code in [
    (dict(fn=0), E), (dict(fn=4), E), (dict(up=None), E), (dict(up=None, up_codes=None), E), (dict(h=0), E),
    (dict(gate=0), E), (dict(up=A[7] + 1), E), (dict(up_stride=C - 1), E), (dict(up_codes=None), E),
    (dict(up_scales=None), E), (dict(gate_codes=A[2] + 1), E), (dict(h=A[0]), L),
    (dict(h=A[0] + 2 * C, h_stride=2 * C), L),            # h over up's half
    (dict(up_codes=A[2] + CODES - 16), L), (dict(up_scales=A[3]), L)]]
CASES += [(_glu_b, kw, code) for kw, code in [
    (dict(fn=9), E), (dict(dup=None), E), (dict(up_scales=None), E), (dict(up_codes=None), E), (dict(dgate=0), E),
    (dict(dh=A[0] + 1), E), (dict(dh_stride=3), E), (dict(h=A[6] + 1), E), (dict(h_stride=C - 1), E),
    (dict(dup=A[1] + 2 * C - 2), L),                        # the halves overlap by an element
    (dict(dup=A[1] + 2 * C + 2), L),                        # the second half runs into the next row
    (dict(dup=A[1], dup_stride=C), L), (dict(dgate=A[0]), L), (dict(h=A[0], h_stride=C), L),
    (dict(dgate=A[2], dgate_stride=C), L)]]
CASES += [(_norm_f, kw, code) for kw, code in [
    (dict(kind=0), E), (dict(kind=3), E), (dict(kind=1), E), (dict(mean=None), E), (dict(eps=0.0), E),
    (dict(eps=float("nan")), E), (dict(alpha=float("inf")), E), (dict(res=None), E), (dict(branch=None), E),
    (dict(cols=16385, x_stride=20000, branch_stride=20000, res_stride=20000, y_stride=20000), E), (dict(y=0), E),
    (dict(x_stride=C - 1), E), (dict(weight=A[2] + 1), E), (dict(bias=A[3] + 1), E), (dict(rstd=0), E),
    (dict(rstd=A[9] + 2), E), (dict(mean=A[8] + 1), E), (dict(codes=0), E), (dict(res=A[1]), L), (dict(y=A[0]), L),
    (dict(res=A[0], res_stride=C + 1), L), (dict(res=A[0] + 2), L), (dict(mean=A[9]), L), (dict(y=A[4]), L),
    (dict(rstd=A[2]), L)]]
CASES += [(_norm_b, kw, code) for kw, code in [
    (dict(kind=0), E), (dict(kind=1), E), (dict(mean=None), E), (dict(alpha=float("nan")), E), (dict(dx=0), E),
    (dict(dy=A[5] + 1), E), (dict(dres_stride=C - 1), E), (dict(dbranch=A[8] + 1), E), (dict(dweight=A[9] + 1), E),
    (dict(dbias=A[10] + 1), E), (dict(rstd=0), E), (dict(workspace=0), E), (dict(workspace=A[11] + 8), E),
    (dict(workspace_bytes=16), E), (dict(dx=A[5]), L), (dict(dbranch=A[6]), L), (dict(dx=A[6] + 2), L),
    (dict(dweight=A[10]), L), (dict(dweight=A[4]), L), (dict(workspace=A[7]), L), (dict(dx=A[8]), L)]]
CASES += [(_wgrad, kw, code) for kw, code in [
    (dict(in_cols=-1), E), (dict(out_cols=-1), E), (dict(rows=1, in_cols=1 << 20, out_cols=1 << 20), E),
    (dict(dy=0), E), (dict(dy=A[0] + 1), E), (dict(dy_stride=76), E), (dict(codes=A[1] + 8), E), (dict(scales=0), E),
    (dict(dweight=0), E), (dict(dweight=A[3] + 1), E), (dict(dbias=A[4] + 1), E), (dict(dweight=A[0]), L),
    (dict(dbias=A[3] + 2), L), (dict(dweight=A[1]), L), (dict(dbias=A[2]), L)]]


@pytest.mark.parametrize("fn,kw,code", CASES, ids=lambda v: getattr(v, "__name__", None) or str(v)[:60])
def test_refusals(fn, kw, code):
    with pytest.raises(abi.ZeroError) as e:
        fn(**kw)
    assert e.value.code == code, str(e.value)
    assert "zero_act_" in str(e.value)


def test_sizes():
    assert abi.zero_act_code_bytes(3, 17) == 3 * 32 and abi.zero_act_code_bytes(0, 5) == 0
    assert abi.zero_act_scale_count(3, 257) == 6 and abi.zero_act_scale_count(3, 0) == 0
    assert abi.zero_act_code_bytes(1 << 26, 256) == 1 << 34
    for bad in ((-1, 5), (5, -1), ((1 << 26) + 1, 1), (1 << 20, 16385), (1, (1 << 30) + 1)):
        for fn in (abi.zero_act_code_bytes, abi.zero_act_scale_count, abi.zero_act_norm_workspace_bytes):
            with pytest.raises(abi.ZeroError):
                fn(*bad)
        with pytest.raises(abi.ZeroError):
            abi.zero_act_weight_grad_workspace_bytes(bad[0], bad[1], 4)
    with pytest.raises(abi.ZeroError):
        abi.zero_act_norm_workspace_bytes(2, 16385)
    assert abi.zero_act_norm_workspace_bytes(0, 100) == 0


def test_a_workspace_for_more_rows_serves_fewer():
    rng = random.Random(3)
    for _ in range(300):
        a, b = rng.choice([1, 40, 1024, 3000, 16384]), rng.randint(1, 20000)
        rows = sorted(rng.randint(1, 40000) for _ in range(12)) + [4095, 4096, 4097, 5000, 127, 128, 129, 65536]
        rows.sort()
        norm = [abi.zero_act_norm_workspace_bytes(r, min(a, 16384)) for r in rows]
        grad = [abi.zero_act_weight_grad_workspace_bytes(r, a, b) for r in rows]
        assert norm == sorted(norm) and grad == sorted(grad), (a, b)
        assert all(g % 4 == 0 for g in grad)


def test_nothing_to_do():
    _save(rows=0, x=0, codes=0, scales=0)
    _restore(cols=0, y=0, codes=0, scales=0)
    _glu_f(rows=0, gate=0, h=0)
    _glu_b(cols=0, dh=0)
    _norm_f(rows=0, x=0)
    _norm_b(cols=0, dy=0)
    _wgrad(out_cols=0, dy=0)
    _norm_b(rows=0, accumulate=True, workspace=None, workspace_bytes=0)
    _wgrad(rows=0, workspace=None, workspace_bytes=0)


def test_tensors_are_checked():
    cpu = torch.zeros(R, C, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="x must be a device tensor"):
        _save(x=cpu)
    with pytest.raises(ValueError, match="codes must be a device tensor"):
        _save(codes=torch.zeros(CODES, dtype=torch.uint8))
    with pytest.raises(ValueError, match="dweight must be a device tensor"):
        _wgrad(dweight=cpu)


class _Fake:
    """What the binding looks at of a device tensor."""

    is_cuda = True

    def __init__(self, shape, stride, index=0, size=2, room=None, offset=0):
        self.shape, self._stride, self._size, self._offset = shape, stride, size, offset
        self._index = index
        self._room = room if room is not None else offset + (shape[0] - 1) * stride[0] + shape[-1]

    def get_device(self):
        return self._index

    def stride(self):
        return self._stride

    def element_size(self):
        return self._size

    def storage_offset(self):
        return self._offset

    def untyped_storage(self):
        return type("S", (), {"nbytes": lambda _: self._room * self._size})()

    def data_ptr(self):
        return A[0]


@pytest.mark.parametrize("fake,match", [
    (_Fake((R, C), (C, 1), index=1), "on device 1"),
    (_Fake((R, C), (C, 1), size=4), "16-bit"),
    (_Fake((R, C), (C, 2)), "adjacent"),
    (_Fake((R, C), (C + 2, 1)), "apart"),
    (_Fake((R - 1, C), (C, 1)), "holds"),
    (_Fake((R * C - 1,), (1,), room=R * C - 1), "holds"),
])
def test_matrices_are_checked(monkeypatch, fake, match):
    monkeypatch.setattr(abi, "_device", lambda: 0)
    with pytest.raises(ValueError, match=match):
        _save(x=fake)
