"""The element types the activation calls' binding takes (CPU: a fake library stands
where the call would be made, and the tensors' device is told to be the current one)."""

import pytest
import torch

from zero_sharded_mixed_flat_amd import abi

R, C, O = 6, 300, 20
BF, HF, F32, F64 = torch.bfloat16, torch.float16, torch.float32, torch.float64


class _Library:
    """Takes every call; sizes come from the real library."""

    def __init__(self, real):
        self._real = real
        self.called = 0

    def __getattr__(self, name):
        if name.endswith("_bytes") or name.endswith("_count"):
            return getattr(self._real, name)

        def call(*args):
            self.called += 1
            return 0
        return call


@pytest.fixture
def library(monkeypatch):
    fake = _Library(abi.lib)
    monkeypatch.setattr(abi, "lib", fake)
    monkeypatch.setattr(abi, "_device", lambda: -1)        # where CPU tensors are
    return fake


def _t(*shape, dtype=BF):
    return torch.zeros(*shape, dtype=dtype)


def _codes(rows=R, cols=C):
    return torch.zeros(abi.zero_act_code_bytes(rows, cols), dtype=torch.uint8)


def _scales(rows=R, cols=C):
    return torch.zeros(abi.zero_act_scale_count(rows, cols))


CALLS = {
    "save": (abi.zero_act_save, lambda: dict(x=_t(R, C), x_stride=C, dtype="bf16", rows=R, cols=C, format=1,
                                             codes=_codes(), scales=_scales(), stream=0)),
    "restore": (abi.zero_act_restore, lambda: dict(codes=_codes(), scales=_scales(), format=1, rows=R, cols=C,
                                                   y=_t(R, C), y_stride=C, dtype=BF, stream=0)),
    "glu_forward": (abi.zero_act_glu_forward, lambda: dict(
        gate=_t(R, C), gate_stride=C, up=_t(R, C), up_stride=C, dtype=2, rows=R, cols=C, fn=1, format=2, h=_t(R, C),
        h_stride=C, gate_codes=_codes(), gate_scales=_scales(), up_codes=_codes(), up_scales=_scales(), stream=0)),
    "glu_backward": (abi.zero_act_glu_backward, lambda: dict(
        gate_codes=_codes(), gate_scales=_scales(), up_codes=_codes(), up_scales=_scales(), format=2, rows=R, cols=C,
        fn=1, dh=_t(R, C), dh_stride=C, dtype="bf16", dgate=_t(R, C), dgate_stride=C, dup=_t(R, C), dup_stride=C,
        h=_t(R, C), h_stride=C, stream=0)),
    "norm_forward": (abi.zero_act_norm_forward, lambda: dict(
        x=_t(R, C), x_stride=C, branch=_t(R, C), branch_stride=C, alpha=1.0, weight=_t(C), bias=_t(C), dtype="bf16",
        rows=R, cols=C, kind=2, eps=1e-5, format=1, res=_t(R, C), res_stride=C, y=_t(R, C), y_stride=C, codes=_codes(),
        scales=_scales(), mean=_t(R, dtype=F32), rstd=_t(R, dtype=F32), stream=0)),
    "norm_backward": (abi.zero_act_norm_backward, lambda: dict(
        codes=_codes(), scales=_scales(), format=1, mean=_t(R, dtype=F32), rstd=_t(R, dtype=F32), weight=_t(C), rows=R,
        cols=C, kind=2, dy=_t(R, C), dy_stride=C, dres=_t(R, C), dres_stride=C, alpha=1.0, dtype="bf16", dx=_t(R, C),
        dx_stride=C, dbranch=_t(R, C), dbranch_stride=C, accumulate=False, dweight=_t(C), dbias=_t(C),
        workspace=_t(abi.zero_act_norm_workspace_bytes(R, C), dtype=torch.uint8), stream=0)),
    "weight_grad": (abi.zero_act_weight_grad, lambda: dict(
        dy=_t(R, O), dy_stride=O, dtype="bf16", codes=_codes(), scales=_scales(), format=1, rows=R, in_cols=C, out_cols=O,
        accumulate=False, dweight=_t(O, C), dbias=_t(O), workspace=_t(1 << 20, dtype=torch.uint8), stream=0)),
}

ARGS = [(c, k, v.dtype) for c, (_, make) in CALLS.items() for k, v in make().items()
        if isinstance(v, torch.Tensor) and v.dtype is not torch.uint8]       # codes and workspaces are bytes


@pytest.mark.parametrize("call", CALLS)
def test_the_calls_own_types_are_taken(library, call):
    fn, make = CALLS[call]
    fn(**make())
    assert library.called == 1


@pytest.mark.parametrize("call,arg,dtype", ARGS, ids=lambda v: str(v))
def test_another_type_of_values_is_refused(library, call, arg, dtype):
    fn, make = CALLS[call]
    others = {BF: [HF, F32], F32: [F64, BF]}[dtype]
    for other in others:
        kw = make()
        kw[arg] = torch.zeros_like(kw[arg], dtype=other) if other.itemsize >= dtype.itemsize else \
            torch.zeros(4 * kw[arg].numel(), dtype=other)
        with pytest.raises(ValueError, match=arg):
            fn(**kw)
    assert library.called == 0


@pytest.mark.parametrize("call,arg,dtype", ARGS, ids=lambda v: str(v))
def test_bit_patterns_and_bytes_are_taken(library, call, arg, dtype):
    # Buffers that hold the values under a type without a meaning of its own: patterns of the same
    # size, and for what is flat memory also bytes.
    fn, make = CALLS[call]
    kw = make()
    kw[arg] = kw[arg].view({BF: torch.int16, F32: torch.int32}[dtype])
    fn(**kw)
    if kw[arg].dim() == 1:
        kw[arg] = kw[arg].view(torch.uint8)
        fn(**kw)
    assert library.called in (1, 2)


def test_codes_of_8_bit_floats_are_taken(library):
    fn, make = CALLS["save"]
    kw = make()
    kw.update(codes=kw["codes"].view(torch.float8_e4m3fn), format=2)
    fn(**kw)
    assert library.called == 1


def test_a_dtype_the_library_refuses_is_the_librarys_to_report():
    with pytest.raises(abi.ZeroError, match="dtype"):
        abi.zero_act_save(0, C, 7, R, C, 1, 0, 0, stream=0)
