"""Pins of the activation-checkpoint oracle (CPU)."""

import numpy as np
import pytest
import torch

from oracle import act, quant, rounding


def test_e4m3_table_is_torchs():
    codes = np.arange(256, dtype=np.uint8)
    ref = torch.from_numpy(codes.copy()).view(torch.float8_e4m3fn).float().numpy()
    finite = (codes & 0x7F) < 127
    assert np.array_equal(act.e4m3_decode(codes)[finite], ref[finite])
    # rounding: every midpoint, its neighbours and random values against torch's cast
    mid = act._E4M3_MID.astype(np.float32)
    q = np.concatenate([mid, np.nextafter(mid, np.float32(0)), np.nextafter(mid, np.float32(1e3)),
                        np.random.default_rng(0).uniform(-448, 448, 20000).astype(np.float32),
                        np.exp2(np.random.default_rng(1).uniform(-12, 8.8, 20000)).astype(np.float32)])
    q = np.concatenate([q, -q])
    ref = torch.from_numpy(q).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(act.e4m3_encode(q), ref)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_int8_rows_of_whole_blocks_are_the_flat_quantiser(dtype):
    rng = np.random.default_rng(3)
    x = rounding.narrow(rng.standard_normal(6 * 512).astype(np.float32), dtype)
    codes, scales = act.save(x.reshape(6, 512), dtype, "int8")
    ref_codes, ref_scales = quant.quantize(x, dtype, 8)
    assert np.array_equal(codes.view(np.int8).ravel(), ref_codes) and np.array_equal(scales.ravel(), ref_scales)
    assert np.array_equal(act.restore(codes, scales, dtype, "int8").ravel(), quant.dequantize(ref_codes, ref_scales, dtype))


@pytest.mark.parametrize("fmt,bound", [("int8", 0.5 / 127), ("e4m3", 2.0 ** -4)])
def test_restored_values_are_close(fmt, bound):
    # INT8: half a step of the block's scale; E4M3: half an ulp (2^-4 relative) of the value
    rng = np.random.default_rng(4)
    x = rounding.narrow(rng.standard_normal((7, 300)).astype(np.float32), "f16").reshape(7, 300)
    codes, scales = act.save(x, "f16", fmt)
    v, back = rounding.widen(x, "f16"), rounding.widen(act.restore(codes, scales, "f16", fmt), "f16")
    amax = np.repeat(np.stack([np.abs(v[:, :256]).max(1), np.abs(v[:, 256:]).max(1)], 1), 256, 1)[:, :300]
    size = amax if fmt == "int8" else np.maximum(np.abs(v), amax * 2.0 ** -6 / 448)
    assert np.all(np.abs(back - v) <= size * bound * 1.001 + np.abs(v) * 2.0 ** -11 + 2.0 ** -25)


def test_non_finite_blocks_become_nan_and_zero_blocks_stay_zero():
    x = np.zeros((3, 512), np.uint16)
    x[0, 5] = 0x7C00                                 # +inf in fp16
    x[1, 300] = 0x7E00                               # NaN
    x[2, :256] = 0x3C00
    codes, scales = act.save(x, "f16", "int8")
    assert np.isnan(scales[0, 0]) and scales[0, 1] == 0 and np.isnan(scales[1, 1]) and scales[1, 0] == 0
    assert not codes[0].any() and not codes[1].any() and (codes[2, :256].view(np.int8) == 127).all()
    back = rounding.widen(act.restore(codes, scales, "f16", "int8"), "f16")
    assert np.isnan(back[0, :256]).all() and (back[0, 256:] == 0).all() and np.isnan(back[1, 256:]).all()


@pytest.mark.parametrize("fn,ref", [("silu", torch.nn.functional.silu), ("gelu", torch.nn.functional.gelu),
                                    ("gelu_tanh", lambda t: torch.nn.functional.gelu(t, approximate="tanh"))])
def test_activations_are_torchs(fn, ref):
    g = torch.linspace(-12, 12, 4001, dtype=torch.float64, requires_grad=True)
    y = ref(g)
    y.sum().backward()
    f, _, df, _ = act.act(g.detach().numpy(), fn)
    assert np.allclose(f, y.detach().numpy(), rtol=1e-12, atol=1e-14)
    assert np.allclose(df, g.grad.numpy(), rtol=1e-11, atol=1e-13)


@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_norm_backward_is_autograds(kind):
    rng = np.random.default_rng(7)
    r = torch.tensor(rng.standard_normal((5, 24)), requires_grad=True)
    w = torch.tensor(rng.standard_normal(24), requires_grad=True)
    b = torch.tensor(rng.standard_normal(24), requires_grad=True)
    dy, dres = rng.standard_normal((5, 24)), rng.standard_normal((5, 24))
    eps = float(np.float32(1e-5))
    m = r.mean(1, keepdim=True) if kind == "layer" else 0.0
    y = (r - m) / ((r - m).square().mean(1, keepdim=True) + eps).sqrt() * w + b
    ((y * torch.tensor(dy)).sum() + (r * torch.tensor(dres)).sum()).backward()
    (yo, _), (rstd, _), (mean, _) = act.norm_forward(r.detach().numpy(), w.detach().numpy(), b.detach().numpy(), kind, eps)
    assert np.allclose(yo, y.detach().numpy(), rtol=1e-12)
    (dr, _), (dw, _), (db, _) = act.norm_backward(r.detach().numpy(), mean, rstd, w.detach().numpy(), dy, dres, kind, 1)
    assert np.allclose(dr, r.grad.numpy(), rtol=1e-10, atol=1e-12)
    assert np.allclose(dw, w.grad.numpy(), rtol=1e-10) and np.allclose(db, b.grad.numpy(), rtol=1e-12)
