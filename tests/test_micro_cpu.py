"""The 4-bit operands' host side: arguments that are refused before anything is
launched (fake device addresses, no GPU), and the definition that the GPU tests use
against hand-worked values."""
import ctypes

import numpy as np
import pytest
import torch

from tests import micro_ref as ref
from logprob_drift_scoring_gb300 import binding as B

FAKE = 0x7F0000000000


def operand(ptr=FAKE, block=16, stride=64, scales=FAKE, t=None):
    return B.LpdMicroScaled(ptr, block, 0, stride, scales, t)


def quantize_rc(x=FAKE, dtype=B.LPD_BF16, x_stride=100, rows=8, cols=100, transpose=0, out=operand(), values=None,
                vdtype=B.LPD_BF16, vstride=100):
    return B.lib().lpd_micro_quantize(x, dtype, x_stride, rows, cols, transpose, ctypes.byref(out) if out else None,
                                      values, vdtype, vstride, None)


def matmul_rc(a=operand(), b=operand(), m=8, n=8, k=100, out=FAKE, dtype=B.LPD_F32, stride=8, ws=FAKE, ws_bytes=1 << 30):
    return B.lib().lpd_micro_matmul(ctypes.byref(a) if a else None, ctypes.byref(b) if b else None, m, n, k, out, dtype,
                                    stride, ws, ws_bytes, None)


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), B.LPD_ERR_BAD_SIZE), (dict(cols=-1), B.LPD_ERR_BAD_SIZE), (dict(transpose=2), B.LPD_ERR_BAD_SIZE),
    (dict(rows=1 << 31), B.LPD_ERR_UNSUPPORTED),
    (dict(rows=(1 << 31) - 1, cols=(1 << 31) - 1, x_stride=1 << 31), B.LPD_ERR_UNSUPPORTED),
    (dict(x=None), B.LPD_ERR_NULL_POINTER), (dict(dtype=B.LPD_E4M3), B.LPD_ERR_BAD_DTYPE),
    (dict(x_stride=99), B.LPD_ERR_BAD_STRIDE), (dict(x=FAKE + 1), B.LPD_ERR_ALIGNMENT),
    (dict(x=FAKE + 2, dtype=B.LPD_F32), B.LPD_ERR_ALIGNMENT), (dict(out=None), B.LPD_ERR_NULL_POINTER),
    (dict(out=operand(ptr=None)), B.LPD_ERR_NULL_POINTER), (dict(out=operand(scales=None)), B.LPD_ERR_NULL_POINTER),
    (dict(out=operand(block=64)), B.LPD_ERR_BAD_SIZE), (dict(out=operand(block=0)), B.LPD_ERR_BAD_SIZE),
    (dict(out=operand(stride=49)), B.LPD_ERR_BAD_STRIDE), (dict(transpose=1, out=operand(stride=3)), B.LPD_ERR_BAD_STRIDE),
    (dict(out=operand(scales=FAKE + 8)), B.LPD_ERR_ALIGNMENT), (dict(out=operand(t=FAKE + 2)), B.LPD_ERR_ALIGNMENT),
    (dict(values=FAKE + 64, vdtype=B.LPD_E5M2), B.LPD_ERR_BAD_DTYPE), (dict(values=FAKE + 64, vstride=99), B.LPD_ERR_BAD_STRIDE),
    (dict(values=FAKE + 1), B.LPD_ERR_ALIGNMENT), (dict(values=FAKE), B.LPD_ERR_UNSUPPORTED),
])
def test_quantize_refuses(kw, code):
    assert quantize_rc(**kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(m=-1), B.LPD_ERR_BAD_SIZE), (dict(n=-1), B.LPD_ERR_BAD_SIZE), (dict(k=-1), B.LPD_ERR_BAD_SIZE),
    (dict(k=1 << 31), B.LPD_ERR_UNSUPPORTED), (dict(a=None), B.LPD_ERR_NULL_POINTER), (dict(b=None), B.LPD_ERR_NULL_POINTER),
    (dict(a=operand(ptr=None)), B.LPD_ERR_NULL_POINTER), (dict(b=operand(scales=None)), B.LPD_ERR_NULL_POINTER),
    (dict(a=operand(block=8)), B.LPD_ERR_BAD_SIZE), (dict(a=operand(block=32)), B.LPD_ERR_UNSUPPORTED),
    (dict(a=operand(stride=48)), B.LPD_ERR_BAD_STRIDE), (dict(b=operand(stride=56)), B.LPD_ERR_ALIGNMENT),
    (dict(a=operand(ptr=FAKE + 8)), B.LPD_ERR_ALIGNMENT), (dict(b=operand(scales=FAKE + 4)), B.LPD_ERR_ALIGNMENT),
    (dict(a=operand(t=FAKE + 1)), B.LPD_ERR_ALIGNMENT), (dict(out=None), B.LPD_ERR_NULL_POINTER),
    (dict(dtype=B.LPD_E4M3), B.LPD_ERR_BAD_DTYPE), (dict(stride=7), B.LPD_ERR_BAD_STRIDE),
    (dict(out=FAKE + 2), B.LPD_ERR_ALIGNMENT), (dict(ws=None), B.LPD_ERR_WORKSPACE), (dict(ws_bytes=255), B.LPD_ERR_WORKSPACE),
])
def test_matmul_refuses(kw, code):
    assert matmul_rc(**kw) == code


def test_empty_sizes_are_no_work():
    none = operand(ptr=None, scales=None)
    assert quantize_rc(x=None, rows=0, out=none) == B.LPD_OK
    assert quantize_rc(x=None, cols=0, x_stride=0, out=none) == B.LPD_OK
    assert matmul_rc(a=none, m=0, out=None) == B.LPD_OK
    assert matmul_rc(b=none, n=0, out=None, stride=0) == B.LPD_OK


def test_sizes():
    assert B.lpd_micro_scale_bytes(16, 1, 1) == 512 and B.lpd_micro_scale_bytes(16, 129, 65) == 4 * 512
    assert B.lpd_micro_scale_bytes(32, 128, 128) == 512 and B.lpd_micro_scale_bytes(32, 128, 129) == 1024
    assert B.lpd_micro_scale_bytes(16, 0, 50) == 0 and B.lpd_micro_scale_bytes(8, 4, 50) == 0
    assert B.lpd_micro_scale_bytes(16, -1, 50) == 0
    assert B.lpd_micro_workspace_size(4, 4, -1) == 0 and B.lpd_micro_workspace_size(4, 4, 4) >= 256


def test_binding_refuses():
    ok = B.micro_empty(4, 50, device="cpu")
    assert ok.codes.shape == (4, 25) and ok.codes.stride(0) == 32
    for kw in (dict(block=8), dict(k=80), dict(codes=ok.codes.float()), dict(scales=ok.scales[:-1]), dict(codes=ok.codes.T),
               dict(scales=ok.scales.float()), dict(tensor_scale=torch.ones(2)), dict(tensor_scale=torch.ones(1).double())):
        with pytest.raises(ValueError):
            B.MicroScaled(**{"codes": ok.codes, "scales": ok.scales, "k": 50, **kw})
    x = torch.zeros(4, 50)
    for args in ((x, ok), (x.T, ok), (x[:, :49], ok), (x, ok, True)):
        with pytest.raises(ValueError):  # (host tensors, where everything else fits)
            B.lpd_micro_quantize(*args)
    for out in (torch.zeros(4, 3), torch.zeros(4, 4)):
        with pytest.raises(ValueError):
            B.lpd_micro_matmul(ok, ok, out, torch.zeros(256, dtype=torch.uint8))


def test_definition_by_hand():
    v = np.array([0.0, -0.0, 0.25, 0.26, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 5.1, 100.0, -0.75, -7.0], dtype=np.float32)
    assert list(ref.e2m1(v)) == [0, 8, 0, 1, 2, 2, 4, 4, 6, 6, 7, 7, 10, 15]
    x = np.zeros((1, 40), dtype=np.float32)
    x[0, :16] = np.linspace(-6, 6, 16)
    x[0, 16:32], x[0, 39] = 1e-3, 12.0
    codes, scales, values = ref.quantize(x, 16)
    assert scales.shape == (1, 3) and list(scales[0]) == [0x38, 0x00, 0x40]  # 1, 0 (1e-3 / 6 is below half of 2^-9), 2
    assert codes[0, 0] == 15 and codes[0, 15] == 7 and not codes[0, 16:32].any() and codes[0, 39] == 7
    assert values[0, 39] == 12.0 and values[0, 20] == 0.0
    codes, scales, values = ref.quantize(x, 32)
    assert scales.shape == (1, 2) and list(scales[0]) == [127, 128] and values[0, 39] == 12.0
    assert list(ref.quantize(np.full((1, 32), 6.1, dtype=np.float32), 32)[1][0]) == [128]
    bad = x.copy()
    bad[0, 3] = np.inf
    assert np.isnan(ref.quantize(bad, 16)[2][0, :16]).all() and np.isfinite(ref.quantize(bad, 16)[2][0, 16:]).all()
    p = ref.packed(codes)
    assert p.shape == (1, 20) and np.array_equal(ref.unpacked(p, 40), codes) and p[0, 19] == 7 << 4 | codes[0, 38]
    assert ref.at(129, 5)[128, 4] == (1 * 2 + 1) * 512 and ref.at(129, 5)[33, 2] == 1 * 16 + 4 + 2
    back = ref.tiled(scales)
    assert np.array_equal(back[ref.at(1, 2)], scales)
    assert np.array_equal(ref.stands_for(codes, scales, 32), values.astype(np.float64))
