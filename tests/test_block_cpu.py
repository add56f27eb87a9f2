"""The 8-bit operands' host side: arguments refused before anything is launched
(fake device addresses, no GPU), and the binding's checks."""
import contextlib
import ctypes

import pytest
import torch

from logprob_drift_scoring_gb300 import binding as B

FAKE = 0x7F0000000000
WS = FAKE + 0x100000


def operand(**kw):
    return B.LpdBlockScaled(**{**dict(ptr=FAKE, dtype=B.LPD_E4M3, block=0, row_stride=512, scales=FAKE, scale_stride=4), **kw})


BAD = [(dict(ptr=None), B.LPD_ERR_NULL_POINTER), (dict(scales=None), B.LPD_ERR_NULL_POINTER),
       (dict(dtype=B.LPD_BF16), B.LPD_ERR_BAD_DTYPE), (dict(dtype=4), B.LPD_ERR_BAD_DTYPE),
       (dict(block=2), B.LPD_ERR_BAD_SIZE), (dict(row_stride=496), B.LPD_ERR_BAD_STRIDE),
       (dict(scale_stride=3), B.LPD_ERR_BAD_STRIDE), (dict(scales=FAKE + 2), B.LPD_ERR_ALIGNMENT)]


def matmul_rc(a=None, b=None, m=8, n=9, k=500, out=FAKE, out_dtype=B.LPD_F32, out_stride=9, ws=WS, ws_bytes=1 << 20):
    a, b = a or operand(), b or operand()
    return B.lib().lpd_block_matmul(ctypes.byref(a), ctypes.byref(b), m, n, k, out, out_dtype, out_stride, ws, ws_bytes, None)


def quantize_rc(x=FAKE, dtype=B.LPD_BF16, stride=500, rows=8, cols=500, transpose=0, pow2=0, out=None):
    out = out or operand()
    return B.lib().lpd_block_quantize(x, dtype, stride, rows, cols, transpose, pow2, ctypes.byref(out), None)


@pytest.mark.parametrize("kw,code", BAD)
def test_bad_operands(kw, code):
    assert matmul_rc(a=operand(**kw)) == code
    assert matmul_rc(b=operand(**kw)) == code
    assert quantize_rc(out=operand(**kw)) == code


@pytest.mark.parametrize("kw,code", [
    (dict(a=operand(ptr=FAKE + 8)), B.LPD_ERR_ALIGNMENT), (dict(b=operand(row_stride=520)), B.LPD_ERR_ALIGNMENT),
    (dict(m=-1), B.LPD_ERR_BAD_SIZE), (dict(n=-1), B.LPD_ERR_BAD_SIZE), (dict(k=-1), B.LPD_ERR_BAD_SIZE),
    (dict(m=1 << 31), B.LPD_ERR_UNSUPPORTED), (dict(out=None), B.LPD_ERR_NULL_POINTER),
    (dict(out_dtype=B.LPD_E4M3), B.LPD_ERR_BAD_DTYPE), (dict(out_stride=8), B.LPD_ERR_BAD_STRIDE),
    (dict(out=FAKE + 2), B.LPD_ERR_ALIGNMENT), (dict(ws=None), B.LPD_ERR_WORKSPACE), (dict(ws_bytes=255), B.LPD_ERR_WORKSPACE),
    (dict(ws=WS + 128), B.LPD_ERR_ALIGNMENT),
])
def test_matmul_refusals(kw, code):
    assert matmul_rc(**kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), B.LPD_ERR_BAD_SIZE), (dict(cols=-1), B.LPD_ERR_BAD_SIZE), (dict(transpose=2), B.LPD_ERR_BAD_SIZE),
    (dict(pow2=-1), B.LPD_ERR_BAD_SIZE), (dict(x=None), B.LPD_ERR_NULL_POINTER), (dict(dtype=B.LPD_E4M3), B.LPD_ERR_BAD_DTYPE),
    (dict(stride=499), B.LPD_ERR_BAD_STRIDE), (dict(x=FAKE + 1), B.LPD_ERR_ALIGNMENT),
    (dict(rows=1 << 31), B.LPD_ERR_UNSUPPORTED), (dict(transpose=1, rows=600), B.LPD_ERR_BAD_STRIDE),
])
def test_quantize_refusals(kw, code):
    assert quantize_rc(**kw) == code


def test_null_structs():
    L = B.lib()
    a = operand()
    assert L.lpd_block_matmul(None, ctypes.byref(a), 8, 9, 500, FAKE, B.LPD_F32, 9, WS, 1 << 20, None) == B.LPD_ERR_NULL_POINTER
    assert L.lpd_block_quantize(FAKE, B.LPD_BF16, 500, 8, 500, 0, 0, None, None) == B.LPD_ERR_NULL_POINTER


def test_workspace_size():
    assert B.lpd_block_workspace_size(-1, 5, 5) == 0 and B.lpd_block_workspace_size(5, 5, 1 << 31) == 0
    assert B.lpd_block_workspace_size(4096, 151936, 4096) >= 256


def test_binding_checks():
    f8 = torch.float8_e4m3fn
    good = B.BlockScaled(torch.zeros(130, 256, dtype=torch.uint8).view(f8), torch.ones(130, 2))
    B.BlockScaled(torch.zeros(130, 256, dtype=torch.uint8).view(f8), torch.ones(2, 2), block=True)
    for values, scales, block in ((torch.zeros(130, 256), torch.ones(130, 2), False),
                                  (good.values, torch.ones(130, 3), False), (good.values, torch.ones(130, 2), True),
                                  (good.values, torch.ones(130, 2, dtype=torch.float64), False),
                                  (good.values.t(), torch.ones(256, 2), False)):
        with pytest.raises(ValueError):
            B.BlockScaled(values, scales, block)
    with pytest.raises(ValueError, match="shape"):
        B.lpd_block_quantize(torch.zeros(256, 130), good)
    with pytest.raises(ValueError, match="device memory"):
        B.lpd_block_quantize(torch.zeros(130, 256), good)
    with pytest.raises(ValueError, match="fit"):
        B.lpd_block_matmul(good, good, torch.zeros(130, 131), torch.zeros(256, dtype=torch.uint8))
    with pytest.raises(ValueError, match="device memory"):
        B.lpd_block_matmul(good, good, torch.zeros(130, 130), torch.zeros(256, dtype=torch.uint8))


def test_block_empty_rows_fit_the_product():
    op = B.block_empty(5, 300, torch.float8_e5m2, device="cpu")
    assert op.values.shape == (5, 300) and op.values.stride(0) == 304 and op.scales.shape == (5, 3)
    assert B.block_empty(300, 130, torch.float8_e4m3fn, True, "cpu").scales.shape == (3, 2)
    one = B.block_empty(1, 20, torch.float8_e4m3fn, device="cpu")
    assert one._struct.row_stride == 32 and one._struct.scale_stride == 1


class Recorder:
    """In place of the library: the arguments of each call, nothing launched."""

    def __init__(self, monkeypatch):
        self.calls = []
        monkeypatch.setattr(B, "lib", lambda: self)
        monkeypatch.setattr(B, "_on", lambda t: contextlib.nullcontext())

    def __getattr__(self, name):
        return lambda *a: self.calls.append((name, a)) or B.LPD_OK


def overlapping(rows, cols, dtype=torch.bfloat16):
    """A repeated row and rows one element apart: strides (0, 1) and (1, 1)."""
    return torch.zeros(cols, dtype=dtype).expand(rows, cols), torch.zeros(rows + cols - 1, dtype=dtype).unfold(0, cols, 1)


def test_rows_that_overlap_keep_their_stride(monkeypatch):
    """The quantiser's input and the product's output are handed over with the stride that they have, and
    the library refuses it: their storage is smaller than rows x width."""
    assert quantize_rc(stride=0) == quantize_rc(stride=1) == B.LPD_ERR_BAD_STRIDE
    assert matmul_rc(out_stride=0) == matmul_rc(out_stride=1) == B.LPD_ERR_BAD_STRIDE
    a, b = (B.block_empty(r, 256, torch.float8_e4m3fn, device="cpu") for r in (40, 130))
    ws = torch.zeros(256, dtype=torch.uint8)
    lib = Recorder(monkeypatch)
    for x, stride in zip(overlapping(40, 256), (0, 1)):
        B.lpd_block_quantize(x, a, stream=0)
        assert lib.calls[-1][1][2] == stride
    for out, stride in zip(overlapping(40, 130), (0, 1)):
        B.lpd_block_matmul(a, b, out, ws, stream=0)
        assert lib.calls[-1][1][7] == stride
    # padded rows; a single row may have any stride
    B.lpd_block_quantize(torch.zeros(40, 300)[:, :256], a, stream=0)
    assert lib.calls[-1][1][2] == 300
    one = B.block_empty(1, 256, torch.float8_e4m3fn, device="cpu")
    B.lpd_block_quantize(torch.zeros(256).expand(1, 256), one, stream=0)
    assert lib.calls[-1][1][2] == 256
    B.lpd_block_matmul(one, b, torch.zeros(130).expand(1, 130), ws, stream=0)
    assert lib.calls[-1][1][7] == 130


def test_a_product_workspace_of_repeated_elements_or_elsewhere_is_refused(monkeypatch):
    a, b = (B.block_empty(r, 256, torch.float8_e4m3fn, device="cpu") for r in (40, 130))
    out = torch.zeros(40, 130)
    lib = Recorder(monkeypatch)
    for bad in (torch.zeros(1).expand(4096), torch.zeros(4096, device="meta"), torch.zeros(8192)[::2]):
        with pytest.raises(ValueError, match="workspace"):
            B.lpd_block_matmul(a, b, out, bad, stream=0)
    assert lib.calls == []
    B.lpd_block_matmul(a, b, out, torch.zeros(4096), stream=0)
    assert lib.calls[-1][1][9] == 4096 * 4
