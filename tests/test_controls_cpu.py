"""The sampling controls' host side: arguments that are refused before anything
is launched (fake device addresses, no GPU), and the definition that the GPU
tests use against hand-worked values."""
import contextlib
import ctypes

import numpy as np
import pytest
import torch

from tests import controls_ref as ref
from logprob_drift_scoring_gb300 import binding as B

FAKE = 0x7F0000000000
WS = FAKE + 0x100000


def controls(**kw):
    base = dict(history=FAKE, n_history=10, hist_begin=FAKE, hist_split=FAKE, hist_end=FAKE, repetition=FAKE,
                bias_ids=FAKE, bias=FAKE, n_bias=2, mask=FAKE, n_masks=8, mask_stride=2)
    return B.LpdControls(**{**base, **kw})


BAD_CONTROLS = [
    (dict(n_history=-1), B.LPD_ERR_BAD_SIZE),
    (dict(n_bias=-1), B.LPD_ERR_BAD_SIZE),
    (dict(n_masks=-1), B.LPD_ERR_BAD_SIZE),
    (dict(n_bias=B.LPD_MAX_BIAS + 1), B.LPD_ERR_UNSUPPORTED),
    (dict(hist_begin=None), B.LPD_ERR_NULL_POINTER),
    (dict(hist_split=None), B.LPD_ERR_NULL_POINTER),
    (dict(hist_end=None), B.LPD_ERR_NULL_POINTER),
    (dict(bias_ids=None), B.LPD_ERR_NULL_POINTER),
    (dict(bias=None), B.LPD_ERR_NULL_POINTER),
    (dict(mask_stride=1), B.LPD_ERR_BAD_STRIDE),
    (dict(n_masks=3), B.LPD_ERR_BAD_SIZE),
    (dict(history=FAKE + 2), B.LPD_ERR_ALIGNMENT),
    (dict(hist_end=FAKE + 4), B.LPD_ERR_ALIGNMENT),
    (dict(mask=FAKE + 1), B.LPD_ERR_ALIGNMENT),
    (dict(scale=FAKE + 2), B.LPD_ERR_ALIGNMENT),
]


def logits(ptr=FAKE, dtype=B.LPD_BF16, stride=40):
    return B.LpdLogits(ptr, dtype, 0, stride)


def apply_rc(x=None, c=None, n_rows=8, vocab=40, out=FAKE + 0x10000, out_dtype=B.LPD_F32, out_stride=40):
    x = x or logits()
    return B.lib().lpd_controls_apply(ctypes.byref(x), ctypes.byref(c) if c else None, n_rows, vocab, out, out_dtype,
                                      out_stride, None)


def score_rc(ct=None, cr=None, n_rows=8, vocab=40, met=FAKE, ids=FAKE, mask=FAKE, lo=0.8, hi=1.2, ws=WS, ws_bytes=1 << 20):
    x, y = logits(), logits(dtype=B.LPD_F32)
    return B.lib().lpd_score_controlled(ctypes.byref(x), ctypes.byref(y), ctypes.byref(ct) if ct else None,
                                        ctypes.byref(cr) if cr else None, n_rows, vocab, ids, mask, lo, hi, None,
                                        None, None, met, ws, ws_bytes, None)


def grad_rc(x=None, c=None, n_rows=8, vocab=40, ids=FAKE, mask=FAKE, logp=FAKE, grad=FAKE, out=FAKE + 0x10000,
            out_dtype=B.LPD_F32, out_stride=40):
    x = x or logits()
    return B.lib().lpd_logprob_backward_controlled(ctypes.byref(x), ctypes.byref(c) if c else None, n_rows, vocab,
                                                   ids, mask, logp, grad, out, out_dtype, out_stride, None)


@pytest.mark.parametrize("kw,code", BAD_CONTROLS)
def test_bad_controls_are_refused_everywhere(kw, code):
    c = controls(**kw)
    assert apply_rc(c=c) == code
    assert score_rc(ct=c) == code
    assert score_rc(cr=c) == code
    assert grad_rc(c=c) == code


@pytest.mark.parametrize("kw,code", [
    (dict(n_rows=-1), B.LPD_ERR_BAD_SIZE), (dict(vocab=0), B.LPD_ERR_BAD_SIZE),
    (dict(x=logits(None)), B.LPD_ERR_NULL_POINTER), (dict(x=logits(dtype=9)), B.LPD_ERR_BAD_DTYPE),
    (dict(x=logits(stride=39)), B.LPD_ERR_BAD_STRIDE), (dict(x=logits(FAKE + 1)), B.LPD_ERR_ALIGNMENT),
    (dict(out=None), B.LPD_ERR_NULL_POINTER), (dict(out_dtype=2), B.LPD_ERR_BAD_DTYPE),
    (dict(out_stride=39), B.LPD_ERR_BAD_STRIDE), (dict(out=FAKE + 0x10002), B.LPD_ERR_ALIGNMENT),
    (dict(out=FAKE), B.LPD_ERR_UNSUPPORTED),
])
def test_apply_and_gradient_refusals(kw, code):
    assert apply_rc(**kw) == code
    assert grad_rc(**kw) == code


def test_in_place_rules():
    # another type or stride in the same place; the gradient never in place
    assert apply_rc(out=FAKE, out_dtype=B.LPD_BF16, out_stride=48) == B.LPD_ERR_UNSUPPORTED
    assert grad_rc(out=FAKE, out_dtype=B.LPD_BF16) == B.LPD_ERR_UNSUPPORTED


@pytest.mark.parametrize("name", ["ids", "mask", "logp", "grad"])
def test_gradient_null_rows(name):
    assert grad_rc(**{name: None}) == B.LPD_ERR_NULL_POINTER


@pytest.mark.parametrize("kw,code", [
    (dict(met=None), B.LPD_ERR_NULL_POINTER), (dict(ids=None), B.LPD_ERR_NULL_POINTER),
    (dict(mask=None), B.LPD_ERR_NULL_POINTER), (dict(lo=1.3), B.LPD_ERR_BAD_CLIP), (dict(ws=None), B.LPD_ERR_WORKSPACE),
    (dict(ws_bytes=100), B.LPD_ERR_WORKSPACE), (dict(ws=WS + 16), B.LPD_ERR_ALIGNMENT),
])
def test_score_refusals(kw, code):
    assert score_rc(**kw) == code


def test_workspace_size():
    size = B.lpd_workspace_size
    assert size(B.LPD_KIND_CONTROLLED, 100, 0) == 0 and size(B.LPD_KIND_CONTROLLED, -1, 50) == 0
    assert 0 < size(B.LPD_KIND_CONTROLLED, 0, 50) < size(B.LPD_KIND_CONTROLLED, 1000, 50)
    assert size(B.LPD_KIND_CONTROLLED, 1000, 50) < size(B.LPD_KIND_CONTROLLED, 1000, 151936)
    need = size(B.LPD_KIND_CONTROLLED, 1000, 151936)
    assert score_rc(n_rows=1000, vocab=40, ws_bytes=size(B.LPD_KIND_CONTROLLED, 1000, 40) - 1) == B.LPD_ERR_WORKSPACE
    assert need % 256 == 0


def good():
    i, f = torch.int32, torch.float32
    return dict(history=torch.zeros(9, dtype=i), hist_begin=torch.zeros(4, dtype=torch.int64),
                hist_split=torch.zeros(4, dtype=torch.int64), hist_end=torch.zeros(4, dtype=torch.int64),
                repetition=torch.ones(4, dtype=f), scale=torch.ones(4, dtype=f),
                bias_ids=torch.zeros(4, 2, dtype=i), bias=torch.zeros(4, 2, dtype=f),
                mask=torch.zeros(3, 5, dtype=i), mask_row=torch.zeros(4, dtype=i))


@pytest.mark.parametrize("change", [
    dict(history=torch.zeros(9, dtype=torch.int64)), dict(scale=torch.ones(5)), dict(scale=torch.ones(8)[::2]),
    dict(repetition=torch.ones(4, dtype=torch.float64)), dict(hist_end=None), dict(bias=None),
    dict(bias=torch.zeros(4, 3)), dict(mask=torch.zeros(5, 3, dtype=torch.int32).t()),
    dict(mask=torch.zeros(5, dtype=torch.int32)), dict(mask_row=torch.zeros(4, dtype=torch.int64)),
])
def test_controls_object_checks_its_tensors(change):
    B.Controls(**good())
    with pytest.raises(ValueError):
        B.Controls(**{**good(), **change})


def test_binding_checks_shapes_and_memory():
    c = B.Controls(**good())
    x = torch.zeros(4, 160)
    with pytest.raises(ValueError, match="device memory"):
        B.lpd_controls_apply(x, c, torch.zeros(4, 160))
    with pytest.raises(ValueError, match="rows"):
        B.lpd_controls_apply(torch.zeros(3, 160), c, torch.zeros(3, 160))
    with pytest.raises(ValueError, match="shape"):
        B.lpd_controls_apply(x, c, torch.zeros(4, 150))
    ids, act = torch.zeros(4, dtype=torch.int32), torch.ones(4, dtype=torch.uint8)
    with pytest.raises(ValueError, match="token_ids"):
        B.lpd_score_controlled(x, x, c, c, ids.long(), act, 0.8, 1.2, None, None, None, None, None)
    with pytest.raises(ValueError, match="logp"):
        B.lpd_logprob_backward_controlled(x, c, ids, act, torch.zeros(3), torch.zeros(4), torch.zeros(4, 160))


def test_mask_of_one_row_passes_its_width():
    c = B.Controls(mask=torch.zeros(1, 7, dtype=torch.int32), mask_row=torch.zeros(4, dtype=torch.int32))
    assert c._struct.mask_stride == 7 and c._struct.n_masks == 1


def test_definition_by_hand():
    """Four tokens, every control, worked by hand."""
    c = {"history": np.array([0, 1, 1, 9], np.int32), "hist_begin": np.array([0]), "hist_split": np.array([1]),
         "hist_end": np.array([4]), "repetition": np.array([2.0]), "frequency": np.array([0.5]),
         "presence": np.array([0.25]), "scale": np.array([2.0]), "bias_ids": np.array([[2, 2, -1]]),
         "bias": np.array([[1.0, 0.5, 9.0]]), "mask": np.array([[0b0111]], np.int32), "mask_row": np.array([0])}
    z, slope = ref.row(c, np.array([4.0, -1.0, 1.0, 3.0]), 0)
    # 4 / 2; (-1 * 2 - 2 * 0.5 - 0.25); 1 + 1.5; masked; all times 2
    assert z.tolist() == [4.0, -6.5, 5.0, -np.inf]
    assert slope.tolist() == [1.0, 4.0, 2.0, 0.0]


@pytest.fixture
def recorded(monkeypatch):
    """The library's calls, by their arguments; nothing is launched."""
    calls = []

    class Recorder:
        def __getattr__(self, name):
            return lambda *a: calls.append((name, a)) or B.LPD_OK

    monkeypatch.setattr(B, "lib", lambda: Recorder())
    monkeypatch.setattr(B, "_on", lambda t: contextlib.nullcontext())
    return calls


def call_all(c, x):
    """Each controlled entry point once, on logits x."""
    n = x.shape[0]
    ids, act = torch.zeros(n, dtype=torch.int32), torch.ones(n, dtype=torch.uint8)
    f = torch.zeros(n)
    met, ws = torch.zeros(B.METRICS_BYTES, dtype=torch.uint8), torch.zeros(1 << 16, dtype=torch.uint8)
    return [lambda: B.lpd_controls_apply(x, c, torch.empty_like(x), stream=0),
            lambda: B.lpd_score_controlled(x, x, c, None, ids, act, 0.8, 1.2, f, f, f, met, ws, stream=0),
            lambda: B.lpd_score_controlled(x, x, None, c, ids, act, 0.8, 1.2, f, f, f, met, ws, stream=0),
            lambda: B.lpd_logprob_backward_controlled(x, c, ids, act, f, f, torch.empty_like(x), stream=0)]


def test_a_mask_slice_narrower_than_the_vocabulary_is_refused(recorded):
    """A slice keeps its rows' stride, which is what the library checks: the last row's words would be read
    behind the table."""
    table = torch.zeros(4, 10, dtype=torch.int32)
    c = B.Controls(mask=table[:, 5:])  # 5 words a row, 10 apart
    for call in call_all(c, torch.zeros(4, 161)):
        with pytest.raises(ValueError, match="words a row"):
            call()
    assert recorded == []
    for call in call_all(c, torch.zeros(4, 160)):
        call()
    assert len(recorded) == 4


def test_a_mask_table_of_no_rows_is_not_no_mask(recorded):
    """Its rows allow nothing; without mask_row it has too few rows."""
    table = torch.zeros(0, 5, dtype=torch.int32)
    x = torch.zeros(4, 160)
    for call in call_all(B.Controls(mask=table, mask_row=torch.zeros(4, dtype=torch.int32)), x):
        call()
    side = {"lpd_controls_apply": (1,), "lpd_score_controlled": (2, 3), "lpd_logprob_backward_controlled": (1,)}
    for name, args in recorded:
        c = next(args[k] for k in side[name] if args[k] is not None)._obj
        assert c.mask and c.n_masks == 0 and c.mask_stride == 5


def test_a_mask_table_of_no_rows_needs_mask_row():
    assert apply_rc(c=B.Controls(mask=torch.zeros(0, 2, dtype=torch.int32))._struct) == B.LPD_ERR_BAD_SIZE


def test_score_buffers_that_are_too_small_or_elsewhere_are_refused(recorded):
    """The library takes addresses: a repeated element's storage, a short record or another device's memory
    would be written past its end."""
    x, f = torch.zeros(4, 160), torch.zeros(4)
    ids, act = torch.zeros(4, dtype=torch.int32), torch.ones(4, dtype=torch.uint8)
    byte = lambda n, **kw: torch.zeros(n, dtype=torch.uint8, **kw)  # noqa: E731
    met, ws = byte(B.METRICS_BYTES), byte(1 << 16)

    def call(met, ws):
        B.lpd_score_controlled(x, x, None, None, ids, act, 0.8, 1.2, f, f, f, met, ws, stream=0)

    for bad in (byte(B.METRICS_BYTES - 1), byte(1).expand(B.METRICS_BYTES), byte(2 * B.METRICS_BYTES)[::2],
                byte(B.METRICS_BYTES, device="meta")):
        with pytest.raises(ValueError, match="out_metrics"):
            call(bad, ws)
    for bad in (byte(1).expand(1 << 16), byte(1 << 17)[::2], byte(1 << 16, device="meta")):
        with pytest.raises(ValueError, match="workspace"):
            call(met, bad)
    assert recorded == []
    call(met, ws.view(torch.float32))
    assert recorded[0][1][-2] == 1 << 16
    call(None, None)  # (NULL: the library's to refuse)
