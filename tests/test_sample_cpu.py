"""The sampling calls' host side: arguments that are refused before anything is
launched (fake device addresses, no GPU), the definition that the GPU tests use
against hand-worked values, and the weights' arithmetic compiled for the host."""
import ctypes
import math
import shutil
import subprocess
from pathlib import Path

import numpy as np
import pytest
import torch

from tests import sample_ref as ref
from logprob_drift_scoring_gb300 import binding as B

FAKE = 0x7F0000000000
ROOT = Path(__file__).resolve().parent.parent


def logits(ptr=FAKE, dtype=B.LPD_BF16, stride=40):
    return B.LpdLogits(ptr, dtype, 0, stride)


def sample_rc(x=None, f=None, n_rows=8, vocab=40, u=FAKE, ids=FAKE, logp=FAKE, kept=FAKE):
    x = x or logits()
    return B.lib().lpd_sample(ctypes.byref(x), ctypes.byref(f) if f else None, n_rows, vocab, u, ids, logp, kept, None)


def mask_rc(x=None, f=None, n_rows=8, vocab=40, ids=FAKE, act=FAKE, mask=FAKE, stride=2, lse=FAKE, kept=FAKE):
    x = x or logits()
    return B.lib().lpd_filter_mask(ctypes.byref(x), ctypes.byref(f) if f else None, n_rows, vocab, ids, act, mask,
                                   stride, lse, kept, None)


SHARED = [
    (dict(n_rows=-1), B.LPD_ERR_BAD_SIZE), (dict(vocab=0), B.LPD_ERR_BAD_SIZE),
    (dict(x=logits(None)), B.LPD_ERR_NULL_POINTER), (dict(x=logits(dtype=B.LPD_E4M3)), B.LPD_ERR_BAD_DTYPE),
    (dict(x=logits(stride=39)), B.LPD_ERR_BAD_STRIDE), (dict(x=logits(FAKE + 1)), B.LPD_ERR_ALIGNMENT),
    (dict(x=logits(FAKE + 2, B.LPD_F32)), B.LPD_ERR_ALIGNMENT),
    (dict(x=logits(stride=1 << 20), vocab=B.LPD_SAMPLE_MAX_VOCAB + 1, ), B.LPD_ERR_UNSUPPORTED),
    (dict(n_rows=1 << 29), B.LPD_ERR_UNSUPPORTED),
    (dict(f=B.LpdFilter(FAKE + 2, None, None, None)), B.LPD_ERR_ALIGNMENT),
    (dict(f=B.LpdFilter(None, FAKE + 1, None, None)), B.LPD_ERR_ALIGNMENT),
    (dict(f=B.LpdFilter(None, None, FAKE + 2, None)), B.LPD_ERR_ALIGNMENT),
    (dict(f=B.LpdFilter(None, None, None, FAKE + 3)), B.LPD_ERR_ALIGNMENT),
    (dict(kept=FAKE + 2), B.LPD_ERR_ALIGNMENT),
]


@pytest.mark.parametrize("kw,code", SHARED)
def test_refused_by_both(kw, code):
    assert sample_rc(**kw) == code
    assert mask_rc(**{"stride": 1 << 20, **kw}) == code


@pytest.mark.parametrize("kw,code", [(dict(u=None), B.LPD_ERR_NULL_POINTER), (dict(ids=None), B.LPD_ERR_NULL_POINTER),
                                     (dict(u=FAKE + 2), B.LPD_ERR_ALIGNMENT), (dict(ids=FAKE + 2), B.LPD_ERR_ALIGNMENT),
                                     (dict(logp=FAKE + 1), B.LPD_ERR_ALIGNMENT)])
def test_sample_refuses(kw, code):
    assert sample_rc(**kw) == code


@pytest.mark.parametrize("kw,code", [(dict(mask=None), B.LPD_ERR_NULL_POINTER), (dict(stride=1), B.LPD_ERR_BAD_STRIDE),
                                     (dict(mask=FAKE + 2), B.LPD_ERR_ALIGNMENT), (dict(ids=FAKE + 1), B.LPD_ERR_ALIGNMENT),
                                     (dict(lse=FAKE + 2), B.LPD_ERR_ALIGNMENT)])
def test_mask_refuses(kw, code):
    assert mask_rc(**kw) == code


def test_no_rows_is_no_work():
    assert sample_rc(x=logits(None), n_rows=0, u=None, ids=None, logp=None, kept=None) == B.LPD_OK
    assert mask_rc(x=logits(None), n_rows=0, ids=None, act=None, mask=None, lse=None, kept=None) == B.LPD_OK


def test_binding_refuses():
    f = torch.ones(4)
    with pytest.raises(ValueError):
        B.Filter(scale=f.double())
    with pytest.raises(ValueError):
        B.Filter(top_k=f)
    with pytest.raises(ValueError):
        B.Filter(scale=f, top_p=torch.ones(3))
    with pytest.raises(ValueError):
        B.Filter(scale=torch.ones(8)[::2])
    x, ok = torch.zeros(4, 40), B.Filter(scale=f)
    ids, mask = torch.zeros(4, dtype=torch.int32), torch.zeros(4, 2, dtype=torch.int32)
    for args in ((x, ok, f, ids), (x.T, None, f, ids), (x, B.Filter(scale=torch.ones(5)), f, ids),
                 (x, ok, torch.ones(3), ids), (x, ok, f, ids.long())):
        with pytest.raises(ValueError):  # (host tensors, where everything else fits)
            B.lpd_sample(*args)
    for args in ((x, ok, None, None, mask), (x, ok, None, None, mask[:, :1]), (x, ok, None, None, mask.float()),
                 (x, ok, f, None, mask), (x, ok, None, f, mask), (x, ok, None, None, torch.zeros(2, 4, dtype=torch.int32).T)):
        with pytest.raises(ValueError):
            B.lpd_filter_mask(*args)


def test_definition_by_hand():
    x = np.log([1.0, 4.0, 2.0, 4.0, 1.0])
    kept = lambda **kw: list(np.nonzero(ref.row(x, **kw)[1])[0])  # noqa: E731
    assert kept() == [0, 1, 2, 3, 4]
    assert kept(top_k=1) == [1] and kept(top_k=2) == [1, 3] and kept(top_k=4) == [0, 1, 2, 3]
    assert kept(top_p=0.3) == [1] and kept(top_p=0.5) == [1, 3] and kept(top_p=0.7) == [1, 2, 3] and kept(top_p=0.0) == [1]
    assert kept(min_p=0.4) == [1, 2, 3] and kept(min_p=1.0) == [1, 3] and kept(min_p=5.0) == [1, 3]
    assert kept(top_k=3, top_p=0.79) == [1, 3] and kept(top_k=3, top_p=0.81) == [1, 2, 3]
    assert kept(min_p=0.4, top_p=0.85) == [1, 2, 3]
    z, k, _ = ref.row(x, top_k=3)
    assert [ref.draw(z, k, u)[0] for u in (0.0, 0.39, 0.41, 0.59, 0.61, 0.99)] == [1, 1, 2, 2, 3, 3]
    assert math.isclose(ref.draw(z, k, 0.5)[1], math.log(0.2), rel_tol=1e-12)
    assert ref.row([np.nan, 1.0]) is None and ref.row([np.inf, 1.0]) is None and ref.row([-np.inf] * 3) is None
    assert ref.row(x, scale=0.0) is None and ref.row(x, top_p=math.nan) is None
    assert list(ref.row([-np.inf, 0.0, -np.inf])[1]) == [False, True, False]


def test_weights_compiled_for_the_host(tmp_path):
    """The weights against long double: a rough one is off by the table's rounding,
    its correction's and one of the argument's (2^-31 each at the mantissa's lower
    end, 2^-32 of the argument times ln 2), so below 2^-29.5, plus a step of 2^-44
    (shifts cut off).  A precise one: three roundings of terms below 2^-20 (2^-44
    each), those of two parts to steps of 2^-44, so below 2^-41 of a weight that is
    1/2 at least, that step, and the argument's lower part, at most 2^-23 of the
    units that x lies from 0, rounded by 2^-24 of itself (times ln 2 / 256: 2^-55)."""
    if not shutil.which("g++"):
        pytest.skip("g++ not found")
    (tmp_path / "w.cpp").write_text(r'''
#include "lpd_weights.cuh"
#include <cstdio>
#include <random>
using namespace lpd;
int main() {
    WeightEntry rough[kUnits];
    uint64_t precise[kUnits];
    for (int i = 0; i < kUnits; ++i) {
        const long double v = exp2l((long double)i / kUnits);
        rough[i].whole = (uint32_t)llroundl(v * 1073741824.0L);
        rough[i].part = (float)(v * 1073741824.0L);
        precise[i] = (uint64_t)llroundl(v * 4611686018427387904.0L);
    }
    std::mt19937_64 g(1);
    std::uniform_real_distribution<double> u(0, 1);
    int bad = 0;
    for (float scale : {1e-20f, 0.01f, 0.7f, 1.f, 1.3f, 10.f, 1000.f, 1e20f})
        for (float top : {13.5f, -3.1f, 0.001f, 300.f, 0.f, -70000.f}) {
            const WeightScale w = weight_scale(scale, top);
            for (int k = 0; k < 20000; ++k) {
                float x = (float)(top - u(g) * 33 / scale);
                if (k % 7 == 0) x = (float)(top * u(g) * 1e-4);
                if (k == 1) x = top;
                if (!(x <= top) || !std::isfinite(x)) continue;
                const long double at = w.wide ? ((long double)x - top) * w.c : (long double)x * w.c - w.origin;
                const long double want = at < -48 * kUnits ? 0 : ldexpl(exp2l(at / kUnits), kWeightOne);
                const long double p = weight_precise(x, w, top, precise);
                const long double far = w.wide ? 0 : fabsl((long double)x * w.c);
                if (fabsl(p - want) > want * (ldexpl(1, -41) + far * ldexpl(1, -55)) + 1.01L) ++bad;
                if (w.wide || !(x > w.cut)) continue;
                const long double r = weight_rough(x, w, rough);
                if (fabsl(r - want) > want * ldexpl(1, -29) * 0.71L + 1.01L) ++bad;
            }
        }
    printf("%d\n", bad);
}
''')
    csrc = ROOT / "logprob_drift_scoring_gb300" / "csrc"
    subprocess.run(["g++", "-O2", "-std=c++17", "-ffp-contract=off", f"-I{csrc}", "-o", str(tmp_path / "w"),
                    str(tmp_path / "w.cpp")], check=True)
    assert subprocess.run([str(tmp_path / "w")], check=True, capture_output=True, text=True).stdout.strip() == "0"


def test_light_weights_lose_less_than_2_45_of_the_top(tmp_path):
    """Weights of the lowest 16 octaves against long double: a step of 2^-45 of the top's
    beside the errors of a rough and of a precise weight (the bounds above).  The steps are
    taken in the units of the weights' origin, 2^(1 / 512) off the top at most."""
    if not shutil.which("g++"):
        pytest.skip("g++ not found")
    (tmp_path / "w.cpp").write_text(r'''
#include "lpd_weights.cuh"
#include <cstdio>
#include <random>
using namespace lpd;
int main() {
    WeightEntry rough[kUnits];
    uint64_t precise[kUnits];
    for (int i = 0; i < kUnits; ++i) {
        const long double v = exp2l((long double)i / kUnits);
        rough[i].whole = (uint32_t)llroundl(v * 1073741824.0L);
        rough[i].part = (float)(v * 1073741824.0L);
        precise[i] = (uint64_t)llroundl(v * 4611686018427387904.0L);
    }
    std::mt19937_64 g(1);
    std::uniform_real_distribution<double> u(0, 1);
    int bad = 0;
    for (float scale : {0.01f, 0.7f, 1.f, 30.f})
        for (float top : {13.5f, -3.1f, 0.f}) {
            const WeightScale w = weight_scale(scale, top);
            for (int k = 0; k < 200000; ++k) {
                const float x = (float)(top - (19.5 + u(g) * 12.5) / scale);
                const long double want = exp2l(((long double)x * w.c - w.origin) / kUnits);
                const long double p = ldexpl(weight_precise(x, w, top, precise), -kWeightOne) - want;
                const long double r = (x > w.cut ? ldexpl(weight_rough(x, w, rough), -kWeightOne) : 0) - want;
                const long double most = want * ldexpl(1, -29) + ldexpl(1.01L, -45);
                if (fabsl(p) > most || fabsl(r) > most) ++bad;
            }
        }
    printf("%d\n", bad);
}
''')
    csrc = ROOT / "logprob_drift_scoring_gb300" / "csrc"
    subprocess.run(["g++", "-O2", "-std=c++17", "-ffp-contract=off", f"-I{csrc}", "-o", str(tmp_path / "w"),
                    str(tmp_path / "w.cpp")], check=True)
    assert subprocess.run([str(tmp_path / "w")], check=True, capture_output=True, text=True).stdout.strip() == "0"
