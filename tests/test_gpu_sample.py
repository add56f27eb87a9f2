"""Sampling and filter masks on the GPU (needs a GPU) against the float64 definition
in sample_ref.py.

Bounds.  A weight is off by less than 2^-29.5 of itself, so is every sum, and a
border (top-p, or the draw's) can only be another where the definition's own lies
within 2^-28 of the whole mass from a sum: such rows are left out of the comparison
of sets and tokens (one in 2^28 times the number of kept tokens).  The logarithm of a sum is off
by 2^-29 and the result is rounded to float32: 2^-24 of itself.
"""
import subprocess
import sys
from pathlib import Path

import numpy as np
import pytest
import torch

from tests import sample_ref as ref
from logprob_drift_scoring_gb300 import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda"
ROOT = Path(__file__).resolve().parent.parent
KINDS = {"bf16": torch.bfloat16, "f32": torch.float32}
NEAR = 2.0 ** -28


def tensor(x, kind, pad=0):
    t = torch.from_numpy(np.asarray(x, dtype=np.float32)).to(DEV).to(KINDS[kind])
    if pad:
        wide = torch.full((t.shape[0], t.shape[1] + pad), float("nan"), dtype=t.dtype, device=DEV)
        wide[:, :t.shape[1]] = t
        t = wide[:, :t.shape[1]]
    return t


def host(t):
    return t.float().cpu().numpy().astype(np.float64)


def params(rng, rows, vocab):
    """Every kind of request among the rows."""
    kind = rng.integers(0, 8, rows)
    k = np.where(np.isin(kind, (1, 5)), rng.integers(1, 80, rows), 0)
    k = np.where(kind == 0, 1, np.where(kind == 6, rng.integers(1, vocab + 2, rows), k))
    p = np.where(np.isin(kind, (2, 5, 6)), rng.uniform(0.05, 0.999, rows), np.where(kind == 7, rng.choice([0.0, 1e-6, 0.999999, 1.0], rows), 1.0))
    m = np.where(np.isin(kind, (3, 5)), rng.uniform(0.001, 0.4, rows), 0.0)
    return dict(scale=rng.uniform(0.5, 2.0, rows).astype(np.float32), min_p=m.astype(np.float32),
                top_k=k.astype(np.int32), top_p=p.astype(np.float32))


def to_filter(f):
    return B.Filter(**{k: torch.from_numpy(np.ascontiguousarray(v)).to(DEV) for k, v in f.items()})


def logits(rng, rows, vocab, peak=14.0):
    x = rng.normal(0, 1.5, (rows, vocab))
    for r in range(rows):
        x[r, rng.integers(0, vocab, 40)] += peak * rng.uniform(0, 1, 40)
    return x


def check(x, f, u, keep=None, active=None):
    """Both calls on the same rows against the definition."""
    n, vocab = x.shape
    xh = host(x)
    filt = to_filter(f) if f else None
    ids, logp, kept = B.sample(x, torch.from_numpy(u.astype(np.float32)).to(DEV), filt)
    mask, lse, mkept = B.filter_mask(x, filt, None if keep is None else torch.from_numpy(keep.astype(np.int32)).to(DEV),
                                     None if active is None else torch.from_numpy(active.astype(np.uint8)).to(DEV))
    torch.cuda.synchronize()
    ids, logp, kept, mask, lse, mkept = (t.cpu().numpy() for t in (ids, logp, kept, mask, lse, mkept))
    got = ref.bits(mask, mask.shape[1] * 32)
    assert not got[:, vocab:].any()
    got = got[:, :vocab]
    compared = 0
    for r in range(n):
        want = ref.row(xh[r], **{k: float(v[r]) if k != "top_k" else int(v[r]) for k, v in (f or {}).items()})
        live = active is None or active[r]
        if want is None:
            compared += 1
            assert ids[r] == -1 and np.isnan(logp[r]) and kept[r] == 0, r
            assert not got[r].any() and mkept[r] == 0 and (np.isnan(lse[r]) if live else lse[r] == 0), r
            continue
        z, k, margin = want
        if not live:
            assert not got[r].any() and mkept[r] == 0 and lse[r] == 0, r
        if margin < NEAR:
            continue
        compared += 1
        assert kept[r] == k.sum(), (r, kept[r], k.sum())
        j, lp, near = ref.draw(z, k, float(np.float32(u[r])))
        if near >= NEAR:
            assert ids[r] == j, (r, ids[r], j)
            assert abs(logp[r] - lp) <= 2.0 ** -24 * abs(lp) + 2.0 ** -28 + 2.0 ** -52 * np.abs(z[k]).max(), (r, logp[r], lp)
        if not live:
            continue
        forced = k.copy()
        if keep is not None and 0 <= keep[r] < vocab and np.isfinite(xh[r, keep[r]]):
            forced[keep[r]] = True
        assert np.array_equal(got[r], forced), (r, np.nonzero(got[r] != forced)[0][:8])
        assert mkept[r] == forced.sum(), r
        want_lse = ref.lse(z, forced)
        if abs(want_lse) > np.finfo(np.float32).max:  # (half a step of float32 past its range is infinity)
            assert np.isinf(lse[r]) and np.sign(lse[r]) == np.sign(want_lse)
            continue
        assert abs(lse[r] - want_lse) <= 2.0 ** -24 * abs(want_lse) + 2.0 ** -28 + 2.0 ** -52 * np.abs(z[forced]).max(), (r, lse[r], want_lse)
    assert compared >= n * 0.9 - 1
    return ids, kept


# so few that clusters take them, and so many that a CTA takes each
ROWS = [24, 136]


@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("vocab,pad", [(1, 0), (2, 1), (31, 0), (32, 3), (33, 7), (64, 0), (65, 0), (1000, 8), (1024, 0),
                                       (2049, 5), (8193, 7), (20011, 1), (50021, 1), (131077, 3)])
def test_sizes(vocab, pad, kind, rows):
    rng = np.random.default_rng(vocab)
    check(tensor(logits(rng, rows, vocab), kind, pad), params(rng, rows, vocab), rng.uniform(0, 1, rows),
          keep=rng.integers(-1, vocab + 1, rows), active=rng.uniform(0, 1, rows) < 0.8)


@pytest.mark.parametrize("kind,vocab", [("f32", 262208), ("f32", B.LPD_SAMPLE_MAX_VOCAB), ("bf16", B.LPD_SAMPLE_MAX_VOCAB)])
def test_largest_vocabularies(kind, vocab):
    rng = np.random.default_rng(7)
    check(tensor(logits(rng, 9, vocab), kind), params(rng, 9, vocab), rng.uniform(0, 1, 9))


@pytest.mark.parametrize("rows", [1, 2, 40, 300, 1000])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_rows(rows, kind):
    """The number of rows decides over how many CTAs each is spread."""
    rng = np.random.default_rng(rows)
    check(tensor(logits(rng, rows, 9001), kind), params(rng, rows, 9001), rng.uniform(0, 1, rows))


@pytest.mark.parametrize("rows", [32, 136])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("peak", [0.0, 3.0])
def test_flat_rows(peak, kind, rows):
    """Nuclei of most of the vocabulary: the borders lie below every list."""
    rng = np.random.default_rng(11)
    vocab = 60013
    f = params(rng, rows, vocab)
    f["top_k"][::4] = rng.integers(2000, vocab, rows // 4)
    f["top_p"][1::4] = rng.uniform(0.5, 0.9999, rows // 4)
    f["min_p"][2::8] = 1e-4
    check(tensor(rng.normal(0, 0.7, (rows, vocab)) + peak, kind), f, rng.uniform(0, 1, rows))


@pytest.mark.parametrize("rows", [30, 135])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("vocab", [7, 700, 30011])
def test_ties(vocab, kind, rows):
    """Rows of one value, of a few values, and of both zeros: ties go by token."""
    rng = np.random.default_rng(vocab)
    x = np.round(rng.normal(0, 1.5, (rows, vocab)))
    x[::5] = 2.5
    x[1::5] = np.where(rng.uniform(0, 1, (rows // 5, vocab)) < 0.5, 0.0, -0.0)
    f = params(rng, rows, vocab)
    f["top_k"][::3] = rng.integers(1, vocab + 1, rows // 3)
    f["top_p"][1::3] = rng.uniform(0, 1, rows // 3)
    f["scale"][:] = np.where(np.arange(rows) % 2, 1.0, f["scale"])
    # (equal weights: every sum is a whole number of them, so keep the borders between two)
    n_top = (x == x.max(1, keepdims=True)).sum(1)
    f["top_p"] = np.where((f["top_p"] > 0) & (f["top_p"] < 1), np.minimum((np.floor(f["top_p"] * n_top) + 0.4) / n_top, 0.9999), f["top_p"]).astype(np.float32)
    check(tensor(x, kind), f, rng.uniform(0, 1, rows))


@pytest.mark.parametrize("rows", [40, 136])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_masked_logits_and_rows_without_a_distribution(kind, rows):
    rng = np.random.default_rng(5)
    vocab = 20011
    x = logits(rng, rows, vocab)
    x[rng.uniform(0, 1, x.shape) < 0.9] = -np.inf
    x[3] = -np.inf
    x[4], x[4, 777] = -np.inf, -3.0
    x[5, 20010] = np.nan
    x[6, 0] = np.inf
    x[7, 5000:] = -np.inf
    x[8] = np.where(np.isfinite(x[8]), -3.38e38, x[8])
    x[9, :] = torch.finfo(torch.bfloat16).min
    x[9, 11] = 1.0
    f = params(rng, rows, vocab)
    f["scale"][10:15] = [0.0, -1.0, np.nan, np.inf, 1.0]
    f["top_p"][14], f["min_p"][15] = np.nan, np.nan
    check(tensor(x, kind), f, rng.uniform(0, 1, rows), keep=rng.integers(0, vocab, rows))


@pytest.mark.parametrize("rows", [16, 136])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("scale", [1e-30, 1e-6, 0.01, 50.0, 3000.0, 1e9, 1e30])
@pytest.mark.parametrize("offset", [0.0, 1000.0, -300.0, 30000.0])
def test_extreme_scales_and_offsets(scale, offset, kind, rows):
    rng = np.random.default_rng(9)
    vocab = 5003
    f = params(rng, rows, vocab)
    f["scale"] = np.full(rows, scale, dtype=np.float32)
    check(tensor(rng.normal(0, 2, (rows, vocab)) + offset, kind), f, rng.uniform(0, 1, rows))


@pytest.mark.parametrize("rows", [16, 136])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("scale,spread", [(1.5e-45, 2.0), (3.4e38, 2.0), (1.0, 8e37), (3.4e38, 8e37), (1.5e-45, 8e37)])
def test_ends_of_the_range(scale, spread, kind, rows):
    """The smallest and largest scales, and logits whose differences leave float32."""
    rng = np.random.default_rng(10)
    vocab = 3001
    f = params(rng, rows, vocab)
    f["scale"] = np.full(rows, scale, dtype=np.float32)
    check(tensor(np.clip(rng.normal(0, spread, (rows, vocab)), -3.3e38, 3.3e38), kind), f, rng.uniform(0, 1, rows))


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_values_next_to_zero_and_lowest_masks(kind):
    """Rows whose border, or top, lies within 2^-10 of 0, rows masked with the type's
    lowest value, and rows of float32 values that bf16 has."""
    rng = np.random.default_rng(13)
    rows, vocab = 140, 9000
    x = rng.normal(0, 1, (rows, vocab))
    x[:70] *= 1e-4
    x[40:70] -= 3.0
    x[40:70, :50] = rng.normal(0, 1e-5, (30, 50))
    x[70:100, 1000:] = float(torch.finfo(torch.bfloat16).min)
    x[100:120, ::2] = -20000.0
    x = torch.from_numpy(x).to(torch.bfloat16).float().numpy() if kind == "f32" else x
    f = params(rng, rows, vocab)
    f["top_k"][70:90:3] = rng.integers(900, vocab, 7)
    check(tensor(x, kind), f, rng.uniform(0, 1, rows))


def test_uniforms_at_the_ends():
    rng = np.random.default_rng(2)
    vocab = 4001
    x = np.repeat(logits(rng, 1, vocab), 7, 0)
    u = np.array([0.0, -1.0, 1.0, 2.0, np.nan, 1 - 2.0 ** -24, 2.0 ** -149], dtype=np.float32)
    ids, logp, kept = B.sample(tensor(x, "f32"), torch.from_numpy(u).to(DEV), to_filter(dict(top_k=np.full(7, 5, np.int32))))
    ids, logp, kept = ids.cpu().numpy(), logp.cpu().numpy(), kept.cpu().numpy()
    top = np.sort(np.argsort(-host(tensor(x, "f32"))[0], kind="stable")[:5])
    assert list(ids) == [top[0], top[0], top[-1], top[-1], -1, top[-1], top[0]]
    assert np.isnan(logp[4]) and np.isfinite(logp[[0, 1, 2, 3, 5, 6]]).all() and (kept[[0, 1, 2, 3, 5, 6]] == 5).all()


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [1, 200])
def test_tokens_that_are_nearly_certain(rows, kind):
    """A token alone has the logprob 0; next to 1 the others' share keeps its digits:
    2^-29 of it and the steps of 2^-44 that each of the others may lose."""
    rng = np.random.default_rng(rows)
    vocab = 5000
    x = rng.normal(0, 0.3, (rows, vocab))
    x[:, 77] = 18.0
    t = tensor(x, kind)
    ids, logp, kept = B.sample(t, torch.full((rows,), 0.5, device=DEV), to_filter(dict(top_k=np.ones(rows, np.int32))))
    assert bool((ids == 77).all()) and bool((logp == 0).all()) and bool((kept == 1).all())
    ids, logp, kept = B.sample(t, torch.full((rows,), 0.5, device=DEV))
    xh = host(t)
    others = np.exp(xh - xh[:, 77:78]).sum(1) - 1
    got = logp.cpu().numpy().astype(np.float64)
    assert bool((ids == 77).all())
    assert np.all(np.abs(got + np.log1p(others)) <= (2.0 ** -23 + 2.0 ** -29) * others + vocab * 2.0 ** -44)


def test_no_filter_and_outputs_left_out():
    rng = np.random.default_rng(3)
    x = tensor(logits(rng, 6, 3001), "bf16", 7)
    check(x, None, rng.uniform(0, 1, 6))
    u = torch.rand(6, device=DEV)
    ids, _, _ = B.sample(x, u)
    only = torch.full((6,), 99, dtype=torch.int32, device=DEV)
    B.lpd_sample(x, None, u, only)
    assert torch.equal(ids, only)
    mask, _, _ = B.filter_mask(x, None)
    wide = torch.full((6, 101), 77, dtype=torch.int32, device=DEV)
    B.lpd_filter_mask(x, None, None, None, wide)
    assert torch.equal(wide[:, :94], mask) and bool((wide[:, 94:] == 77).all())


def test_a_row_does_not_depend_on_its_batch():
    rng = np.random.default_rng(4)
    vocab, rows = 33007, 400
    x = tensor(logits(rng, rows, vocab, 8.0), "bf16")
    f = params(rng, rows, vocab)
    u = torch.rand(rows, device=DEV)
    ids, logp, kept = B.sample(x, u, to_filter(f))
    for r in range(0, rows, 37):
        one = to_filter({k: v[r:r + 1] for k, v in f.items()})
        for got, want in zip(B.sample(x[r:r + 1], u[r:r + 1], one), (ids, logp, kept)):
            assert torch.equal(got, want[r:r + 1])


@pytest.mark.parametrize("rows", [3, 150])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_rows_far_apart(kind, rows):
    """Offsets beyond 32 bits, of logits and of masks: the bits of the same rows side by side."""
    rng = np.random.default_rng(12)
    vocab, words = 5003, 157
    x = tensor(logits(rng, rows, vocab), kind)
    f = to_filter(params(rng, rows, vocab))
    u = torch.rand(rows, device=DEV)
    far = (2 ** 31 + 2 ** 20) // (rows - 1) // 8 * 8 + 8  # (the last row lies behind 2^31 elements)
    room = torch.empty(far * (rows - 1) + vocab, dtype=x.dtype, device=DEV)
    y = room.as_strided((rows, vocab), (far, 1))
    y.copy_(x)
    bits = torch.empty(far * (rows - 1) + words, dtype=torch.int32, device=DEV)
    mask = bits.as_strided((rows, words), (far, 1))
    for got, want in zip(B.sample(y, u, f), B.sample(x, u, f)):
        assert torch.equal(got, want)
    B.lpd_filter_mask(y, f, None, None, mask)
    assert torch.equal(mask, B.filter_mask(x, f)[0])


def test_first_call_is_captured():
    """In a process that has called nothing yet."""
    code = """
import torch
from logprob_drift_scoring_gb300 import binding as B
x = torch.randn(200, 5003, device="cuda").bfloat16()
u = torch.rand(200, device="cuda")
ids = torch.empty(200, dtype=torch.int32, device="cuda")
mask = torch.empty(200, 157, dtype=torch.int32, device="cuda")
g, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
torch.cuda.synchronize()
with torch.cuda.stream(side), torch.cuda.graph(g, stream=side):
    B.lpd_sample(x, None, u, ids)
    B.lpd_filter_mask(x, None, ids, None, mask)
g.replay()
torch.cuda.synchronize()
assert torch.equal(ids, B.sample(x, u)[0]) and torch.equal(mask, B.filter_mask(x, None)[0])
"""
    done = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert done.returncode == 0, done.stderr[-2000:]


def test_repeated_streams_and_graph():
    """The same bits each time, on two streams at once, and replayed with new inputs."""
    rng = np.random.default_rng(8)
    rows, vocab = 64, 40009
    x = tensor(logits(rng, rows, vocab), "bf16")
    filt = to_filter(params(rng, rows, vocab))
    u = torch.rand(rows, device=DEV)
    want = B.sample(x, u, filt)
    wmask = B.filter_mask(x, filt)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for _ in range(3):
        for s in streams:
            with torch.cuda.stream(s):
                got.append((B.sample(x, u, filt), B.filter_mask(x, filt)))
    torch.cuda.synchronize()
    for a, b in got:
        assert all(torch.equal(p, q) for p, q in zip(a, want)) and all(torch.equal(p, q) for p, q in zip(b, wmask))
    ids, logp, kept = (torch.empty_like(t) for t in want)
    mask, lse, mkept = (torch.empty_like(t) for t in wmask)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        B.lpd_sample(x, filt, u, ids, logp, kept)
        with torch.cuda.graph(g, stream=side):
            B.lpd_sample(x, filt, u, ids, logp, kept)
            B.lpd_filter_mask(x, filt, ids, None, mask, lse, mkept)
    torch.cuda.synchronize()
    x.copy_(tensor(logits(np.random.default_rng(9), rows, vocab), "bf16"))
    u.copy_(torch.rand(rows, device=DEV))
    g.replay()
    torch.cuda.synchronize()
    want = B.sample(x, u, filt)
    assert all(torch.equal(p, q) for p, q in zip((ids, logp, kept), want))
    assert all(torch.equal(p, q) for p, q in zip((mask, lse, mkept), B.filter_mask(x, filt, ids)))


def test_filtered_rollout_scored_under_its_own_sets():
    """Sampled, masked, scored and differentiated: the scorer's rollout logprob is the
    sampler's, and the gradient that of the filtered softmax."""
    rng = np.random.default_rng(6)
    rows, vocab = 48, 12007
    x = tensor(logits(rng, rows, vocab), "bf16")
    train = (x.float() + 1e-2 * torch.randn(rows, vocab, device=DEV)).to(torch.bfloat16)
    f = params(rng, rows, vocab)
    filt = to_filter(f)
    ids, logp, kept = B.sample(x, torch.rand(rows, device=DEV), filt)
    mask, lse, mkept = B.filter_mask(x, filt, ids)
    assert torch.equal(kept, mkept)
    c = B.Controls(scale=filt.scale, mask=mask)
    active = torch.ones(rows, dtype=torch.uint8, device=DEV)
    res = B.score_controlled(train, x, ids, active, train_controls=c, rollout_controls=c)
    assert res.metrics["status"] == 0 and res.metrics["n_active"] == rows
    # (the scorer's own bound: 1e-5 and float32's rounding, as derived in test_gpu_controls.py)
    assert torch.all((res.logp_rollout - logp).abs() <= 1.1e-5 + 2.0 ** -23 * logp.abs())
    grad = torch.ones(rows, device=DEV)
    dx = torch.empty(rows, vocab, device=DEV)
    B.lpd_logprob_backward_controlled(train, c, ids, active, res.logp_train, grad, dx)
    got, th = host(dx), host(train)
    bits = ref.bits(mask.cpu().numpy(), vocab)
    for r in range(0, rows, 5):
        s = float(f["scale"][r])
        z = np.where(bits[r], th[r] * s, -np.inf)
        p = np.exp(z - z.max())
        p /= p.sum()
        want = -s * p
        want[int(ids[r])] += s
        assert np.all(np.abs(got[r] - want) <= s * (2e-5 * p + 2.0 ** -22)), r


@pytest.mark.parametrize("rows", [16, 136])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("scale,log_min_p", [
    (0.004, -65.81875),  # the bound lies at -16454.7: -16384 is the next bf16 value that it leaves
    (0.004, -65.536),    # at -16384 itself, or by the logarithm's rounding a little beside it
    (0.002, -33.0),      # at -16500
    (0.002, -32.8),      # at -16400
    (0.004, -66.1),      # at -16525: -16512 is left too
])
def test_min_p_next_to_the_lowest_values_that_are_counted(scale, log_min_p, kind, rows):
    """Bounds at and around -2^14, with tokens on both sides: how many are kept."""
    rng = np.random.default_rng(17)
    vocab = 5003
    x = rng.normal(-3000, 700, (rows, vocab))
    x[:, ::3] = rng.choice([-16256.0, -16320.0, -16384.0, -16512.0, -16640.0, -20000.0, -3e38], (rows, len(range(0, vocab, 3))))
    x[:, 7] = 0.0
    x[1::4] = np.where(x[1::4] <= -16384, -np.inf, x[1::4])  # (and rows without any)
    x[2::4, ::3] = -20000.0
    f = dict(scale=np.full(rows, scale, np.float32), min_p=np.full(rows, np.exp(log_min_p), np.float32))
    u = rng.uniform(0, 1, rows)
    t = tensor(x, kind)
    ids, kept = check(t, f, u)
    xh = host(t)
    for r in range(rows):  # (every row, none left out)
        want = ref.row(xh[r], float(f["scale"][r]), float(f["min_p"][r]))[1].sum()
        assert kept[r] == want, (r, kept[r], want)


@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("vocab", [40, 5003, 60013])
@pytest.mark.parametrize("form", ["none", "top-k", "min-p", "all", "nucleus"])
def test_uniforms_at_the_ends_of_sets_with_unlikely_tokens(form, vocab, kind, rows):
    """0 and less draw the first kept token and 1 and more the last, however little they weigh."""
    rng = np.random.default_rng(19)
    x = rng.normal(0, 0.3, (rows, vocab))
    x[:, :3], x[:, -2:] = -np.inf, -np.inf
    x[:, 3], x[:, 4], x[:, -3], x[:, -4] = -70.0, -50.0, -60.0, -34.0
    x[::2, 3], x[::2, -3] = -40.0, -33.0
    f = dict(none={}, **{"top-k": dict(top_k=np.full(rows, min(vocab - 6, 400), np.int32)),
                         "min-p": dict(min_p=np.full(rows, 1e-25, np.float32)),
                         "all": dict(min_p=np.full(rows, 1e-30, np.float32), top_k=np.full(rows, vocab - 7, np.int32)),
                         "nucleus": dict(top_p=np.full(rows, 0.99, np.float32))})[form]
    u = np.array([0.0, -1.0, 1.0, 2.0, -0.0, np.inf], dtype=np.float32)[np.arange(rows) % 6]
    t = tensor(x, kind)
    ids, logp, kept = (v.cpu().numpy() for v in B.sample(t, torch.from_numpy(u).to(DEV), to_filter(f) if f else None))
    xh = host(t)
    for r in range(rows):
        z, k, margin = ref.row(xh[r], **{name: v[r].item() for name, v in f.items()})
        assert margin >= NEAR and kept[r] == k.sum(), r
        want = np.nonzero(k)[0][0 if u[r] <= 0 else -1]
        assert ids[r] == want, (r, u[r], ids[r], want)
        lp = z[want] - ref.lse(z, k)
        assert abs(logp[r] - lp) <= 2.0 ** -24 * abs(lp) + 2.0 ** -28 + 2.0 ** -52 * 70, (r, logp[r], lp)


@pytest.mark.parametrize("rows", [2, 136])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("tail", [-27.75, -29.875, -30.625, -31.0, -31.25])
def test_flat_tails_far_below_a_dominant_token(tail, kind, rows):
    """What many light tokens weigh together: a step of 2^-45 each, 2^-29 of their sum, and
    the result's rounding."""
    vocab = 151936
    x = torch.full((rows, vocab), tail, device=DEV).to(KINDS[kind])
    x[:, 5] = 0.0
    others = (vocab - 1) * np.exp(tail)
    ids, logp, kept = B.sample(x, torch.full((rows,), 0.5, device=DEV))
    mask, lse, mkept = B.filter_mask(x, None)
    assert bool((ids == 5).all()) and bool((kept == vocab).all()) and bool((mkept == vocab).all())
    bound = vocab * 2.0 ** -45 + 2.0 ** -29 * others
    for got, want in ((logp, -np.log1p(others)), (lse, np.log1p(others))):
        err = np.abs(got.cpu().numpy().astype(np.float64) - want)
        assert (err <= bound + 2.0 ** -24 * abs(want)).all(), (err.max(), bound)


def settled(rng, x, scale, min_p, top_k, nucleus):
    """(top_p, u) of a row whose borders lie in the middle of tokens that weigh 2^-21 of the whole
    and more: no sum's error (2^-29 and vocab 2^-45 of it) and no rounding of top_p or u to
    float32 (2^-25) reaches a neighbour."""
    top_p = 1.0
    if nucleus:
        z, kept, _ = ref.row(x, scale, min_p, top_k)
        order = np.argsort(-x, kind="stable")
        order = order[kept[order]]
        mass = np.exp(z[order] - z[order[0]])
        upto = np.cumsum(mass)
        i = int(np.searchsorted(upto, rng.uniform(0.3, 0.95) * upto[-1]))
        while mass[i] < 2.0 ** -21 * upto[-1]:
            i -= 1
        top_p = np.float32((upto[i] - mass[i] / 2) / upto[-1])
    z, kept, _ = ref.row(x, scale, min_p, top_k, float(top_p))
    mass = np.where(kept, np.exp(np.where(kept, z, -np.inf) - z[kept].max()), 0.0)
    upto = np.cumsum(mass)
    j = rng.choice(np.nonzero(mass >= 2.0 ** -21 * upto[-1])[0])
    return top_p, np.float32((upto[j] - mass[j] / 2) / upto[-1])


@pytest.mark.parametrize("copies", [1, 8])
@pytest.mark.parametrize("kind,vocab", [("bf16", B.LPD_SAMPLE_MAX_VOCAB), ("f32", B.LPD_SAMPLE_MAX_VOCAB), ("f32", 262147)])
def test_largest_vocabularies_at_few_and_many_rows(kind, vocab, copies):
    """Peaked, flat, constant rows and rows next to zero under every kind of filter, none left
    out of the comparison; few rows go to clusters, many to a CTA each and what that leaves to
    clusters.  (A constant row's masses add up to the most that there is.)"""
    rng = np.random.default_rng(23)
    n = 17
    x = logits(rng, n, vocab)
    x[1::4] = rng.normal(0, 0.7, x[1::4].shape)
    x[2::4] = 1.5
    x[3::4] = rng.normal(0, 0.02, x[3::4].shape)
    x = np.where(x > 12.0, 12.0 + rng.uniform(0, 1, x.shape), x)
    t = tensor(x, kind)
    xh = host(t)
    scale = rng.uniform(0.5, 1.5, n).astype(np.float32)
    form = np.arange(n) % 5  # 0: none, 1: top-p, 2: a large top-k, 3: a small one and top-p, 4: min-p and top-p
    top_k = np.where(form == 2, rng.integers(3000, vocab // 2, n), np.where(form == 3, rng.integers(20, 400, n), 0)).astype(np.int32)
    min_p = np.where(form == 4, rng.uniform(0.005, 0.2, n), 0).astype(np.float32)
    pairs = [settled(rng, xh[r], float(scale[r]), float(min_p[r]), int(top_k[r]), form[r] in (1, 3, 4)) for r in range(n)]
    f = dict(scale=scale, min_p=min_p, top_k=top_k, top_p=np.array([p for p, _ in pairs], np.float32))
    u = np.array([v for _, v in pairs], np.float32)
    many = to_filter({k: np.tile(v, copies) for k, v in f.items()})
    t = t.repeat(copies, 1)
    ids, logp, kept = (v.cpu().numpy() for v in B.sample(t, torch.from_numpy(np.tile(u, copies)).to(DEV), many))
    mask, lse, mkept = B.filter_mask(t, many)
    for r in range(n):
        z, k, margin = ref.row(xh[r], **{name: v[r].item() for name, v in f.items()})
        j, lp, near = ref.draw(z, k, float(u[r]))
        assert margin >= 2.0 ** -23 and near >= 2.0 ** -23, r
        words = torch.from_numpy(np.packbits(np.pad(k, (0, -vocab % 32)), bitorder="little").view(np.int32)).to(DEV)
        sums = 2.0 ** -29 + vocab * 2.0 ** -45
        want_lse = ref.lse(z, k)
        for c in range(r, n * copies, n):
            assert ids[c] == j and kept[c] == k.sum() == mkept[c], (c, ids[c], j, kept[c], k.sum())
            assert torch.equal(mask[c], words), c
            assert abs(logp[c] - lp) <= 2.0 ** -24 * abs(lp) + sums, (c, logp[c], lp)
            assert abs(float(lse[c]) - want_lse) <= 2.0 ** -24 * abs(want_lse) + sums, (c, lse[c], want_lse)
