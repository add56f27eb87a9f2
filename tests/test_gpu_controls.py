"""Sampling controls on the GPU (needs a GPU): the controlled logits, the scores
and the gradients against the float64 definition in controls_ref.py.

Bounds.  Apply: a touched logit is carried as two floats and scaled in one
multiply-add, an untouched one is one product, so float32 is within two
roundings (2^-23) of the value, plus 2^-46 of the intermediate terms (at most
some hundreds here: 1e-10); bf16 adds its half step, 2^-8.  Logprobs: an exponent
a = (x - m) s log2 e carries three roundings, 3 * 2^-24 |a|, and terms below
2^-40 do not count, so a term is off by at most 40 * 3 * 2^-24 * ln 2 = 5e-6
relative, and so is the sum; the special-function unit adds 2^-22 and the sums
some 2^-24: 1e-5 in all, and the float32 result 2^-24 of itself.  Gradients:
the same 1e-5 on p, three roundings on the rest.
"""
import numpy as np
import pytest
import torch

from tests import controls_ref as ref
from logprob_drift_scoring_gb300 import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda"
KINDS = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "f32": 0.0}


def to_device(c):
    return B.Controls(**{k: torch.from_numpy(np.ascontiguousarray(v)).to(DEV) for k, v in c.items()})


def tensor(x, kind, pad=0):
    t = torch.from_numpy(x.astype(np.float32)).to(DEV).to(KINDS[kind])
    if pad:
        wide = torch.full((t.shape[0], t.shape[1] + pad), float("nan"), dtype=t.dtype, device=DEV)
        wide[:, :t.shape[1]] = t
        t = wide[:, :t.shape[1]]
    return t


def host(t):
    return t.float().cpu().numpy().astype(np.float64)


def check_apply(c, x, out_kind, out):
    got, xh = host(out), host(x)
    for r in range(len(xh)):
        z, _ = ref.row(c, xh[r], r)
        inf = np.isneginf(z)
        assert np.array_equal(np.isneginf(got[r]), inf), r
        err = np.abs(got[r][~inf] - z[~inf])
        assert np.all(err <= (2.0 ** -23 + HALF[out_kind]) * np.abs(z[~inf]) + 1e-10), (r, err.max())


@pytest.mark.parametrize("vocab,pad", [(1, 0), (5, 3), (31, 0), (33, 7), (1000, 8), (2048, 0), (2049, 0), (8193, 7),
                                       (20011, 0), (20016, 0)])
@pytest.mark.parametrize("xk,ok", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32"), ("f32", "bf16")])
def test_apply(vocab, pad, xk, ok):
    rng = np.random.default_rng(vocab + pad)
    rows = 7
    c = ref.random_controls(rng, rows, vocab, history=70)
    x = tensor(rng.normal(0, 3, (rows, vocab)), xk, pad)
    check_apply(c, x, ok, B.controls_apply(x, to_device(c), KINDS[ok]))


@pytest.mark.parametrize("rows,vocab,history", [(200, 20008, 300), (3, 50000, 40000), (90, 40007, 900)])
def test_apply_many_units(rows, vocab, history):
    """Both chunk widths, several units a block (the table is zero again after each)."""
    rng = np.random.default_rng(rows)
    c = ref.random_controls(rng, rows, vocab, history=history, masks=3, bias=40)
    x = tensor(rng.normal(0, 3, (rows, vocab)), "bf16")
    check_apply(c, x, "bf16", B.controls_apply(x, to_device(c)))


@pytest.mark.parametrize("leave", ["history", "bias", "masks", "scale", "penalties", "all"])
def test_apply_parts_left_out(leave):
    rng = np.random.default_rng(3)
    parts = ("repetition", "frequency", "presence", "scale")
    kw = {"history": dict(history=None), "bias": dict(bias=0), "masks": dict(masks=0), "scale": dict(parts=parts[:3]),
          "penalties": dict(parts=("scale",)), "all": dict(history=None, bias=0, masks=0, parts=())}[leave]
    c = ref.random_controls(rng, 5, 700, **kw)
    x = tensor(rng.normal(0, 3, (5, 700)), "f32")
    check_apply(c, x, "f32", B.controls_apply(x, to_device(c)))
    if leave == "all":
        assert torch.equal(B.controls_apply(x, None), x)
        assert torch.equal(B.controls_apply(x, None, torch.bfloat16), x.to(torch.bfloat16))


@pytest.mark.parametrize("name", ["repetition", "frequency", "presence"])
def test_apply_one_penalty(name):
    rng = np.random.default_rng(4)
    c = ref.random_controls(rng, 6, 900, bias=0, masks=0, parts=(name,))
    x = tensor(rng.normal(0, 3, (6, 900)), "f32")
    check_apply(c, x, "f32", B.controls_apply(x, to_device(c)))


def test_apply_in_place_and_zero_rows():
    rng = np.random.default_rng(5)
    for kind, vocab, pad in (("bf16", 9001, 7), ("f32", 4096, 0)):
        c = to_device(ref.random_controls(rng, 40, vocab, history=200))
        x = tensor(rng.normal(0, 3, (40, vocab)), kind, pad)
        want = B.controls_apply(x, c)
        B.lpd_controls_apply(x, c, x)
        assert torch.equal(x, want)
    empty = torch.empty(0, 16, device=DEV)
    B.lpd_controls_apply(empty, None, empty)


def test_apply_leaves_the_padding():
    rng = np.random.default_rng(6)
    for vocab in (100, 8200, 8203):
        c = to_device(ref.random_controls(rng, 9, vocab))
        x = tensor(rng.normal(0, 3, (9, vocab)), "bf16", 5)
        wide = torch.full((10, vocab + 11), 7.0, device=DEV)
        B.lpd_controls_apply(x, c, wide[:9, :vocab])
        assert bool((wide[:, vocab:] == 7).all()) and bool((wide[9] == 7).all())


def test_ranges_are_clamped():
    """Offsets outside the history, crossed offsets, a begin that passes 32 bits."""
    rng = np.random.default_rng(7)
    c = ref.random_controls(rng, 6, 300, history=20)
    c["hist_begin"][:] = [-5, 3, 1 << 40, 15, 0, -(1 << 62)]
    c["hist_split"][:] = [-9, 1, 5, 30, 1 << 50, 0]
    c["hist_end"][:] = [9, 50, 1 << 41, 4, 21, (1 << 62)]
    x = tensor(rng.normal(0, 3, (6, 300)), "f32")
    check_apply(c, x, "f32", B.controls_apply(x, to_device(c)))


def test_masks():
    """Every row its own mask; nothing allowed; a mask row behind the table."""
    rng = np.random.default_rng(8)
    c = ref.random_controls(rng, 5, 333, masks=5)
    c["mask"][2] = 0
    x = tensor(rng.normal(0, 3, (5, 333)), "f32")
    for rows in (None, np.array([0, 5, 2, -7, 1 << 30], np.int32)):
        d = dict(c)
        if rows is None:
            del d["mask_row"]
        else:
            d["mask_row"] = rows
        out = B.controls_apply(x, to_device(d))
        check_apply(d, x, "f32", out)
        assert bool(torch.isneginf(out[2]).all())
    # a mask table with rows wider than the vocabulary, set bits behind its end
    wide = np.full((5, 40), -1, np.int32)
    d = dict(c, mask=wide)
    check_apply(d, x, "f32", B.controls_apply(x, to_device(d)))


def test_what_masked_places_hold_does_not_matter():
    rng = np.random.default_rng(9)
    rows, vocab = 6, 9000
    ids = rng.integers(0, vocab, rows).astype(np.int32)
    c = ref.random_controls(rng, rows, vocab, masks=rows, keep=ids)
    c["mask_row"] = np.arange(rows, dtype=np.int32)
    for r in range(rows):
        c["mask"][r, ids[r] // 32] |= np.int32(np.uint32(1 << (ids[r] % 32)).view(np.int32))
    x = rng.normal(0, 3, (rows, vocab))
    dirty = x.copy()
    for r in range(rows):
        z, _ = ref.row(c, x[r], r)
        off = np.flatnonzero(np.isneginf(z))
        dirty[r, off] = rng.choice([np.nan, np.inf, -np.inf, 3.4e38, -3.4e38], len(off))
    h = to_device(c)
    idt, act = torch.from_numpy(ids).to(DEV), torch.ones(rows, dtype=torch.uint8, device=DEV)
    a, b = tensor(x, "f32"), tensor(dirty, "f32")
    assert torch.equal(B.controls_apply(a, h), B.controls_apply(b, h))
    s1, s2 = (B.score_controlled(t, t, idt, act, h, h) for t in (a, b))
    assert s2.metrics["status"] == 0
    for k in ("logp_train", "logp_rollout", "dlogp"):
        assert torch.equal(getattr(s1, k), getattr(s2, k))
    g = torch.randn(rows, device=DEV)
    o1, o2 = torch.empty_like(a), torch.empty_like(a)
    B.lpd_logprob_backward_controlled(a, h, idt, act, s1.logp_train, g, o1)
    B.lpd_logprob_backward_controlled(b, h, idt, act, s1.logp_train, g, o2)
    assert torch.equal(o1, o2)


def test_extreme_logits():
    """The type's lowest value as a mask, infinities among touched tokens."""
    rng = np.random.default_rng(10)
    c = ref.random_controls(rng, 4, 500, history=400, masks=0)
    c["repetition"][:] = 2.0
    for kind in KINDS:
        x = rng.normal(0, 3, (4, 500))
        x[:, ::2] = torch.finfo(KINDS[kind]).min
        x[1, 1::4] = -np.inf
        t = tensor(x, kind)
        out = host(B.controls_apply(t, to_device(c), torch.float32))
        for r in range(4):
            z, _ = ref.row(c, host(t)[r], r)
            z = np.where(z < -3.4028235e38, -np.inf, z)
            ok = np.isclose(out[r], z, rtol=2.0 ** -22, atol=1e-6) | (out[r] == z)
            assert ok.all(), (kind, r)
        ids = torch.full((4,), 3, dtype=torch.int32, device=DEV)
        s = B.score_controlled(t, t, ids, torch.ones(4, dtype=torch.uint8, device=DEV), to_device(c), to_device(c))
        for r in (0, 2, 3):
            z, _ = ref.row(c, host(t)[r], r)
            assert abs(float(s.logp_train[r]) - ref.logp(z, 3)) <= 1e-5 + 2.0 ** -23 * abs(ref.logp(z, 3))
            assert float(s.dlogp[r]) == 0.0


def check_score(ct, cr, x, y, ids, act, res):
    xh, yh = host(x), host(y)
    for side, c, v, got in (("t", ct, xh, res.logp_train), ("r", cr, yh, res.logp_rollout)):
        got = got.double().cpu().numpy()
        for r in range(len(ids)):
            if not act[r]:
                assert got[r] == 0.0
                continue
            want = ref.logp(ref.row(c, v[r], r)[0], ids[r])
            assert abs(got[r] - want) <= 1e-5 + 2.0 ** -23 * abs(want), (side, r, got[r], want)
    d = res.dlogp.double().cpu().numpy()
    for r in np.flatnonzero(act):
        want = ref.logp(ref.row(ct, xh[r], r)[0], ids[r]) - ref.logp(ref.row(cr, yh[r], r)[0], ids[r])
        assert abs(d[r] - want) <= 2e-5 + 2.0 ** -23 * abs(want)
    # the metrics are those of the per-token differences (the scorer's own stage, held to the oracle elsewhere)
    m = B.drift_metrics_from_dlogp(res.dlogp, torch.from_numpy(act).to(DEV))
    assert res.metrics["n_active"] == m["n_active"] == int(act.sum()) and res.metrics["status"] == 0
    for k in ("mean_abs_dlogp", "max_abs_dlogp", "p95_abs_dlogp", "ratio0_mean"):
        assert abs(res.metrics[k] - m[k]) <= 1e-6 * (1 + abs(m[k]))


@pytest.mark.parametrize("vocab,pad", [(1, 0), (2, 1), (40, 0), (1000, 3), (8192, 0), (8200, 8), (16385, 7), (30000, 0)])
@pytest.mark.parametrize("xk,yk", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("sides", ["both", "own", "rollout", "train", "none"])
def test_score(vocab, pad, xk, yk, sides):
    if sides != "both" and xk != yk:
        pytest.skip("the type pairs are covered with one handle")
    rng = np.random.default_rng(vocab * 7 + pad)
    rows = 9
    ids = rng.integers(0, vocab, rows).astype(np.int32)
    x = rng.normal(0, 3, (rows, vocab))
    y = x + rng.normal(0, 2e-3, x.shape)
    c = ref.random_controls(rng, rows, vocab, keep=ids, history=60)
    c["history"][5] = ids[0]
    other = ref.random_controls(rng, rows, vocab, keep=ids, history=33, bias=2)
    ct, cr = {"both": (c, c), "own": (c, other), "rollout": ({}, c), "train": (c, {}), "none": ({}, {})}[sides]
    h = to_device(c)
    ht, hr = {"both": (h, h), "own": (h, to_device(other)), "rollout": (None, h), "train": (h, None),
              "none": (None, None)}[sides]
    act = (rng.random(rows) < 0.8).astype(np.uint8)
    act[0] = 1
    xt, yt = tensor(x, xk, pad), tensor(y, yk, pad)
    res = B.score_controlled(xt, yt, torch.from_numpy(ids).to(DEV), torch.from_numpy(act).to(DEV), ht, hr)
    check_score(ct, cr, xt, yt, ids, act, res)


def test_score_differing_bias_over_one_history():
    """One history, one bias list, other values and penalties a side: one table serves both."""
    rng = np.random.default_rng(11)
    rows, vocab = 8, 9000
    ids = rng.integers(0, vocab, rows).astype(np.int32)
    c = ref.random_controls(rng, rows, vocab, history=500, masks=0, bias=20)
    ids[:4] = c["bias_ids"][:4, 1].clip(0, vocab - 1)
    d = dict(c, bias=-c["bias"], repetition=c["repetition"][::-1].copy(), scale=c["scale"][::-1].copy())
    shared = {k: torch.from_numpy(v).to(DEV) for k, v in c.items()}
    ht = B.Controls(**shared)
    hr = B.Controls(**{**shared, **{k: torch.from_numpy(d[k]).to(DEV) for k in ("bias", "repetition", "scale")}})
    x = tensor(rng.normal(0, 3, (rows, vocab)), "bf16")
    act = np.ones(rows, np.uint8)
    check_score(c, d, x, x, ids, act, B.score_controlled(x, x, torch.from_numpy(ids).to(DEV), torch.from_numpy(act).to(DEV), ht, hr))


def test_score_of_applied_logits():
    """lpd_score on the float32 controlled logits gives the same logprobs."""
    rng = np.random.default_rng(12)
    rows, vocab = 50, 33000
    ids = rng.integers(0, vocab, rows).astype(np.int32)
    c = ref.random_controls(rng, rows, vocab, keep=ids, history=800)
    h, idt = to_device(c), torch.from_numpy(ids).to(DEV)
    act = torch.ones(rows, dtype=torch.uint8, device=DEV)
    x = tensor(rng.normal(0, 3, (rows, vocab)), "bf16")
    y = (x.float() + 1e-3 * torch.randn(rows, vocab, device=DEV)).to(torch.bfloat16)
    a = B.score_controlled(x, y, idt, act, h, h)
    b = B.score(B.controls_apply(x, h, torch.float32), B.controls_apply(y, h, torch.float32), idt, act)
    # the applied logits are rounded to float32: 2^-24 of at most 64, twice
    for k in ("logp_train", "logp_rollout"):
        assert float((getattr(a, k) - getattr(b, k)).abs().max()) <= 2e-5 + 8e-6
    n = B.score_controlled(x, y, idt, act)
    m = B.score(x, y, idt, act)
    assert float((n.dlogp - m.dlogp).abs().max()) <= 2e-5


def test_batch_invariance_and_load_paths():
    """A row's bits do not depend on its batch, its place, or its alignment."""
    rng = np.random.default_rng(13)
    rows, vocab = 30, 20003
    ids = rng.integers(0, vocab, rows).astype(np.int32)
    c = ref.random_controls(rng, rows, vocab, keep=ids, history=400, masks=4, bias=9)
    x = rng.normal(0, 3, (rows, vocab))
    y = x + rng.normal(0, 2e-3, x.shape)

    def run(at, pad, kind="f32"):
        d = {k: (v[at] if k not in ("history", "mask") else v) for k, v in c.items()}
        h = to_device(d)
        r = B.score_controlled(tensor(x[at], kind, pad), tensor(y[at], kind, pad), torch.from_numpy(ids[at]).to(DEV),
                               torch.ones(len(at), dtype=torch.uint8, device=DEV), h, h)
        return [r.logp_train, r.logp_rollout, r.dlogp]

    full = run(np.arange(rows), 0)
    for at in ([4], [29, 4, 0], list(range(10, 20))):
        for pad in (0, 1, 5):
            for a, b in zip(full, run(np.array(at), pad)):
                assert torch.equal(a[at], b), (at, pad)
    # bf16 values scored as bf16 and as their float32 copies
    x = host(tensor(x, "bf16"))
    y = host(tensor(y, "bf16"))
    for a, b in zip(run(np.arange(rows), 0, "bf16"), run(np.arange(rows), 3, "f32")):
        assert torch.equal(a, b)


def test_batch_invariance_over_unit_shapes():
    """Many rows take whole rows at a time, few rows segments: the same bits.  One row's history has more
    distinct tokens than the kernel counts at a time."""
    rng = np.random.default_rng(23)
    rows, vocab = 330, 130000
    ids = rng.integers(0, vocab, rows).astype(np.int32)
    c = ref.random_controls(rng, rows, vocab, keep=ids, history=6000, masks=3, bias=5)
    c["hist_begin"][1], c["hist_split"][1], c["hist_end"][1] = 0, 100, 6001
    x = torch.randn(rows, vocab, device=DEV, generator=torch.Generator(DEV).manual_seed(5)).mul_(3).to(torch.bfloat16)
    y = (x.float() + 1e-3).to(torch.bfloat16)

    def run(at):
        h = to_device({k: (v[at] if k not in ("history", "mask") else v) for k, v in c.items()})
        r = B.score_controlled(x[at], y[at], torch.from_numpy(ids[at]).to(DEV),
                               torch.ones(len(at), dtype=torch.uint8, device=DEV), h, h)
        return [r.logp_train, r.logp_rollout, r.dlogp]

    full = run(np.arange(rows))
    for at in ([1], [0, 1, 2], list(range(200, 260))):
        for a, b in zip(full, run(np.array(at))):
            assert torch.equal(a[at], b), at
    for r in (0, 1, 77):
        want = ref.logp(ref.row(c, host(x[r:r + 1])[0], r)[0], ids[r])
        assert abs(float(full[0][r]) - want) <= 1e-5 + 2.0 ** -23 * abs(want)


def test_repeated_calls_give_the_same_bits():
    """Long rows, ring stages reused at once: every call gives the first call's bits."""
    rng = np.random.default_rng(25)
    rows, vocab = 330, 130000
    ids = rng.integers(0, vocab, rows).astype(np.int32)
    h = to_device(ref.random_controls(rng, rows, vocab, keep=ids, history=6000, masks=3, bias=5))
    x = torch.randn(rows, vocab, device=DEV, generator=torch.Generator(DEV).manual_seed(6)).mul_(3).to(torch.bfloat16)
    y = (x.float() + 1e-3).to(torch.bfloat16)
    idt, act = torch.from_numpy(ids).to(DEV), torch.ones(rows, dtype=torch.uint8, device=DEV)
    first = B.score_controlled(x, y, idt, act, h, h)
    z = B.controls_apply(x, h)
    g = torch.empty_like(x)
    B.lpd_logprob_backward_controlled(x, h, idt, act, first.logp_train, first.dlogp, g)
    for _ in range(24):
        r = B.score_controlled(x, y, idt, act, h, h)
        for k in ("logp_train", "logp_rollout", "dlogp"):
            assert torch.equal(getattr(first, k), getattr(r, k)), k
    out = torch.empty_like(x)
    for _ in range(12):
        B.lpd_controls_apply(x, h, out)
        assert torch.equal(out, z)
        B.lpd_logprob_backward_controlled(x, h, idt, act, first.logp_train, first.dlogp, out)
        assert torch.equal(out, g)


def test_more_touched_tokens_than_counted_at_a_time():
    """Elementwise forms with thousands of distinct tokens in a unit, in place too, and a long bias list."""
    rng = np.random.default_rng(24)
    rows, vocab = 3, 9000
    c = ref.random_controls(rng, rows, vocab, history=30000, masks=2, bias=600)
    c["hist_begin"][:], c["hist_split"][:], c["hist_end"][:] = 0, [5, 20000, 29000], 30001
    x = tensor(rng.normal(0, 3, (rows, vocab)), "f32")
    h = to_device(c)
    out = B.controls_apply(x, h)
    check_apply(c, x, "f32", out)
    # enough rows that a unit is a whole row
    many = 700
    big = {k: (np.repeat(v, 234, axis=0)[:many] if k not in ("history", "mask") else v) for k, v in c.items()}
    xs = x.repeat_interleave(234, 0)[:many].contiguous()
    hb = to_device(big)
    got = B.controls_apply(xs, hb)
    assert torch.equal(got, out.repeat_interleave(234, 0)[:many])
    B.lpd_controls_apply(xs, hb, xs)
    assert torch.equal(xs, got)


@pytest.mark.parametrize("kind,vocab,pad", [("bf16", 9001, 7), ("bf16", 20000, 0), ("f32", 12003, 2), ("f32", 8192, 0)])
@pytest.mark.parametrize("rows", [1, 60, 500])
def test_apply_in_place_over_many_units(kind, vocab, pad, rows):
    """Several rows a block and several units a row, on 16-byte boundaries and
    off them, some rows with more touched tokens than are counted at a time."""
    rng = np.random.default_rng(25)
    c = ref.random_controls(rng, rows, vocab, history=16000, masks=3, bias=9)
    wide = rng.random(rows) < 0.3
    c["hist_begin"][wide], c["hist_end"][wide] = 0, 16000
    h = to_device(c)
    x = tensor(rng.normal(0, 3, (rows, vocab)), kind, pad)
    want = B.controls_apply(x, h)
    for _ in range(3):
        y = tensor(np.zeros((rows, vocab)), kind, pad)
        y.copy_(x)
        B.lpd_controls_apply(y, h, y)
        assert torch.equal(y, want)


@pytest.mark.parametrize("what", ["masked_id", "nothing_allowed", "bad_scale", "nan_logit", "oob"])
def test_score_status(what):
    rng = np.random.default_rng(14)
    rows, vocab = 4, 600
    ids = np.array([1, 2, 3, 4], np.int32)
    c = ref.random_controls(rng, rows, vocab, keep=ids, masks=rows)
    c["mask_row"] = np.arange(rows, dtype=np.int32)
    for r in range(rows):
        c["mask"][r, 0] |= 0x1E
    x = rng.normal(0, 3, (rows, vocab))
    if what == "masked_id":
        c["mask"][1, 0] &= ~4
    elif what == "nothing_allowed":
        c["mask"][1] = 0
    elif what == "bad_scale":
        c["scale"][1] = 0.0
    elif what == "nan_logit":
        x[1, 2] = np.nan
    else:
        ids[1] = vocab
    h, t = to_device(c), tensor(x, "f32")
    act = torch.ones(rows, dtype=torch.uint8, device=DEV)
    idt = torch.from_numpy(ids).to(DEV)
    res = B.score_controlled(t, t, idt, act, h, h)
    assert res.metrics["status"] == (B.LPD_STATUS_TOKEN_OOB if what == "oob" else B.LPD_STATUS_NONFINITE)
    for r in (0, 2, 3):
        want = ref.logp(ref.row(c, host(t)[r], r)[0], ids[r])
        assert abs(float(res.logp_train[r]) - want) <= 1e-5 + 2.0 ** -23 * abs(want)
    assert not np.isfinite(float(res.logp_train[1]))
    out = torch.empty(rows, vocab, device=DEV)
    B.lpd_logprob_backward_controlled(t, h, idt, act, res.logp_train, torch.ones(rows, device=DEV), out)
    assert bool(torch.isfinite(out[[0, 2, 3]]).all())
    if what == "nothing_allowed":
        assert bool((out[1] == 0).all())
    else:
        assert bool(torch.isnan(out[1]).any())
    # the row counts nowhere when it is inactive
    act[1] = 0
    res = B.score_controlled(t, t, idt, act, h, h)
    assert res.metrics["status"] == 0 and res.metrics["n_active"] == 3
    none = B.score_controlled(t, t, idt, torch.zeros_like(act), h, h)
    assert none.metrics["n_active"] == 0 and none.metrics["flags"] == B.LPD_FLAG_NO_ACTIVE


@pytest.mark.parametrize("vocab,pad", [(1, 0), (7, 2), (65, 0), (2050, 0), (8192, 0), (20011, 3)])
@pytest.mark.parametrize("xk,ok", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32"), ("f32", "bf16")])
def test_gradient(vocab, pad, xk, ok):
    rng = np.random.default_rng(vocab + 1)
    rows = 8
    ids = rng.integers(0, vocab, rows).astype(np.int32)
    c = ref.random_controls(rng, rows, vocab, keep=ids, history=60)
    c["history"][7] = ids[1]
    x = tensor(rng.normal(0, 3, (rows, vocab)), xk, pad)
    xh = host(x)
    act = np.ones(rows, np.uint8)
    act[3] = 0
    g = rng.normal(0, 1, rows).astype(np.float32)
    lp = np.array([ref.logp(ref.row(c, xh[r], r)[0], ids[r]) for r in range(rows)]).astype(np.float32)
    lp[3] = np.nan
    wide = torch.full((rows, vocab + pad), 5.0, dtype=KINDS[ok], device=DEV)
    out = wide[:, :vocab]
    B.lpd_logprob_backward_controlled(x, to_device(c), *(torch.from_numpy(v).to(DEV) for v in (ids, act, lp, g)), out)
    got = host(out)
    assert bool((wide[:, vocab:] == 5).all())
    for r in range(rows):
        if not act[r]:
            assert np.all(got[r] == 0)
            continue
        z, slope = ref.row(c, xh[r], r)
        p = np.exp(z - z[ids[r]] + np.float64(lp[r]))
        hot = np.arange(vocab) == ids[r]
        want = g[r] * slope * (hot - p)
        # logp's own rounding is an input: p follows it on both sides
        tol = np.abs(g[r] * slope) * 1e-5 * p + (2.0 ** -21 + HALF[ok]) * np.abs(want) + 2.0 ** -24 * np.abs(g[r] * slope) * hot
        assert np.all(np.abs(got[r] - want) <= tol + 1e-38), (r, np.max(np.abs(got[r] - want) - tol))


def test_gradient_against_differences():
    """Central differences of the float64 logprob with respect to single raw logits."""
    rng = np.random.default_rng(15)
    rows, vocab, h = 6, 300, 1e-4
    ids = rng.integers(0, vocab, rows).astype(np.int32)
    c = ref.random_controls(rng, rows, vocab, keep=ids, history=100)
    c["history"][:rows] = ids
    x = rng.normal(0, 3, (rows, vocab)).astype(np.float32)
    x[np.abs(x) < 1e-3] = 0.5  # the penalty's kink
    t = tensor(x, "f32")
    x = host(t)
    idt, act = torch.from_numpy(ids).to(DEV), torch.ones(rows, dtype=torch.uint8, device=DEV)
    hc = to_device(c)
    res = B.score_controlled(t, t, idt, act, hc, hc)
    out = torch.empty_like(t)
    B.lpd_logprob_backward_controlled(t, hc, idt, act, res.logp_train, torch.ones(rows, device=DEV), out)
    got = host(out)
    for r in range(rows):
        begin, _, end = ref.clamp_range(c, r)
        for j in [int(ids[r])] + [int(v) for v in c["history"][begin:end][:4] if 0 <= v < vocab] + rng.integers(0, vocab, 6).tolist():
            f = []
            for d in (h, -h):
                v = x[r].copy()
                v[j] += d
                f.append(ref.logp(ref.row(c, v, r)[0], ids[r]))
            # third derivative at most slope^3 <= 64: h^2 * 64 / 6 = 1e-7; the forward's 1e-5 on p
            assert abs((f[0] - f[1]) / (2 * h) - got[r, j]) <= 4e-5 + 2.0 ** -20 * abs(got[r, j]), (r, j)


def test_long_history_counts():
    """More occurrences than a small counter holds; a history far longer than a row."""
    rng = np.random.default_rng(16)
    n, vocab = 200_000, 700
    c = {"history": rng.integers(0, 5, n).astype(np.int32), "hist_begin": np.zeros(2, np.int64),
         "hist_split": np.array([0, 150_000], np.int64), "hist_end": np.array([n, n - 1], np.int64),
         "frequency": np.array([1e-4, 2e-5], np.float32), "presence": np.array([0.5, 0.0], np.float32),
         "repetition": np.array([1.1, 1.3], np.float32)}
    x = tensor(rng.normal(0, 3, (2, vocab)), "f32")
    check_apply(c, x, "f32", B.controls_apply(x, to_device(c)))


def test_streams_graphs_and_determinism():
    """Two streams with a workspace each; a captured and replayed run on new inputs; the same bits each time."""
    rng = np.random.default_rng(17)
    rows, vocab = 60, 40000
    ids = rng.integers(0, vocab, rows).astype(np.int32)
    h = to_device(ref.random_controls(rng, rows, vocab, keep=ids, history=3000, masks=6, bias=30))
    x = tensor(rng.normal(0, 3, (rows, vocab)), "bf16")
    y = (x.float() + 1e-3).to(torch.bfloat16)
    idt, act = torch.from_numpy(ids).to(DEV), torch.ones(rows, dtype=torch.uint8, device=DEV)
    g = torch.randn(rows, device=DEV)

    def buffers():
        outs = [torch.empty(rows, device=DEV) for _ in range(3)]
        met = torch.empty(B.METRICS_BYTES, dtype=torch.uint8, device=DEV)
        ws = torch.empty(B.lpd_workspace_size(B.LPD_KIND_CONTROLLED, rows, vocab), dtype=torch.uint8, device=DEV)
        return outs, met, ws, torch.empty_like(x), torch.empty_like(x)

    def step(b):
        outs, met, ws, z, dx = b
        B.lpd_controls_apply(x, h, z)
        B.lpd_score_controlled(x, y, h, h, idt, act, 0.8, 1.2, *outs, met, ws)
        B.lpd_logprob_backward_controlled(x, h, idt, act, outs[0], g, dx)

    def results(b):
        torch.cuda.synchronize()
        # as bytes: the flipped ids select masked tokens, whose logprob is not finite
        return [t.view(torch.uint8).clone() for t in (*b[0], b[1], b[3], b[4])]

    first = buffers()
    step(first)
    want = results(first)
    sets = [buffers(), buffers()]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(3):
        for s, b in zip(streams, sets):
            with torch.cuda.stream(s):
                step(b)
    for b in sets:
        for a, w in zip(results(b), want):
            assert torch.equal(a, w)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(first)
    x.copy_((x.float() * 0.9).to(torch.bfloat16))
    idt.copy_(idt.flip(0))
    h.scale.mul_(1.1)
    h.hist_end.sub_(7)
    for t in (*first[0], first[1], first[3], first[4]):
        t.zero_()
    graph.replay()
    replayed = results(first)
    step(sets[0])
    for a, b in zip(replayed, results(sets[0])):
        assert torch.equal(a, b)
    assert not torch.equal(replayed[0], want[0])


def test_a_mask_table_of_no_rows_allows_nothing():
    rng = np.random.default_rng(31)
    rows, vocab = 4, 300
    c = {"mask": np.zeros((0, 10), np.int32), "mask_row": np.array([0, -1, 3, -1], np.int32)}
    x = tensor(rng.normal(0, 3, (rows, vocab)), "f32")
    out = B.controls_apply(x, to_device(c))
    check_apply(c, x, "f32", out)
    assert bool(torch.isneginf(out[::2]).all()) and torch.equal(out[1::2], x[1::2])
    ids, act = torch.zeros(rows, dtype=torch.int32, device=DEV), torch.ones(rows, dtype=torch.uint8, device=DEV)
    s = B.score_controlled(x, x, ids, act, to_device(c), None)
    assert s.metrics["status"] == B.LPD_STATUS_NONFINITE and bool(torch.isfinite(s.logp_train[1::2]).all())


def logp64(z, ids):
    """Selected logprobs of float64 rows on the device."""
    return torch.gather(z, 1, ids.long()[:, None])[:, 0] - torch.logsumexp(z, 1)


@pytest.mark.parametrize("vocab", [57345, 57347, 57350, 114690, 172033])
@pytest.mark.parametrize("xk,yk", [("bf16", "bf16"), ("f32", "f32"), ("bf16", "f32")])
def test_score_where_a_segment_of_few_columns_is_left(vocab, xk, yk):
    """The last columns carry most of each row's sum, so none of them may be lost or read twice, in the tensor's
    last row neither; and a row's bits are the same alone (a unit a segment) and among many (whole rows), on
    16-byte boundaries and off them."""
    gen = torch.Generator(DEV).manual_seed(vocab)
    many = 310
    x = torch.randn(many, vocab, device=DEV, generator=gen)
    x[:, -24:] += 8
    y = x + 2e-3 * torch.randn(many, vocab, device=DEV, generator=gen)
    ids = (vocab - 1 - torch.arange(many, device=DEV) % 20).int()

    def run(at, pad):
        n = len(at)
        room = torch.full((n, vocab + pad), 50.0, device=DEV)
        sides = []
        for v, k in ((x, xk), (y, yk)):
            t = room.to(KINDS[k])
            t[:, :vocab] = v[at].to(KINDS[k])
            sides.append(t[:, :vocab] if pad else t[:, :vocab].contiguous())
        act = torch.ones(n, dtype=torch.uint8, device=DEV)
        r = B.score_controlled(*sides, ids[at].contiguous(), act)
        assert r.metrics["status"] == 0
        for got, t in ((r.logp_train, sides[0]), (r.logp_rollout, sides[1])):
            want = logp64(t[-4:].double(), ids[at][-4:])
            err = (got[-4:].double() - want).abs()
            assert bool((err <= 1e-5 + 2.0 ** -23 * want.abs()).all()), (n, pad, err)
        return [r.logp_train, r.logp_rollout, r.dlogp]

    full = run(torch.arange(many), 0)
    for at in (torch.arange(many - 3, many), torch.tensor([7]), torch.tensor([3, 200])):
        for pad in (0, 1, -vocab % 8):
            for a, b in zip(full, run(at, pad)):
                assert torch.equal(a[at], b), (at, pad)
    for a, b in zip(full, run(torch.arange(many), -vocab % 8)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("rows,vocab", [(2, 57346), (2, 114689)])
def test_score_controlled_at_a_small_last_segment(rows, vocab):
    """The same place with controls that touch the columns around it."""
    rng = np.random.default_rng(vocab)
    ids = np.array([vocab - 2, vocab - 1], np.int32)
    c = ref.random_controls(rng, rows, vocab, keep=ids, history=60, bias=6)
    c["history"][:12] = np.arange(vocab - 12, vocab)
    c["hist_begin"][:], c["hist_split"][:], c["hist_end"][:] = 0, 5, 40
    c["bias_ids"][:, :3] = [[vocab - 3, vocab - 9, vocab - 1]] * 2
    x = rng.normal(0, 1, (rows, vocab))
    x[:, -20:] += 8
    y = x + rng.normal(0, 2e-3, x.shape)
    xt, yt = tensor(x, "bf16"), tensor(y, "bf16")
    h = to_device(c)
    act = np.ones(rows, np.uint8)
    res = B.score_controlled(xt, yt, torch.from_numpy(ids).to(DEV), torch.from_numpy(act).to(DEV), h, h)
    check_score(c, c, xt, yt, ids, act, res)


def check_float64(ct, cr, x, y, ids, res):
    """Logprobs and their difference within the bounds at the head of this file."""
    xh, yh = host(x), host(y)
    assert res.metrics["status"] == 0
    for r, j in enumerate(ids):
        t, u = ref.logp(ref.row(ct, xh[r], r)[0], j), ref.logp(ref.row(cr, yh[r], r)[0], j)
        for got, want, off in ((res.logp_train, t, 1e-5), (res.logp_rollout, u, 1e-5), (res.dlogp, t - u, 2e-5)):
            assert abs(float(got[r]) - want) <= off + 2.0 ** -23 * abs(want), (r, off, float(got[r]), want)


def score_sides(ct, cr, x, y, ids):
    ht, hr = (to_device(c) if c else None for c in (ct, cr))
    if ct is cr:
        hr = ht
    return B.score_controlled(x, y, torch.from_numpy(ids).to(DEV), torch.ones(len(ids), dtype=torch.uint8, device=DEV), ht, hr)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("scale", [1.0, 20.0, 100.0])
@pytest.mark.parametrize("how", ["rollout_mask", "train_mask", "rollout_only", "train_only", "penalty", "bias"])
def test_score_sides_whose_peaks_lie_apart(kind, scale, how):
    """One side's controls take the other's peak away: at a low temperature the sides' sums then lie hundreds of
    octaves apart, and each has to be kept beside its own maximum."""
    rng = np.random.default_rng(41)
    rows, vocab = 6, 20000
    x = rng.normal(0, 3, (rows, vocab))
    y = x + rng.normal(0, 2e-3, x.shape)
    xt, yt = tensor(x, kind), tensor(y, kind)
    top = [np.argsort(host(t), 1)[:, -40:] for t in (xt, yt)]
    ids = np.array([np.setdiff1d(np.arange(500), top[0][r])[r] for r in range(rows)], np.int32)
    s = np.full(rows, scale, np.float32)
    one = {"scale": s}
    if how in ("rollout_mask", "train_mask"):
        words = np.full((rows, vocab // 32), 0xFFFFFFFF, np.uint32)
        for r in range(rows):
            for j in top[0][r]:
                words[r, j // 32] &= ~np.uint32(1 << (j % 32))
        masked = {"scale": s, "mask": words.view(np.int32)}
        ct, cr = (one, masked) if how == "rollout_mask" else (masked, one)
    elif how in ("rollout_only", "train_only"):
        ct, cr = ({}, one) if how == "rollout_only" else (one, {})
    elif how == "penalty":
        hist = top[0].reshape(-1).astype(np.int32)
        at = np.arange(rows, dtype=np.int64) * top[0].shape[1]
        cr = {"scale": s, "history": hist, "hist_begin": at, "hist_split": at, "hist_end": at + top[0].shape[1],
              "repetition": np.full(rows, 2.5, np.float32), "presence": np.full(rows, 4, np.float32)}
        ct = one
    else:
        ct = {"scale": s, "bias_ids": top[0].astype(np.int32), "bias": np.full(top[0].shape, -30, np.float32)}
        cr = one
    check_float64(ct, cr, xt, yt, ids, score_sides(ct, cr, xt, yt, ids))


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("shift", [150.0, -150.0, 3.0])
@pytest.mark.parametrize("scale", [None, 10.0])
def test_score_sides_shifted_against_each_other(kind, shift, scale):
    """A shift of one side's logits leaves its logprobs as they are."""
    rng = np.random.default_rng(42)
    rows, vocab = 5, 30000
    ids = rng.integers(0, vocab, rows).astype(np.int32)
    c = {} if scale is None else {"scale": np.full(rows, scale, np.float32)}
    x = rng.normal(0, 3, (rows, vocab))
    xt, yt = tensor(x, kind), tensor(x + shift, kind)
    check_float64(c, c, xt, yt, ids, score_sides(c, c, xt, yt, ids))


@pytest.mark.parametrize("side", ["train", "rollout"])
def test_score_one_side_rising(side):
    """One side rises by 5 with each of a thread's tiles and the other stays, at a scale of 4: the rising side's
    maximum may not carry the other's reference along."""
    rng = np.random.default_rng(43)
    rows, vocab = 4, 57344
    ids = rng.integers(0, vocab, rows).astype(np.int32)
    c = {"scale": np.full(rows, 4, np.float32)}
    flat = rng.normal(0, 1, (rows, vocab))
    flat, rising = tensor(flat, "f32"), tensor(flat + 5.0 * (np.arange(vocab) // 8192), "f32")
    x, y = (rising, flat) if side == "train" else (flat, rising)
    check_float64(c, c, x, y, ids, score_sides(c, c, x, y, ids))


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("offset", [60.0, 500.0, 1000.0, -700.0])
@pytest.mark.parametrize("scale", [None, 10.0])
def test_score_of_logits_with_an_offset(kind, offset, scale):
    """A row's common offset is not part of its spread, so the logprobs' error may not grow with it."""
    rng = np.random.default_rng(44)
    rows, vocab = 5, 60000
    ids = rng.integers(0, vocab, rows).astype(np.int32)
    c = {} if scale is None else {"scale": np.full(rows, scale, np.float32)}
    x = rng.normal(0, 3, (rows, vocab)) + offset
    xt, yt = tensor(x, kind), tensor(x + rng.normal(0, 2e-3, x.shape), kind)
    check_float64(c, c, xt, yt, ids, score_sides(c, c, xt, yt, ids))
    check_float64(c, c, xt, xt, ids, score_sides(c, c, xt, xt, ids))


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("offset", [0.0, 60.0, 1000.0, -700.0])
@pytest.mark.parametrize("scale", [1.0, 10.0])
@pytest.mark.parametrize("vocab", [9001, 20000])
def test_gradient_of_logits_with_an_offset(kind, offset, scale, vocab):
    """The bound of test_gradient holds wherever the row lies; some columns touched, one row's token far below
    the peak."""
    rng = np.random.default_rng(45)
    rows = 5
    x = tensor(rng.normal(0, 3, (rows, vocab)) + offset, kind)
    xh = host(x)
    ids = np.argsort(xh, 1)[:, -7].astype(np.int32)
    ids[1] = np.argmin(xh[1])
    c = {"scale": np.full(rows, scale, np.float32), "bias_ids": ids[:, None] + np.array([[0, -1, 1]], np.int32),
         "bias": rng.normal(0, 0.5, (rows, 3)).astype(np.float32)}
    lp = np.array([ref.logp(ref.row(c, xh[r], r)[0], ids[r]) for r in range(rows)]).astype(np.float32)
    g = rng.normal(0, 1, rows).astype(np.float32)
    act = np.ones(rows, np.uint8)
    out = torch.empty(rows, vocab, device=DEV)
    B.lpd_logprob_backward_controlled(x, to_device(c), *(torch.from_numpy(v).to(DEV) for v in (ids, act, lp, g)), out)
    got = host(out)
    for r in range(rows):
        z, slope = ref.row(c, xh[r], r)
        p = np.exp(z - z[ids[r]] + np.float64(lp[r]))
        hot = np.arange(vocab) == ids[r]
        want = g[r] * slope * (hot - p)
        # (a p below float32's smallest normal number, 2^-126, becomes 0: exponents are flushed)
        tol = np.abs(g[r] * slope) * (1e-5 * p + 2.0 ** -24 * hot + 2.0 ** -126) + 2.0 ** -21 * np.abs(want)
        assert np.all(np.abs(got[r] - want) <= tol), (r, np.max(np.abs(got[r] - want) - tol))


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("scale", [1e-38, 1e-30, 1e-20, 1e6, 1e20, 1e37, 3e38])
def test_scales_at_the_ends_of_their_range(kind, scale):
    """Any finite scale > 0: nothing masked counts at a tiny one, equal maxima share the sum at a huge one."""
    rng = np.random.default_rng(46)
    rows, vocab = 4, 20000
    # (the differences times the scale stay inside float32, as the logprobs have to)
    x = rng.integers(-60, 60, (rows, vocab)) / 64
    top = tensor(x, kind)
    xh = host(top)
    words = rng.integers(0, 1 << 32, (rows, vocab // 32), dtype=np.uint64).astype(np.uint32)
    ids = np.array([rng.choice(np.flatnonzero(xh[r] == xh[r].max())) for r in range(rows)], np.int32)
    for r in range(rows):
        words[r, ids[r] // 32] |= np.uint32(1 << (ids[r] % 32))
    c = {"scale": np.full(rows, scale, np.float32), "mask": words.view(np.int32)}
    if scale < 1e38:  # (else the logprob passes float32)
        ids[1] = np.flatnonzero(np.isfinite(ref.row(c, xh[1], 1)[0]) & (xh[1] < 0.3) & (xh[1] > 0.2))[0]
    s = score_sides(c, c, top, top, ids)
    check_float64(c, c, top, top, ids, s)
    y = tensor(x + rng.integers(0, 2, x.shape) / 128, kind)
    check_float64(c, c, top, y, ids, score_sides(c, c, top, y, ids))
    g = torch.ones(rows, device=DEV)
    out = torch.empty(rows, vocab, device=DEV)
    act = torch.ones(rows, dtype=torch.uint8, device=DEV)
    B.lpd_logprob_backward_controlled(top, to_device(c), torch.from_numpy(ids).to(DEV), act, s.logp_train, g, out)
    got, lp = host(out), host(s.logp_train)
    for r in (0, 2, 3):  # (row 1's logprob says little about the others' where the scale is huge)
        z, slope = ref.row(c, xh[r], r)
        p = np.exp(z - z[ids[r]] + lp[r])
        hot = np.arange(vocab) == ids[r]
        want = slope * (hot - p)
        tol = np.abs(slope) * (1e-5 * p + 2.0 ** -24 * hot) + 2.0 ** -21 * np.abs(want)
        assert np.all(np.abs(got[r] - want) <= tol + 1e-37), (r, np.max(np.abs(got[r] - want) - tol))


def test_a_bias_of_minus_infinity_bans_a_token():
    """Alone, beside another bias of the same token, and on a token with a penalty."""
    rng = np.random.default_rng(52)
    rows, vocab = 4, 5000
    x = rng.normal(0, 3, (rows, vocab))
    xt = tensor(x, "bf16")
    ids = rng.integers(100, vocab, rows).astype(np.int32)
    c = ref.random_controls(rng, rows, vocab, keep=ids, history=50, masks=0, bias=0)
    c["history"][:20] = np.arange(20)
    c["hist_begin"][:], c["hist_split"][:], c["hist_end"][:] = 0, 5, 40
    c["bias_ids"] = np.tile(np.array([[7, 30, 30, 2, 50]], np.int32), (rows, 1))
    c["bias"] = np.tile(np.array([[-np.inf, -np.inf, 4.0, -np.inf, 1.0]], np.float32), (rows, 1))
    h = to_device(c)
    out = B.controls_apply(xt, h, torch.float32)
    check_apply(c, xt, "f32", out)
    assert bool(torch.isneginf(out[:, [7, 30, 2]]).all()) and int(torch.isinf(out).sum()) == 3 * rows
    act = np.ones(rows, np.uint8)
    for ct, cr, ht, hr in ((c, c, h, h), (c, {}, h, None)):
        s = B.score_controlled(xt, xt, torch.from_numpy(ids).to(DEV), torch.from_numpy(act).to(DEV), ht, hr)
        check_float64(ct, cr, xt, xt, ids, s)
    dx = torch.empty(rows, vocab, device=DEV)
    B.lpd_logprob_backward_controlled(xt, h, torch.from_numpy(ids).to(DEV), torch.from_numpy(act).to(DEV),
                                      B.score_controlled(xt, xt, torch.from_numpy(ids).to(DEV), torch.from_numpy(act).to(DEV), h, h).logp_train,
                                      torch.ones(rows, device=DEV), dx)
    assert bool(torch.isfinite(dx).all()) and bool((dx[:, [7, 30, 2]] == 0).all())


@pytest.mark.parametrize("name", ["frequency", "presence"])
def test_an_infinite_penalty_bans_repeats(name):
    """x1 - inf is -inf for the generated tokens; frequency * 0 is not formed for the prompt's."""
    rng = np.random.default_rng(53)
    rows, vocab = 3, 3000
    xt = tensor(rng.normal(0, 3, (rows, vocab)), "f32")
    ids = rng.integers(100, vocab, rows).astype(np.int32)
    c = ref.random_controls(rng, rows, vocab, keep=ids, history=40, masks=0, bias=0, parts=("repetition", "frequency", "presence"))
    c["history"][:] = np.arange(41)
    c["hist_begin"][:], c["hist_split"][:], c["hist_end"][:] = 0, 20, 40
    c[name][:] = np.inf
    c["bias_ids"], c["bias"] = np.full((rows, 1), 25, np.int32), np.full((rows, 1), 3.0, np.float32)
    h = to_device(c)
    out = B.controls_apply(xt, h)
    check_apply(c, xt, "f32", out)
    assert bool(torch.isneginf(out[:, 20:40]).all()) and int(torch.isinf(out).sum()) == 20 * rows
    check_float64(c, c, xt, xt, ids, score_sides(c, c, xt, xt, ids))


@pytest.mark.parametrize("rows,vocab,kind", [(1, 129025, "bf16"), (1, 129031, "f32"), (2, 172033, "bf16"), (2, 172001, "f32"),
                                             (160, 172033, "bf16"), (160, 172040, "bf16"), (160, 172001, "f32")])
def test_elementwise_forms_at_the_seams_of_their_units(rows, vocab, kind):
    """Last units of a few columns, and rows longer than a unit where rows are many: on 16-byte boundaries and off
    them, in place too."""
    rng = np.random.default_rng(vocab)
    x = rng.normal(0, 1, (rows, vocab)).astype(np.float32)
    xt = tensor(x, kind)
    ids = np.full(rows, vocab - 1, np.int32)
    ids[rows // 2:] = rng.integers(0, vocab, rows - rows // 2)
    c = ref.random_controls(rng, rows, vocab, keep=ids, history=300, masks=2, bias=4)
    c["history"][:30] = np.arange(vocab - 30, vocab)
    c["hist_begin"][:], c["hist_split"][:], c["hist_end"][:] = 0, 10, 280
    h = to_device(c)
    out = B.controls_apply(xt, h)
    some = sorted({0, rows // 2, rows - 1})
    sub = lambda v: v[some] if len(v) == rows else v  # noqa: E731
    cs = {k: (v if k in ("history", "mask") else sub(v)) for k, v in c.items()}
    check_apply(cs, xt[some], kind, out[some])
    again = xt.clone()
    B.lpd_controls_apply(again, h, again)
    assert torch.equal(again, out)
    lp = np.zeros(rows, np.float32)
    lp[some] = [ref.logp(ref.row(cs, host(xt[r:r + 1])[0], i)[0], ids[r]) for i, r in enumerate(some)]
    g = rng.normal(0, 1, rows).astype(np.float32)
    act = np.ones(rows, np.uint8)
    dx = torch.empty(rows, vocab, device=DEV)
    B.lpd_logprob_backward_controlled(xt, h, *(torch.from_numpy(v).to(DEV) for v in (ids, act, lp, g)), dx)
    for i, r in enumerate(some):
        z, slope = ref.row(cs, host(xt[r:r + 1])[0], i)
        p = np.exp(z - z[ids[r]] + np.float64(lp[r]))
        hot = np.arange(vocab) == ids[r]
        want = g[r] * slope * (hot - p)
        tol = np.abs(g[r] * slope) * (1e-5 * p + 2.0 ** -24 * hot + 2.0 ** -126) + 2.0 ** -21 * np.abs(want)
        assert np.all(np.abs(host(dx[r:r + 1])[0] - want) <= tol), r


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_score_of_rows_longer_than_a_unit(kind):
    """More than 172032 columns with many rows, two units each, under controls that reach into both."""
    rng = np.random.default_rng(51)
    rows, vocab = 320, 200003
    x = torch.randn(rows, vocab, device=DEV, generator=torch.Generator(DEV).manual_seed(51)).to(KINDS[kind])
    y = (x.float() + 1e-3).to(KINDS[kind])
    ids = rng.integers(0, vocab, rows).astype(np.int32)
    ids[::3] = rng.integers(172032, vocab, len(ids[::3]))
    c = ref.random_controls(rng, rows, vocab, keep=ids, history=3000, masks=3, bias=5)
    h = to_device(c)
    act = np.ones(rows, np.uint8)
    res = B.score_controlled(x, y, torch.from_numpy(ids).to(DEV), torch.from_numpy(act).to(DEV), h, h)
    assert res.metrics["status"] == 0
    for r in (0, 3, 151, 152, 319):
        for v, got in ((x, res.logp_train), (y, res.logp_rollout)):
            want = ref.logp(ref.row(c, host(v[r:r + 1])[0], r)[0], ids[r])
            assert abs(float(got[r]) - want) <= 1e-5 + 2.0 ** -23 * abs(want), r
    at = np.array([3, 152, 319])
    few = to_device({k: (v if k in ("history", "mask") else v[at]) for k, v in c.items()})
    part = B.score_controlled(x[at], y[at], torch.from_numpy(ids[at]).to(DEV), torch.ones(3, dtype=torch.uint8, device=DEV), few, few)
    for k in ("logp_train", "logp_rollout", "dlogp"):
        assert torch.equal(getattr(res, k)[at], getattr(part, k)), k


def test_zero_rows():
    x = torch.empty(0, 300, device=DEV)
    none = lambda t: torch.empty(0, dtype=t, device=DEV)  # noqa: E731
    s = B.score_controlled(x, x, none(torch.int32), none(torch.uint8), B.Controls(scale=none(torch.float32)))
    assert s.metrics["n_active"] == 0 and s.metrics["flags"] & B.LPD_FLAG_NO_ACTIVE
    B.lpd_logprob_backward_controlled(x, None, none(torch.int32), none(torch.uint8), none(torch.float32), none(torch.float32), x.clone())


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("low", [-3e38, -1e35])
def test_touched_tokens_of_the_lowest_logits(kind, low):
    """A penalised token far below the others has a rounding error, the two floats' lower part, of 1e28 and more:
    it may not count beside the reference."""
    rng = np.random.default_rng(61)
    rows, vocab = 6, 1200
    x = rng.normal(0, 1, (rows, vocab))
    where = rng.random(x.shape) < 0.9
    ids = rng.integers(0, vocab, rows).astype(np.int32)
    where[np.arange(rows), ids] = False
    y = x + 1e-3
    x[where], y[where] = low, -np.inf
    c = ref.random_controls(rng, rows, vocab, history=300, masks=0, bias=3)
    c["repetition"][:] = [0.77, 0.9, 0.99, 1.01, 1.1, 0.7]
    for a, b in ((x, y), (y, x), (x, x)):
        xt, yt = tensor(a, kind), tensor(b, kind)
        for ct, cr in ((c, c), (c, {}), ({}, c)):
            with np.errstate(invalid="ignore"):
                check_float64(ct, cr, xt, yt, ids, score_sides(ct, cr, xt, yt, ids))


@pytest.mark.parametrize("scale", [1e8, 1e12, 1e30])
def test_touched_tokens_at_huge_scales(scale):
    """A touched token that is the largest has a logprob of 0, and far below it the scaled gap, to float32's
    rounding of the logits."""
    rng = np.random.default_rng(62)
    rows, vocab = 5, 3000
    x = rng.normal(0, 1, (rows, vocab)).astype(np.float32)
    ids = np.array([17, 18, 19, 20, 21], np.int32)
    x[np.arange(rows), ids] = 9.1 + rng.random(rows)
    c = {"scale": np.full(rows, scale, np.float32), "history": ids, "hist_begin": np.arange(rows), "hist_split": np.arange(rows),
         "hist_end": np.arange(rows) + 1, "repetition": np.full(rows, 1.3, np.float32), "presence": np.full(rows, 0.1, np.float32)}
    c = {k: v.astype(np.int64) if k.startswith("hist_") else v for k, v in c.items()}
    t = tensor(x, "f32")
    s = score_sides(c, c, t, t, ids)
    assert s.metrics["status"] == 0 and bool((s.logp_train.abs() <= 1e-5).all()) and bool((s.dlogp == 0).all())
    other = np.array([40, 41, 42, 43, 44], np.int32)
    s = score_sides(c, c, t, t, other)
    for r in range(rows):
        z, _ = ref.row(c, host(t)[r], r)
        want = ref.logp(z, other[r])
        # the largest logit, rounded to float32 where the scale leaves no room for its lower part
        assert abs(float(s.logp_train[r]) - want) <= 2.0 ** -23 * abs(want) + 2.0 ** -24 * abs(z.max())


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("scale", [20.0, 50.0, 300.0])
def test_score_of_a_sharp_side_beside_a_flat_one(kind, scale):
    """One side's sum is a few terms from the start. The other's is thousands until its dominant token, a biased
    one, is met: the rounding of those may not stay in the difference of the logprobs."""
    rng = np.random.default_rng(63)
    rows, vocab = 20, 30000
    ids = rng.integers(0, vocab, rows).astype(np.int32)
    t = tensor(rng.normal(0, 1, (rows, vocab)), kind)
    sharp = {"scale": np.full(rows, scale, np.float32)}
    flat = {"bias_ids": ids[:, None], "bias": np.full((rows, 1), 40.0, np.float32)}
    check_float64(sharp, flat, t, t, ids, score_sides(sharp, flat, t, t, ids))
    check_float64(flat, sharp, t, t, ids, score_sides(flat, sharp, t, t, ids))


@pytest.mark.parametrize("xk,yk", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("vocab", [600, 9003, 57346])
def test_column_slices(xk, yk, vocab):
    """Rows that start anywhere in a wider tensor, the sides and the output at different places: the same bits as
    dense ones, nothing written around them."""
    rng = np.random.default_rng(71)
    rows = 5
    ids = rng.integers(0, vocab, rows).astype(np.int32)
    h = to_device(ref.random_controls(rng, rows, vocab, keep=ids, history=300))
    x = tensor(rng.normal(0, 3, (rows, vocab)), xk)
    y = (x.float() + 2e-3).to(KINDS[yk])

    def sliced(t, lead, behind):
        wide = torch.full((rows + 2, lead + vocab + behind), 7.0, dtype=t.dtype, device=DEV)
        wide[1:-1, lead:lead + vocab] = t
        return wide, wide[1:-1, lead:lead + vocab]

    idt, act = torch.from_numpy(ids).to(DEV), torch.ones(rows, dtype=torch.uint8, device=DEV)
    dense = B.score_controlled(x, y, idt, act, h, h)
    want = B.controls_apply(x, h)
    g = torch.randn(rows, device=DEV)
    grad = torch.empty(rows, vocab, device=DEV)
    B.lpd_logprob_backward_controlled(x, h, idt, act, dense.logp_train, g, grad)
    for a, b, o in ((3, 6, 1), (1, 0, 5), (8, 5, 0)):
        (_, xs), (_, ys) = sliced(x, a, 2), sliced(y, b, 3)
        s = B.score_controlled(xs, ys, idt, act, h, h)
        for k in ("logp_train", "logp_rollout", "dlogp"):
            assert torch.equal(getattr(s, k), getattr(dense, k)), (k, a, b)
        for wide, out in (sliced(torch.zeros_like(x), o, a), sliced(torch.zeros_like(grad), o, b)):
            guard = wide.clone()
            if out.dtype == torch.float32:
                B.lpd_logprob_backward_controlled(xs, h, idt, act, dense.logp_train, g, out)
                # A column at a unit's edge is a scout's or the stream's by its place; exponents to -126 carry
                # three roundings of 2^-24 in each, 126 * 3 * 2^-24 * ln 2 = 1.6e-5 of p.
                assert bool(((out - grad).abs() <= 4e-5 * (grad.abs() + 2.0 ** -126)).all())
            if out.dtype == x.dtype:
                B.lpd_controls_apply(xs, h, out)
                assert torch.equal(out, want)
            out.zero_()
            assert torch.equal(wide, guard)
