"""Sampling controls in numpy float64, one row at a time, and random inputs for
the tests.  Written from the definition in include/lpd.h."""
from __future__ import annotations

import numpy as np


def clamp_range(c, r):
    n = len(c["history"])
    end = min(max(int(c["hist_end"][r]), 0), n)
    begin = min(max(int(c["hist_begin"][r]), 0), end)
    split = min(max(int(c["hist_split"][r]), begin), end)
    return begin, split, end


def row(c, x, r):
    """(z, slope): row r's controlled logits and dz/dx, from its float64 logits x.
    c: dict of numpy arrays named as lpd_controls' fields (missing: left out)."""
    V = len(x)
    z = x.astype(np.float64).copy()
    slope = np.ones(V)
    one = lambda name, neutral: float(c[name][r]) if name in c else neutral  # noqa: E731
    if "history" in c and any(k in c for k in ("repetition", "frequency", "presence")):
        begin, split, end = clamp_range(c, r)
        rep, freq, pres = one("repetition", 1.0), one("frequency", 0.0), one("presence", 0.0)
        for j in sorted(set(c["history"][begin:end].tolist())):
            if 0 <= j < V:
                f = 1.0 / rep if z[j] > 0 else rep
                z[j] *= f
                slope[j] = f
                n = int(np.sum(c["history"][split:end] == j))
                if n:
                    z[j] -= freq * n + pres
    if "bias_ids" in c:
        for j, b in zip(c["bias_ids"][r].tolist(), c["bias"][r].tolist()):
            if 0 <= j < V:
                z[j] += b
    s = one("scale", 1.0)
    z *= s
    slope *= s
    if "mask" in c:
        k = int(c["mask_row"][r]) if "mask_row" in c else r
        if k >= 0:
            words = c["mask"][k].astype(np.int64) & 0xFFFFFFFF if k < len(c["mask"]) else np.zeros((V + 31) // 32, np.int64)
            j = np.arange(V)
            off = (words[j // 32] >> (j % 32)) & 1 == 0
            z[off] = -np.inf
            slope[off] = 0.0
    return z, slope


def logp(z, j):
    m = z.max()
    return float(z[j] - m - np.log(np.sum(np.exp(z - m))))


def random_controls(rng, rows, vocab, *, history=50, bias=3, masks=2, keep=None, parts=("repetition", "frequency", "presence", "scale")):
    """Random controls of every kind as numpy arrays.  keep: ids[rows] that stay allowed."""
    c = {}
    if history is not None:
        tokens = rng.integers(-2, vocab + 2, size=history + 1) if vocab > 4 else rng.integers(0, vocab, size=history + 1)
        tokens[::3] = tokens[0]  # one token many times
        c["history"] = tokens.astype(np.int32)
        a, b, d = np.sort(rng.integers(0, history + 2, size=(3, rows)), axis=0)
        c["hist_begin"], c["hist_split"], c["hist_end"] = (v.astype(np.int64) for v in (a, b, d))
    lo_hi = {"repetition": (0.7, 1.5), "frequency": (-0.3, 0.5), "presence": (-1, 1), "scale": (0.5, 2)}
    for name in parts:
        lo, hi = lo_hi[name]
        c[name] = rng.uniform(lo, hi, rows).astype(np.float32)
    if bias:
        ids = rng.integers(-1, vocab + 1, size=(rows, bias))
        ids[:, -1] = ids[:, 0]  # the same id twice
        c["bias_ids"] = ids.astype(np.int32)
        c["bias"] = rng.normal(0, 3, (rows, bias)).astype(np.float32)
    if masks:
        words = (vocab + 31) // 32
        allowed = rng.random((masks, words * 32)) < 0.6
        c["mask_row"] = rng.integers(-1, masks, rows).astype(np.int32)
        if keep is not None:
            for r in range(rows):
                if c["mask_row"][r] >= 0:
                    allowed[c["mask_row"][r], keep[r]] = True
        bits = (allowed.reshape(masks, words, 32).astype(np.uint64) << np.arange(32, dtype=np.uint64)).sum(2)
        c["mask"] = bits.astype(np.uint32).view(np.int32)
    return c
