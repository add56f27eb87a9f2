"""What the sampling filters keep of a row and what a draw gives, in float64, from
the definition (include/lpd.h, lpd_filter)."""
import math

import numpy as np


def row(x, scale=1.0, min_p=0.0, top_k=0, top_p=1.0):
    """(z, kept, margin) of one row of logits, or None where it has no distribution.

    margin: how near the top-p border lies to a sum, relative to the whole mass."""
    x = np.asarray(x, dtype=np.float64)
    if np.isnan(x).any() or np.isposinf(x).any() or np.isneginf(x).all():
        return None
    if not (np.isfinite(scale) and scale > 0) or math.isnan(min_p) or math.isnan(top_p):
        return None
    z = x * scale
    order = np.argsort(-x, kind="stable")
    order = order[np.isfinite(x[order])]
    top = z[order[0]]
    if min_p > 0:
        order = order[(x[order] - x[order[0]]) * scale >= math.log(min(min_p, 1.0))]
    if 0 < top_k < len(x):
        order = order[:top_k]
    margin = 1.0
    if top_p < 1:
        mass = np.exp(z[order] - top)
        upto = np.cumsum(mass)
        want = max(top_p, 0.0) * upto[-1]
        n = 1 + int(np.sum(upto < want)) if want > 0 else 1
        margin = float(np.min(np.abs(upto - want)) / upto[-1]) if want > 0 else 1.0
        order = order[:min(n, len(order))]
    kept = np.zeros(len(x), dtype=bool)
    kept[order] = True
    return z, kept, margin


def lse(z, kept):
    top = z[kept].max()
    return top + math.log(np.sum(np.exp(z[kept] - top)))


def draw(z, kept, u):
    """(token, logprob, margin) of the draw with u."""
    top = z[kept].max()
    mass = np.where(kept, np.exp(np.where(kept, z, top) - top), 0.0)
    upto = np.cumsum(mass)
    want = min(max(u, 0.0), 1.0) * upto[-1]
    passed = np.nonzero((upto > want) & kept)[0]
    j = int(passed[0]) if len(passed) else int(np.nonzero(kept)[0][-1])
    return j, z[j] - lse(z, kept), float(np.min(np.abs(upto - want)) / upto[-1]) if u > 0 else 1.0


def bits(mask, vocab):
    """bool [rows, vocab] of int32 words."""
    words = np.ascontiguousarray(mask).view(np.uint32)
    return ((words[:, :, None] >> np.arange(32, dtype=np.uint32)) & 1).reshape(len(words), -1)[:, :vocab] != 0
