"""Cases of the sampling controls (penalties, biases, grammar masks on logits) and of the 8-bit block-scaled
product: their inputs, the calls that a user makes, and the same computations in elementary torch operations.

A case is one call with its sizes.  ``run`` computes it in the plain form, or with ``own`` through the
library's entry points; ``exact`` gives the result of the definition in float64.
"""
import math

import torch

own = False

DEV = "cuda"
BLOCK = 128            # values that share one scale along k
FLOOR = 2.0 ** -64     # smallest magnitude that a scale is made for
FP8 = {"e4m3": (torch.float8_e4m3fn, 448.0), "e5m2": (torch.float8_e5m2, 57344.0)}
FLOATS = {"bf16": torch.bfloat16, "f32": torch.float32}
CLIP = (0.8, 1.2)


# ---- cases ---------------------------------------------------------------------------------------

def listed():
    return [
        # the next token of a single request under penalties and a grammar: latency
        {"name": "apply-one-row", "op": "apply", "seqs": 1, "gen": 1, "teacher": False, "vocab": 128256, "pad": 0,
         "x": "bf16", "out": "f32", "prompt": 300, "history": 600, "bias": 0, "masks": 1},
        # the next token of a serving batch with long conversations, request biases and grammar states
        {"name": "apply-batch", "op": "apply", "seqs": 256, "gen": 1, "teacher": False, "vocab": 151936, "pad": 0,
         "x": "bf16", "out": "bf16", "prompt": 4096, "history": 8192, "bias": 64, "masks": 32},
        # a unit batch of the scorer: latency
        {"name": "score-tiny", "op": "score", "seqs": 2, "gen": 64, "teacher": True, "vocab": 1024, "pad": 0,
         "x": "bf16", "y": "bf16", "prompt": 16, "history": 0, "bias": 4, "masks": 8},
        # an odd vocabulary with rows on no 16-byte boundary, a rollout kept in float32
        {"name": "score-odd", "op": "score", "seqs": 3, "gen": 211, "teacher": True, "vocab": 50021, "pad": 1,
         "x": "bf16", "y": "f32", "prompt": 100, "history": 0, "bias": 0, "masks": 64},
        # teacher-forced rollouts of the benchmark's vocabulary: every row has its own prefix
        {"name": "score-long", "op": "score", "seqs": 4, "gen": 1024, "teacher": True, "vocab": 151936, "pad": 0,
         "x": "bf16", "y": "bf16", "prompt": 512, "history": 0, "bias": 16, "masks": 128},
        # the gradient of an odd batch in float32
        {"name": "backward-odd", "op": "backward", "seqs": 2, "gen": 130, "teacher": True, "vocab": 32003, "pad": 2,
         "x": "f32", "out": "f32", "prompt": 60, "history": 0, "bias": 3, "masks": 0},
        # the gradient of a training step's rows
        {"name": "backward-long", "op": "backward", "seqs": 4, "gen": 512, "teacher": True, "vocab": 151936, "pad": 0,
         "x": "bf16", "out": "bf16", "prompt": 512, "history": 0, "bias": 16, "masks": 64},
        # the hidden rows in front of the 8-bit head
        {"name": "quantize-hidden", "op": "quantize", "rows": 1024, "cols": 4096, "x": "bf16", "fp8": "e4m3",
         "block": False, "transpose": False, "pow2": False},
        # the head's weight laid out for the data gradient
        {"name": "quantize-weight", "op": "quantize", "rows": 151936, "cols": 4096, "x": "bf16", "fp8": "e4m3",
         "block": True, "transpose": True, "pow2": True},
        # the head over a decode batch
        {"name": "matmul-decode", "op": "matmul", "m": 16, "n": 151936, "k": 4096, "a": "e4m3", "b": "e4m3",
         "a_block": False, "b_block": True, "out": "bf16"},
        # the head over the rows of a scoring batch
        {"name": "matmul-head", "op": "matmul", "m": 4096, "n": 128256, "k": 4096, "a": "e4m3", "b": "e4m3",
         "a_block": False, "b_block": True, "out": "bf16"},
        # the weight gradient of one vocabulary shard over an odd number of tokens
        {"name": "matmul-wgrad", "op": "matmul", "m": 37984, "n": 4096, "k": 2051, "a": "e5m2", "b": "e4m3",
         "a_block": False, "b_block": False, "out": "f32"},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["apply", "apply", "score", "score", "backward", "quantize", "matmul", "matmul", "matmul"])
    if op == "quantize":
        rows = _log(rng, 1, 151936)
        return {"op": op, "rows": rows, "cols": _log(rng, 1, min(16384, 151936 * 4096 // rows)), "x": rng.choice(["bf16", "f32"]) if rows < 60000 else "bf16",
                "fp8": rng.choice(["e4m3", "e4m3", "e5m2"]), "block": rng.random() < 0.5, "transpose": rng.random() < 0.5,
                "pow2": rng.random() < 0.5}
    if op == "matmul":
        kind = rng.choice(["head", "data", "weight"])  # the product's three uses
        tokens = _log(rng, 1, 4096)
        vocab, hidden = _log(rng, 1000, 128256), _log(rng, 64, 4096)
        m, n, k = {"head": (tokens, vocab, hidden), "data": (tokens, hidden, vocab), "weight": (vocab, hidden, tokens)}[kind]
        return {"op": op, "m": m, "n": n, "k": k, "a": "e4m3" if kind == "head" else rng.choice(["e4m3", "e5m2"]), "b": "e4m3",
                "a_block": False, "b_block": kind != "weight", "out": "f32" if kind == "weight" else rng.choice(["bf16", "f32"])}
    vocab = rng.choice([1024, 37984, 128256, 151936, _log(rng, 1000, 151936), _log(rng, 1000, 151936)])
    teacher = op != "apply"
    rows = _log(rng, 1, {"apply": 256, "score": 4096, "backward": 2048}[op])
    seqs = min(rows, rng.randint(1, 6)) if teacher else rows
    prompt = _log(rng, 1, 512)
    case = {"op": op, "seqs": seqs, "gen": max(1, rows // seqs) if teacher else 1, "teacher": teacher, "vocab": vocab,
            "pad": rng.choice([0, 0, 1, 8, 24]), "x": rng.choice(["bf16", "bf16", "f32"]) if op != "score" else "bf16",
            "prompt": prompt, "history": 0 if teacher else prompt + _log(rng, 1, 7000), "bias": rng.choice([0, 1, 7, 64]),
            "masks": rng.choice([0, 1, 40])}
    if op == "score":
        case["y"] = "bf16" if seqs * case["gen"] > 2000 else rng.choice(["bf16", "f32"])
    else:
        case["out"] = "bf16" if case["x"] == "bf16" and op == "backward" else rng.choice(["bf16", "f32"]) if case["x"] == "bf16" else case["x"]
    return case


# ---- what a call has to read, write and compute --------------------------------------------------

def _bytes(name):
    return {"bf16": 2, "f32": 4, "e4m3": 1, "e5m2": 1}[name]


def _active(rows):
    return rows - rows // 10 if rows > 10 else rows


def work(case):
    if case["op"] == "quantize":
        r, c = case["rows"], case["cols"]
        return {"bytes": r * c * (_bytes(case["x"]) + 1) + 4 * (r * c // (BLOCK * (BLOCK if case["block"] else 1)))}
    if case["op"] == "matmul":
        m, n, k = case["m"], case["n"], case["k"]
        kb = -(-k // BLOCK)
        scales = 4 * kb * ((m if not case["a_block"] else -(-m // BLOCK)) + (n if not case["b_block"] else -(-n // BLOCK)))
        return {"bytes": (m + n) * k + scales + m * n * _bytes(case["out"]), "flops": 2 * m * n * k}
    rows, vocab = case["seqs"] * case["gen"], case["vocab"]
    active = _active(rows) if case["op"] != "apply" else rows
    tokens = 4 * case["seqs"] * (case["prompt"] + case["gen"] if case["teacher"] else case["history"])
    side = tokens + min(rows, case["masks"]) * -(-vocab // 32) * 4 + rows * (24 + 16 + 4 + 8 * case["bias"])
    if case["op"] == "apply":
        return {"bytes": rows * vocab * (_bytes(case["x"]) + _bytes(case["out"])) + side, "flops": rows * vocab}
    if case["op"] == "score":
        return {"bytes": active * vocab * (_bytes(case["x"]) + _bytes(case["y"])) + side + rows * 17, "flops": 8 * active * vocab}
    return {"bytes": active * vocab * _bytes(case["x"]) + rows * vocab * _bytes(case["out"]) + side + rows * 13, "flops": 5 * active * vocab}


# ---- inputs --------------------------------------------------------------------------------------

def _tokens(g, shape, vocab):
    """Token ids with many repeats, as in text."""
    u = torch.rand(shape, generator=g, device=DEV)
    return (u.pow(6) * vocab).long().clamp_(max=vocab - 1).to(torch.int32)


def _controls(case, g, rows, ids):
    """The rows' controls: a shared token buffer with each row's range of it, the request's parameters, its
    biases and its grammar state.  ``ids`` (the rows' own next tokens) are kept allowed."""
    seqs, gen, vocab, prompt = case["seqs"], case["gen"], case["vocab"], case["prompt"]
    c = {}
    seq = torch.arange(rows, device=DEV) // gen
    step = torch.arange(rows, device=DEV) % gen
    if case["teacher"]:
        text = _tokens(g, (seqs, prompt + gen), vocab)
        text[:, prompt:] = ids.view(seqs, gen)
        c["history"] = text.reshape(-1)
        c["hist_begin"] = seq * (prompt + gen)
        c["hist_split"] = c["hist_begin"] + prompt
        c["hist_end"] = c["hist_split"] + step
    else:
        longest = case["history"]
        c["history"] = _tokens(g, (seqs * longest,), vocab)
        c["hist_begin"] = seq * longest
        c["hist_split"] = c["hist_begin"] + min(prompt, longest)
        c["hist_end"] = c["hist_begin"] + torch.randint(1, longest + 1, (rows,), generator=g, device=DEV)
        c["hist_split"] = torch.minimum(c["hist_split"], c["hist_end"])

    def per_request(lo, hi):
        return (lo + (hi - lo) * torch.rand(seqs, generator=g, device=DEV))[seq].contiguous()

    c["repetition"], c["frequency"], c["presence"] = per_request(1.0, 1.3), per_request(0.0, 0.2), per_request(-0.5, 1.0)
    c["scale"] = per_request(0.8, 1.6)
    if case["bias"]:
        b = _tokens(g, (seqs, case["bias"]), vocab)[seq].contiguous()
        b[::7, -1] = -1  # a row that uses fewer of its entries
        c["bias_ids"], c["bias"] = b, torch.randn(rows, case["bias"], generator=g, device=DEV) * 2
    if case["masks"]:
        states, words = case["masks"], -(-vocab // 32)
        allowed = torch.rand(states, words * 32, generator=g, device=DEV) < torch.rand(states, 1, generator=g, device=DEV).clamp_(min=0.02)
        c["mask_row"] = torch.randint(-1, states, (rows,), generator=g, device=DEV, dtype=torch.int32)
        allowed[c["mask_row"].long().clamp(min=0), ids.long()] = True
        w = (allowed.view(states, words, 32).long() << torch.arange(32, device=DEV)).sum(2)
        c["mask"] = torch.where(w >= 2 ** 31, w - 2 ** 32, w).to(torch.int32)
    return c


def _padded(x, pad):
    if not pad:
        return x
    wide = torch.full((x.shape[0], x.shape[1] + pad), float("nan"), dtype=x.dtype, device=DEV)
    wide[:, :x.shape[1]] = x
    return wide[:, :x.shape[1]]


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    if case["op"] == "quantize":
        x = torch.randn(case["rows"], case["cols"], generator=g, device=DEV, dtype=FLOATS[case["x"]])
        x *= torch.rand(case["rows"], 1, generator=g, device=DEV).add_(0.2).to(x.dtype)
        return {"case": case, "x": x}
    if case["op"] == "matmul":
        s = {"case": case}
        for side, rows in (("a", case["m"]), ("b", case["n"])):
            x = torch.randn(rows, case["k"], generator=g, device=DEV, dtype=torch.bfloat16)
            q, s[side + "_scales"] = _plain_quantize(x, case[side], case[side + "_block"], False, False)
            wide = torch.zeros(rows, -(-case["k"] // 16) * 16, dtype=torch.uint8, device=DEV)
            wide[:, :case["k"]] = q.view(torch.uint8)
            s[side] = wide.view(FP8[case[side]][0])[:, :case["k"]]
        return s
    rows, vocab = case["seqs"] * case["gen"], case["vocab"]
    ids = _tokens(g, (rows,), vocab)
    x = torch.randn(rows, vocab, generator=g, device=DEV, dtype=torch.float32).mul_(3.0)
    x[::100, vocab // 3] += 15
    s = {"case": case, "ids": ids, "controls": _controls(case, g, rows, ids)}
    s["active"] = (torch.arange(rows, device=DEV) % 10 != 9).to(torch.uint8) if rows > 10 else torch.ones(rows, dtype=torch.uint8, device=DEV)
    s["pairs"] = int((s["controls"]["hist_end"] - s["controls"]["hist_begin"]).sum())
    s["x"] = _padded(x.to(FLOATS[case["x"]]), case["pad"])
    if case["op"] == "score":
        y = s["x"].float() + 2e-3 * torch.randn(rows, vocab, generator=g, device=DEV)
        s["y"] = _padded(y.to(FLOATS[case["y"]]), case["pad"])
    if case["op"] == "backward":
        z = _plain_logits(s, s["x"].double()) * s["controls"]["scale"].double()[:, None]
        s["logp"] = _plain_logp(z, ids).float()
        s["grad"] = torch.randn(rows, generator=g, device=DEV)
    return s


# ---- plain forms ---------------------------------------------------------------------------------

def _plain_counts(s, first):
    """[rows, vocab] occurrences of each token in the rows' ranges history[first, hist_end)."""
    c, vocab = s["controls"], s["case"]["vocab"]
    rows = len(s["ids"])
    whole = c["hist_end"] - c["hist_begin"]
    row = torch.repeat_interleave(torch.arange(rows, device=DEV), whole, output_size=s["pairs"])
    at = torch.arange(s["pairs"], device=DEV) - (whole.cumsum(0) - whole)[row] + c["hist_begin"][row]
    counts = torch.zeros(rows * vocab, dtype=torch.int32, device=DEV)
    counts.scatter_add_(0, row * vocab + c["history"][at].long(), (at >= first[row]).to(torch.int32))
    return counts.view(rows, vocab)


def _plain_allowed(s):
    c, vocab = s["controls"], s["case"]["vocab"]
    words = c["mask"][c["mask_row"].long().clamp(min=0)]
    bits = (words[:, :, None] >> torch.arange(32, device=DEV, dtype=torch.int32)) & 1
    return (bits.view(len(words), -1)[:, :vocab] != 0) | (c["mask_row"] < 0)[:, None]


def _plain_logits(s, x):
    """The controlled logits before the scale, in the type of x (the parameters are float32 values)."""
    c, vocab = s["controls"], s["case"]["vocab"]
    rep = c["repetition"][:, None]
    x = torch.where(_plain_counts(s, c["hist_begin"]) > 0, torch.where(x > 0, x / rep, x * rep), x)
    made = _plain_counts(s, c["hist_split"])
    x = torch.where(made > 0, x - c["frequency"][:, None].to(x.dtype) * made - c["presence"][:, None], x)
    if "bias" in c:
        used = (c["bias_ids"] >= 0) & (c["bias_ids"] < vocab)
        dense = torch.zeros(x.shape, dtype=torch.float64, device=DEV)
        dense.scatter_add_(1, c["bias_ids"].long().clamp(0, vocab - 1), torch.where(used, c["bias"], 0.0).double())
        x = x + dense.to(x.dtype)
    if "mask" in c:
        x = torch.where(_plain_allowed(s), x, -math.inf)
    return x


def _plain_logp(z, ids):
    top = z.amax(1, keepdim=True)
    return (z.gather(1, ids.long()[:, None]) - top - (z - top).exp().sum(1, keepdim=True).log())[:, 0]


def _plain_score(s):
    """In float64: the two sides' logprobs nearly agree, and what counts is their difference."""
    scale = s["controls"]["scale"].double()[:, None]
    t = _plain_logp(_plain_logits(s, s["x"].double()) * scale, s["ids"])
    r = _plain_logp(_plain_logits(s, s["y"].double()) * scale, s["ids"])
    act = s["active"] != 0
    t, r = torch.where(act, t, 0.0), torch.where(act, r, 0.0)
    d = t - r
    size = torch.where(act, d.abs(), -1.0)
    n = act.sum()
    order = size.sort().values
    k95, k99 = (len(order) - n + -(-p * n // 100) - 1 for p in (95, 99))
    away = act & ((d < math.log(CLIP[0])) | (d > math.log(CLIP[1])))
    at = torch.where(size == size.amax(), torch.arange(len(d), device=DEV), len(d)).amin()
    values = torch.stack([1 + torch.expm1(d).sum() / n, away.sum() / n, (torch.expm1(d) - d).sum() / n, d.abs().sum() / n,
                          order[k95], order[k99], order[-1]])
    return {"logp_train": t.float(), "logp_rollout": r.float(), "dlogp": d.float(), "n_active": n, "argmax_row": at, "metrics": values.float()}


def _plain_backward(s):
    c, x = s["controls"], s["x"].float()
    z = _plain_logits(s, x) * c["scale"][:, None]
    pick = s["ids"].long()[:, None]
    lse = z.gather(1, pick).double() - s["logp"].double()[:, None]
    hot = torch.zeros_like(z).scatter_(1, pick, 1.0)
    slope = torch.where(x > 0, 1 / c["repetition"][:, None], c["repetition"][:, None])
    slope = torch.where(_plain_counts(s, c["hist_begin"]) > 0, slope, 1.0)
    grad = (s["grad"] * c["scale"])[:, None] * (hot - (z - lse).exp().float()) * slope
    keep = (s["active"] != 0)[:, None] & (z > -math.inf)
    return torch.where(keep, grad, 0.0).to(FLOATS[s["case"]["out"]])


def _plain_quantize(x, fp8, block, transpose, pow2):
    kind, most = FP8[fp8]
    x = (x.t() if transpose else x).float()
    rows, cols = x.shape
    tall = BLOCK if block else 1
    wide = torch.zeros(-(-rows // tall) * tall, -(-cols // BLOCK) * BLOCK, device=x.device)
    wide[:rows, :cols] = x
    tiles = wide.view(-1, tall, wide.shape[1] // BLOCK, BLOCK)
    top = tiles.abs().amax((1, 3), keepdim=True).clamp(min=FLOOR)
    if pow2:
        half, exponent = torch.frexp(top / most)
        scale = torch.ldexp(torch.ones_like(top), torch.where(half == 0.5, exponent - 1, exponent))
        inverse = 1 / scale
    else:
        scale, inverse = top / most, most / top
    q = (tiles * inverse).clamp(-most, most).to(kind)
    return q.view(torch.uint8).reshape(wide.shape)[:rows, :cols].contiguous().view(kind), scale[:, 0, :, 0].contiguous()


def _spread(scales, rows, k):
    """Scales of 1 x 128 or 128 x 128 blocks at every value."""
    tall = scales if len(scales) == rows else scales.repeat_interleave(BLOCK, 0)[:rows]
    return tall.repeat_interleave(BLOCK, 1)[:, :k]


def _plain_matmul(s):
    a = s["a"].float() * _spread(s["a_scales"], *s["a"].shape)
    b = s["b"].float() * _spread(s["b_scales"], *s["b"].shape)
    return (a @ b.t()).to(FLOATS[s["case"]["out"]])


# ---- the library's calls -------------------------------------------------------------------------

def _kept(s, name, make):
    """A buffer that a user's program keeps between calls."""
    if name not in s:
        s[name] = make()
    return s[name]


def _own(s):
    from logprob_drift_scoring_gb300 import binding as B

    case = s["case"]
    if case["op"] == "quantize":
        rows, cols = (case["cols"], case["rows"]) if case["transpose"] else (case["rows"], case["cols"])
        out = _kept(s, "out", lambda: B.block_empty(rows, cols, FP8[case["fp8"]][0], case["block"], device=DEV))
        B.lpd_block_quantize(s["x"], out, transpose=case["transpose"], pow2=case["pow2"])
        return {"values": out.values, "scales": out.scales}
    if case["op"] == "matmul":
        a = B.BlockScaled(s["a"], s["a_scales"], case["a_block"])
        b = B.BlockScaled(s["b"], s["b_scales"], case["b_block"])
        out = _kept(s, "out", lambda: torch.empty(case["m"], case["n"], dtype=FLOATS[case["out"]], device=DEV))
        room = _kept(s, "room", lambda: torch.empty(B.lpd_block_workspace_size(case["m"], case["n"], case["k"]), dtype=torch.uint8, device=DEV))
        B.lpd_block_matmul(a, b, out, room)
        return out
    c = _kept(s, "handle", lambda: B.Controls(**s["controls"]))
    rows, vocab = s["x"].shape
    if case["op"] == "score":
        outs = _kept(s, "outs", lambda: [torch.empty(rows, device=DEV) for _ in range(3)])
        met = _kept(s, "met", lambda: torch.empty(B.METRICS_BYTES, dtype=torch.uint8, device=DEV))
        room = _kept(s, "room", lambda: torch.empty(B.lpd_workspace_size(B.LPD_KIND_CONTROLLED, rows, vocab), dtype=torch.uint8, device=DEV))
        B.lpd_score_controlled(s["x"], s["y"], c, c, s["ids"], s["active"], *CLIP, *outs, met, room)
        return {"logp_train": outs[0], "logp_rollout": outs[1], "dlogp": outs[2], "n_active": met.view(torch.int64)[0],
                "argmax_row": met.view(torch.int64)[1], "metrics": met.view(torch.float64)[3:].float()}
    out = _kept(s, "out", lambda: torch.empty(rows, vocab, dtype=FLOATS[case["out"]], device=DEV))
    if case["op"] == "apply":
        B.lpd_controls_apply(s["x"], c, out)
    else:
        B.lpd_logprob_backward_controlled(s["x"], c, s["ids"], s["active"], s["logp"], s["grad"], out)
    return out


def run(s):
    if own:
        return _own(s)
    op = s["case"]["op"]
    if op == "quantize":
        q, scales = _plain_quantize(s["x"], *(s["case"][k] for k in ("fp8", "block", "transpose", "pow2")))
        return {"values": q, "scales": scales}
    if op == "matmul":
        return _plain_matmul(s)
    if op == "score":
        return _plain_score(s)
    if op == "backward":
        return _plain_backward(s)
    return (_plain_logits(s, s["x"].float()) * s["controls"]["scale"][:, None]).to(FLOATS[s["case"]["out"]])


# ---- the definitions in float64 ------------------------------------------------------------------

def _exact_row(s, x, r):
    """Row r under its controls, and the slope of each of its controlled logits."""
    c, vocab = s["controls"], s["case"]["vocab"]
    z = x[r].double()
    begin, split, end = (int(c[k][r]) for k in ("hist_begin", "hist_split", "hist_end"))
    rep, freq, pres, scale = (float(c[k][r]) for k in ("repetition", "frequency", "presence", "scale"))
    slope = torch.full((vocab,), scale, dtype=torch.float64, device=DEV)
    seen = torch.unique(c["history"][begin:end].long())
    factor = torch.where(z[seen] > 0, 1 / rep, rep)
    z[seen] *= factor
    slope[seen] *= factor
    made, times = torch.unique(c["history"][split:end].long(), return_counts=True)
    z[made] -= freq * times + pres
    if "bias" in c:
        ids = c["bias_ids"][r].long()
        z.index_add_(0, ids[ids >= 0], c["bias"][r][ids >= 0].double())
    if "mask" in c and int(c["mask_row"][r]) >= 0:
        word = c["mask"][int(c["mask_row"][r])].long()
        j = torch.arange(vocab, device=DEV)
        off = (word[j // 32] >> (j % 32)) % 2 == 0
        z[off], slope[off] = -math.inf, 0.0
    return z * scale, slope


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "quantize":
        kind, most = FP8[case["fp8"]]
        x = s["x"].t() if case["transpose"] else s["x"]
        tall = BLOCK if case["block"] else 1
        cut = torch.nn.functional.pad(x.double(), (0, -x.shape[1] % BLOCK, 0, -x.shape[0] % tall))
        top = torch.nn.functional.max_pool2d(cut.abs()[None], (tall, BLOCK))[0].clamp_(min=FLOOR)
        scale = torch.exp2(torch.ceil(torch.log2(top / most))) if case["pow2"] else top / most
        q = cut / scale.repeat_interleave(tall, 0).repeat_interleave(BLOCK, 1)
        return {"values": q[:x.shape[0], :x.shape[1]].clamp(-most, most).to(kind), "scales": scale}
    if case["op"] == "matmul":
        sides = []
        for side in ("a", "b"):
            v, scales = s[side].double(), s[side + "_scales"].double()
            at = torch.arange(v.shape[0], device=DEV) // (BLOCK if case[side + "_block"] else 1)
            sides.append(v * scales[at][:, torch.arange(v.shape[1], device=DEV) // BLOCK])
        return torch.mm(sides[0], sides[1].t())
    rows = len(s["ids"])
    if case["op"] == "apply":
        return torch.stack([_exact_row(s, s["x"], r)[0] for r in range(rows)])
    if case["op"] == "score":
        logp = torch.zeros(2, rows, dtype=torch.float64, device=DEV)
        for r in range(rows):
            if r % 10 != 9 or rows <= 10:
                for side, x in enumerate((s["x"], s["y"])):
                    z = _exact_row(s, x, r)[0]
                    logp[side, r] = z[int(s["ids"][r])] - torch.logsumexp(z, 0)
        d = logp[0] - logp[1]
        live = d[s["active"] != 0]
        size = live.abs().sort().values
        rank = [size[-(-p * len(size) // 100) - 1] for p in (95, 99, 100)]
        ratio = live.exp()
        return {"logp_train": logp[0], "logp_rollout": logp[1], "dlogp": d, "n_active": None, "argmax_row": None,
                "metrics": torch.stack([ratio.mean(), ((ratio < CLIP[0]) | (ratio > CLIP[1])).double().mean(),
                                        (torch.expm1(live) - live).mean(), size.mean(), *rank])}
    grad = torch.zeros(rows, case["vocab"], dtype=torch.float64, device=DEV)
    for r in range(rows):
        if r % 10 != 9 or rows <= 10:
            z, slope = _exact_row(s, s["x"], r)
            at = int(s["ids"][r])
            p = torch.exp(z - z[at] + s["logp"][r].double())
            grad[r] = -p
            grad[r, at] += 1
            grad[r] *= slope * s["grad"][r].double()
    return grad
