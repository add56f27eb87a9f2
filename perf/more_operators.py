"""Cases of token sampling (temperature, min-p, top-k, top-p from given random numbers), of the kept set of such a
filter as masks for the scorer, and of microscaled 4-bit floating point (quantisation and product): their inputs,
the calls that a user makes, and the same computations in elementary torch operations.

A case is one call with its sizes.  ``run`` computes it in the plain form, or with ``own`` through the
library's entry points; ``exact`` gives the result of the definition in float64.
"""
import math

import torch

own = False

DEV = "cuda"
FLOATS = {"bf16": torch.bfloat16, "f32": torch.float32}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)  # the magnitudes of a 4-bit value
FLOOR = 2.0 ** -64                               # smallest magnitude that a power-of-two scale is made for


# ---- cases ---------------------------------------------------------------------------------------

def listed():
    return [
        # the next token of a single request: latency
        {"name": "sample-one-row", "op": "sample", "rows": 1, "vocab": 128256, "pad": 0, "x": "f32", "peak": 16.0, "params": "top"},
        # a serving batch whose requests ask for all kinds of filters, greedy ones among them
        {"name": "sample-batch", "op": "sample", "rows": 256, "vocab": 151936, "pad": 0, "x": "bf16", "peak": 16.0, "params": "mixed"},
        # a rollout's step: plain temperature and nucleus only, an odd number of rows
        {"name": "sample-nucleus", "op": "sample", "rows": 509, "vocab": 151936, "pad": 0, "x": "bf16", "peak": 16.0, "params": "nucleus"},
        # the kept sets of an odd vocabulary whose rows lie on no 16-byte boundary
        {"name": "filter-odd", "op": "filter", "rows": 633, "vocab": 50021, "pad": 1, "x": "f32", "peak": 12.0, "params": "mixed"},
        # the kept sets of a teacher-forced batch, for the scorer's masks
        {"name": "filter-long", "op": "filter", "rows": 4096, "vocab": 151936, "pad": 0, "x": "bf16", "peak": 16.0, "params": "top"},
        # the hidden rows in front of a 4-bit head, with the values that training sees
        {"name": "quantize-hidden", "op": "quantize", "rows": 1024, "cols": 4096, "x": "bf16", "block": 16, "transpose": False},
        # a head's odd shard in float32
        {"name": "quantize-odd", "op": "quantize", "rows": 12661, "cols": 2051, "x": "f32", "block": 32, "transpose": False},
        # the head's weight laid out for the data gradient
        {"name": "quantize-weight", "op": "quantize", "rows": 151936, "cols": 4096, "x": "bf16", "block": 16, "transpose": True},
        # the head over a decode batch
        {"name": "matmul-decode", "op": "matmul", "m": 16, "n": 151936, "k": 4096, "block": 16, "out": "bf16"},
        # the head over the rows of a scoring batch
        {"name": "matmul-head", "op": "matmul", "m": 4096, "n": 128256, "k": 4096, "block": 16, "out": "bf16"},
        # the data gradient of a small batch: a long k axis and few outputs
        {"name": "matmul-dgrad", "op": "matmul", "m": 512, "n": 4096, "k": 151936, "block": 32, "out": "bf16"},
        # the weight gradient of one vocabulary shard over an odd number of tokens
        {"name": "matmul-wgrad", "op": "matmul", "m": 37984, "n": 4096, "k": 2051, "block": 32, "out": "f32"},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["sample", "sample", "sample", "filter", "filter", "quantize", "quantize", "matmul", "matmul", "matmul"])
    if op == "quantize":
        rows = _log(rng, 1, 151936)
        return {"op": op, "rows": rows, "cols": _log(rng, 1, min(16384, 151936 * 4096 // rows)), "x": rng.choice(["bf16", "f32"]) if rows < 60000 else "bf16",
                "block": rng.choice([16, 32]), "transpose": rng.random() < 0.5}
    if op == "matmul":
        kind = rng.choice(["head", "data", "weight"])  # the product's three uses
        tokens = _log(rng, 1, 4096)
        vocab, hidden = _log(rng, 1000, 128256), _log(rng, 64, 4096)
        m, n, k = {"head": (tokens, vocab, hidden), "data": (tokens, hidden, vocab), "weight": (vocab, hidden, tokens)}[kind]
        return {"op": op, "m": m, "n": n, "k": k, "block": rng.choice([16, 32]), "out": "f32" if kind == "weight" else rng.choice(["bf16", "f32"])}
    x = rng.choice(["bf16", "bf16", "f32"])
    rows = _log(rng, 1, 512 if op == "sample" else 4096 if x == "bf16" else 2048)
    return {"op": op, "rows": rows, "vocab": rng.choice([1024, 37984, 128256, 151936, _log(rng, 1000, 151936), _log(rng, 1000, 151936)]),
            "pad": rng.choice([0, 0, 1, 8, 24]), "x": x, "peak": rng.choice([0.0, 8.0, 16.0, 16.0, 24.0]), "params": rng.choice(["mixed", "mixed", "top", "nucleus"])}


# ---- what a call has to read, write and compute --------------------------------------------------

def _bytes(name):
    return {"bf16": 2, "f32": 4}[name]


def _scale_bytes(rows, k, block):
    return -(-rows // 128) * 128 * (-(-k // (4 * block)) * 4)


def work(case):
    if case["op"] == "quantize":
        r, c = case["rows"], case["cols"]
        rows, k = (c, r) if case["transpose"] else (r, c)
        return {"bytes": r * c * _bytes(case["x"]) + rows * -(-k // 2) + _scale_bytes(rows, k, case["block"]) + r * c * _bytes(case["x"])}
    if case["op"] == "matmul":
        m, n, k = case["m"], case["n"], case["k"]
        scales = _scale_bytes(m, k, case["block"]) + _scale_bytes(n, k, case["block"])
        return {"bytes": (m + n) * -(-k // 2) + scales + m * n * _bytes(case["out"]), "flops": 2 * m * n * k}
    rows, vocab = case["rows"], case["vocab"]
    if case["op"] == "sample":
        return {"bytes": rows * (vocab * _bytes(case["x"]) + 20 + 12), "flops": 4 * rows * vocab}
    active = rows - rows // 10
    return {"bytes": active * vocab * _bytes(case["x"]) + rows * (4 * -(-vocab // 32) + 21 + 8), "flops": 4 * active * vocab}


# ---- inputs --------------------------------------------------------------------------------------

def _padded(x, pad):
    if not pad:
        return x
    wide = torch.full((x.shape[0], x.shape[1] + pad), float("nan"), dtype=x.dtype, device=DEV)
    wide[:, :x.shape[1]] = x
    return wide[:, :x.shape[1]]


def _params(kind, rows, g):
    """The requests' parameters: a row's kind of request is drawn, or one of two for the narrower sets."""
    def uniform(lo, hi):
        return lo + (hi - lo) * torch.rand(rows, generator=g, device=DEV)

    pick = torch.randint(0, 6, (rows,), generator=g, device=DEV)
    scale, k = uniform(0.75, 1.7), torch.randint(10, 200, (rows,), generator=g, device=DEV, dtype=torch.int32)
    p, m = uniform(0.75, 0.99), uniform(0.01, 0.2)
    off_k, off = torch.zeros_like(k), torch.zeros_like(m)
    if kind == "top":       # top-k and top-p together, the usual pair
        return {"scale": scale, "min_p": off, "top_k": k, "top_p": p}
    if kind == "nucleus":   # plain temperature, or a nucleus
        return {"scale": scale, "min_p": off, "top_k": off_k, "top_p": torch.where(pick < 2, 1.0, p)}
    # 0: greedy, 1: top-k, 2: top-p, 3: min-p, 4: temperature alone, 5: everything at once
    k = torch.where(pick == 0, 1, torch.where((pick == 1) | (pick == 5), k, 0)).to(torch.int32)
    return {"scale": scale, "min_p": torch.where((pick == 3) | (pick == 5), m, 0.0), "top_k": k,
            "top_p": torch.where((pick == 2) | (pick == 5), p, 1.0)}


def _e2m1_index(a):
    """The nearest of E2M1 to the magnitudes a, ties to the even one."""
    i = (a > 0.25).to(torch.uint8)
    for edge, closed in ((0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5.0, False)):
        i += (a >= edge) if closed else (a > edge)
    return i


def _tiled_scales(scales):
    """[rows, blocks] scale bytes as the operand holds them: 512 bytes for 128 rows x 4 blocks, the rows that share
    row % 32 together, the rest of the last ones 0."""
    rows, blocks = scales.shape
    full = torch.zeros(-(-rows // 128) * 128, -(-blocks // 4) * 4, dtype=torch.uint8, device=scales.device)
    full[:rows, :blocks] = scales
    return full.view(-1, 4, 32, full.shape[1] // 4, 4).permute(0, 3, 2, 1, 4).reshape(-1)


def _row_scales(tiled, rows, blocks):
    wide = -(-blocks // 4)
    return tiled.view(-1, wide, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(-1, wide * 4)[:rows, :blocks]


def _scale_values(scales, block):
    return scales.view(torch.float8_e4m3fn).float() if block == 16 else torch.ldexp(torch.ones(scales.shape, device=scales.device), scales.int() - 127)


def _plain_quantize(x, block, transpose, tensor_scale):
    x = (x.t() if transpose else x).float()
    rows, k = x.shape
    wide = torch.zeros(rows, -(-k // block) * block, device=x.device)
    wide[:, :k] = x
    tiles = wide.view(rows, -1, block)
    top = tiles.abs().amax(2)
    if block == 16:
        scales = (top / (6.0 * tensor_scale)).clamp(max=448.0).to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        half, exponent = torch.frexp(top.clamp(min=FLOOR) / 6.0)
        scales = (torch.where(half == 0.5, exponent - 1, exponent) + 127).to(torch.uint8)
    size = _scale_values(scales, block)
    step = size * tensor_scale
    inverse = torch.where(step == 0, 0.0, 1 / step)
    near = tiles * inverse[:, :, None]
    index = _e2m1_index(near.abs())
    codes = (index + 8 * (near.view(torch.int32) < 0).to(torch.uint8)).view(rows, -1)
    values = torch.tensor(E2M1, device=x.device)[index.int()].copysign_(near).mul_(size[:, :, None]).mul_(tensor_scale).view(rows, -1)[:, :k]
    packed = torch.zeros(rows, -(-k // 32) * 32, dtype=torch.uint8, device=x.device)
    packed[:, :k] = codes[:, :k]
    packed = packed[:, 0::2] + 16 * packed[:, 1::2]
    return packed, _tiled_scales(scales), values


def _tensor_scale(x, block, g):
    """The operand's own scale (blocks of 16): from a calibration, so that it lies a little above what x needs."""
    if block == 32:
        return torch.ones(1, device=DEV)
    return x.abs().amax().float().reshape(1) * (1 + 0.25 * torch.rand(1, generator=g, device=DEV)) / (448.0 * 6.0)


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    if case["op"] == "quantize":
        x = torch.randn(case["rows"], case["cols"], generator=g, device=DEV, dtype=FLOATS[case["x"]])
        x *= torch.rand(case["rows"], 1, generator=g, device=DEV).add_(0.2).to(x.dtype)
        return {"case": case, "x": x, "tensor_scale": _tensor_scale(x, case["block"], g)}
    if case["op"] == "matmul":
        s = {"case": case}
        for side, rows in (("a", case["m"]), ("b", case["n"])):
            x = torch.randn(rows, case["k"], generator=g, device=DEV, dtype=torch.bfloat16)
            s[side + "_tensor_scale"] = _tensor_scale(x, case["block"], g)
            s[side], s[side + "_scales"] = _plain_quantize(x, case["block"], False, s[side + "_tensor_scale"])[:2]
        return s
    rows, vocab = case["rows"], case["vocab"]
    # many unlikely tokens, and some that stand out by up to `peak`, as behind a trained head (0: an untrained one)
    x = torch.randn(rows, vocab, generator=g, device=DEV, dtype=torch.float32).mul_(1.5)
    head = torch.randint(0, vocab, (rows, 64), generator=g, device=DEV)
    x.scatter_add_(1, head, case["peak"] * torch.rand(rows, 64, generator=g, device=DEV))
    s = {"case": case, "x": _padded(x.to(FLOATS[case["x"]]), case["pad"]), "filter": _params(case["params"], rows, g)}
    if case["op"] == "sample":
        s["uniform"] = torch.rand(rows, generator=g, device=DEV)
    else:
        s["ids"] = head[:, 0].to(torch.int32)
        s["active"] = (torch.arange(rows, device=DEV) % 10 != 9).to(torch.uint8)
    return s


# ---- plain forms ---------------------------------------------------------------------------------

def _plain_kept(s):
    """Which tokens the rows' filters keep, and the tokens' scaled logits in float64 (the cumulated masses stand
    next to their borders)."""
    f, x = s["filter"], s["x"]
    z = x.double() * f["scale"].double()[:, None]
    top = z.amax(1, keepdim=True)
    away = z - top
    first = (away >= f["min_p"].double().log()[:, None]) & (z > -math.inf)  # (log 0: -inf, nothing is left out)
    order = x.float().sort(dim=1, descending=True, stable=True).indices
    ok = first.gather(1, order)
    k = torch.where(f["top_k"] > 0, f["top_k"], x.shape[1])
    ok &= torch.arange(x.shape[1], device=DEV)[None] < k[:, None]
    mass = torch.where(ok, away.gather(1, order).exp_(), 0.0)
    before = mass.cumsum(1) - mass
    whole = mass.sum(1, keepdim=True)
    ok &= (before < f["top_p"].double()[:, None] * whole) | (f["top_p"] >= 1)[:, None]
    return torch.zeros_like(ok).scatter_(1, order, ok), away, top[:, 0]


def _plain_sample(s):
    kept, away, _ = _plain_kept(s)
    mass = torch.where(kept, away.exp(), 0.0)
    up_to = mass.cumsum(1)
    ids = (up_to <= s["uniform"].double()[:, None] * up_to[:, -1:]).sum(1)
    last = torch.where(kept, torch.arange(kept.shape[1], device=DEV), -1).amax(1)
    ids = torch.minimum(ids, last)
    logp = away.gather(1, ids[:, None])[:, 0] - mass.sum(1).log()
    return {"ids": ids.to(torch.int32), "logp": logp.float(), "kept": kept.sum(1).to(torch.int32)}


def _plain_filter(s):
    kept, away, top = _plain_kept(s)
    kept.scatter_(1, s["ids"].long()[:, None], True)
    act = s["active"] != 0
    lse = torch.where(act, top + torch.where(kept, away.exp(), 0.0).sum(1).log(), 0.0)
    kept &= act[:, None]
    words = -(-kept.shape[1] // 32)
    bits = torch.zeros(kept.shape[0], words * 32, dtype=torch.int32, device=DEV)
    bits[:, :kept.shape[1]] = kept
    mask = (bits.view(-1, words, 32) << torch.arange(32, device=DEV, dtype=torch.int32)).sum(2, dtype=torch.int32)
    return {"mask": mask, "lse": lse.float(), "kept": kept.sum(1).to(torch.int32)}


def _unpacked(packed, k):
    codes = torch.stack([packed & 15, packed >> 4], 2).view(packed.shape[0], -1)[:, :k]
    return torch.tensor(E2M1 + tuple(-v for v in E2M1), device=packed.device)[codes.int()]


def _plain_operand(s, side, rows):
    k, block = s["case"]["k"], s["case"]["block"]
    size = _scale_values(_row_scales(s[side + "_scales"], rows, -(-k // block)), block)
    return _unpacked(s[side], k) * size.repeat_interleave(block, 1)[:, :k]


def _plain_matmul(s):
    c = s["case"]
    out = _plain_operand(s, "a", c["m"]) @ _plain_operand(s, "b", c["n"]).t()
    return (out * (s["a_tensor_scale"] * s["b_tensor_scale"])).to(FLOATS[c["out"]])


# ---- the library's calls -------------------------------------------------------------------------

def _kept(s, name, make):
    """A buffer that a user's program keeps between calls."""
    if name not in s:
        s[name] = make()
    return s[name]


def _scales_out(scales, block):
    """Scale bytes as what they stand for: 8-bit floats, or whole exponents of two."""
    return scales.view(torch.float8_e4m3fn) if block == 16 else scales


def _own(s):
    from logprob_drift_scoring_gb300 import binding as B

    case = s["case"]
    if case["op"] == "quantize":
        rows, k = (case["cols"], case["rows"]) if case["transpose"] else (case["rows"], case["cols"])
        out = _kept(s, "out", lambda: B.micro_empty(rows, k, case["block"], tensor_scale=s["tensor_scale"], device=DEV))
        values = _kept(s, "values", lambda: torch.empty(rows, k, dtype=s["x"].dtype, device=DEV))
        B.lpd_micro_quantize(s["x"], out, transpose=case["transpose"], out_values=values)
        return {"codes": out.codes, "scales": _scales_out(out.scales, case["block"]), "values": values}
    if case["op"] == "matmul":
        m, n, k = case["m"], case["n"], case["k"]
        a = B.MicroScaled(s["a"], s["a_scales"], k, case["block"], s["a_tensor_scale"])
        b = B.MicroScaled(s["b"], s["b_scales"], k, case["block"], s["b_tensor_scale"])
        out = _kept(s, "out", lambda: torch.empty(m, n, dtype=FLOATS[case["out"]], device=DEV))
        room = _kept(s, "room", lambda: torch.empty(B.lpd_micro_workspace_size(m, n, k), dtype=torch.uint8, device=DEV))
        B.lpd_micro_matmul(a, b, out, room)
        return out
    rows, vocab = s["x"].shape
    f = _kept(s, "handle", lambda: B.Filter(**s["filter"]))
    kept = _kept(s, "kept", lambda: torch.empty(rows, dtype=torch.int32, device=DEV))
    if case["op"] == "sample":
        ids = _kept(s, "out_ids", lambda: torch.empty(rows, dtype=torch.int32, device=DEV))
        logp = _kept(s, "out_logp", lambda: torch.empty(rows, device=DEV))
        B.lpd_sample(s["x"], f, s["uniform"], ids, logp, kept)
        return {"ids": ids, "logp": logp, "kept": kept}
    mask = _kept(s, "out_mask", lambda: torch.empty(rows, -(-vocab // 32), dtype=torch.int32, device=DEV))
    lse = _kept(s, "out_lse", lambda: torch.empty(rows, device=DEV))
    B.lpd_filter_mask(s["x"], f, s["ids"], s["active"], mask, lse, kept)
    return {"mask": mask, "lse": lse, "kept": kept}


def run(s):
    if own:
        return _own(s)
    case = s["case"]
    if case["op"] == "quantize":
        packed, scales, values = _plain_quantize(s["x"], case["block"], case["transpose"], s["tensor_scale"])
        return {"codes": packed[:, :-(-values.shape[1] // 2)], "scales": _scales_out(scales, case["block"]), "values": values.to(s["x"].dtype)}
    if case["op"] == "matmul":
        return _plain_matmul(s)
    return _plain_sample(s) if case["op"] == "sample" else _plain_filter(s)


# ---- the definitions in float64 ------------------------------------------------------------------

def _exact_row(s, r):
    """Row r's scaled logits, and the tokens that its filter keeps, in descending order."""
    f = {name: float(t[r]) for name, t in s["filter"].items()}
    z = s["x"][r].double() * f["scale"]
    tokens = torch.argsort(z, descending=True, stable=True)
    if f["min_p"] > 0:
        tokens = tokens[z[tokens] - z[tokens[0]] >= math.log(f["min_p"])]
    if f["top_k"] > 0:
        tokens = tokens[:int(f["top_k"])]
    if f["top_p"] < 1:
        share = torch.softmax(z[tokens], 0).cumsum(0)
        tokens = tokens[:int((share < f["top_p"]).sum()) + 1]
    return z, tokens


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "quantize":
        x, block = s["x"].t() if case["transpose"] else s["x"], case["block"]
        cut = torch.nn.functional.pad(x.double(), (0, -x.shape[1] % block)).view(x.shape[0], -1, block)
        top, ts = cut.abs().amax(2, keepdim=True), float(s["tensor_scale"])
        if block == 16:  # the operator's scale is an 8-bit float of the float32 quotient
            size = (top.float() / (6.0 * s["tensor_scale"])).clamp(max=448.0).to(torch.float8_e4m3fn).double()
        else:
            size = torch.exp2(torch.ceil(torch.log2(top.clamp(min=FLOOR) / 6.0)))
        grid = torch.tensor(E2M1, dtype=torch.float64, device=DEV)
        at = cut.abs() / torch.where(size > 0, size * ts, math.inf)
        low = (torch.searchsorted(grid, at.contiguous(), right=True) - 1).clamp_(max=6)
        below, above = grid[low], grid[low + 1]
        up = (at - below > above - at) | ((at - below == above - at) & (low % 2 == 1))
        values = torch.where(up, above, below) * cut.sign() * size * ts
        return {"codes": None, "scales": None, "values": values.view(x.shape[0], -1)[:, :x.shape[1]]}
    if case["op"] == "matmul":
        sides = []
        for side, rows in (("a", case["m"]), ("b", case["n"])):
            codes = s[side][:, torch.arange(case["k"], device=DEV) // 2]
            codes = torch.where(torch.arange(case["k"], device=DEV) % 2 == 1, codes >> 4, codes & 15)
            v = torch.tensor(E2M1, dtype=torch.float64, device=DEV)[(codes & 7).long()] * torch.where(codes > 7, -1.0, 1.0)
            r, b = torch.arange(rows, device=DEV)[:, None], torch.arange(case["k"], device=DEV)[None] // case["block"]
            at = ((r // 128) * -(-case["k"] // (4 * case["block"])) + b // 4) * 512 + r % 32 * 16 + r // 32 % 4 * 4 + b % 4
            byte = s[side + "_scales"][at]
            v *= byte.view(torch.float8_e4m3fn).double() if case["block"] == 16 else torch.exp2(byte.double() - 127)
            sides.append(v * s[side + "_tensor_scale"].double())
            del at, byte, codes
        return torch.mm(sides[0], sides[1].t())
    rows = case["rows"]
    out = torch.zeros(rows, dtype=torch.float64, device=DEV)
    for r in range(rows):
        if case["op"] == "filter" and r % 10 == 9:
            continue
        z, tokens = _exact_row(s, r)
        if case["op"] == "filter":
            out[r] = torch.logsumexp(z[torch.unique(torch.cat([tokens, s["ids"][r:r + 1].long()]))], 0)
            continue
        tokens = tokens.sort().values
        logp = torch.log_softmax(z[tokens], 0)
        share = logp.exp().cumsum(0)
        at = torch.searchsorted(share, s["uniform"][r].double() * share[-1], right=True)
        out[r] = logp[at.clamp(max=len(tokens) - 1)]
    return {"ids": None, "logp": out, "kept": None} if case["op"] == "sample" else {"mask": None, "lse": out, "kept": None}
