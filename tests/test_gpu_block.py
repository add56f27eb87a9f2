"""Block-scaled 8-bit operands and their product on the GPU (needs a GPU).

Bounds.  Quantisation: the scales and values are those of the definition in
float32, bit for bit, and a value is within half a step of x (2^-4 relative for
e4m3, 2^-3 for e5m2; half of the smallest subnormal below that).  Product: a
block's 128 products are exact in float32 and are added on the tensor cores in
fixed point relative to the largest, with some 22 bits kept in each of the four
steps of 32: 2^-20 of the sum of magnitudes; each block then costs two roundings
of at most 2^-24 of the running magnitude; bf16 adds its half step, 2^-8.
"""
import numpy as np
import pytest
import torch

from logprob_drift_scoring_gb300 import binding as B
from tests import controls_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
KINDS = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
FP8 = {"e4m3": (torch.float8_e4m3fn, 448.0, 2.0 ** -4, 2.0 ** -10), "e5m2": (torch.float8_e5m2, 57344.0, 2.0 ** -3, 2.0 ** -17)}


def spread(scales, rows, k, block):
    s = scales.double().cpu()
    if block:
        s = s.repeat_interleave(128, 0)[:rows]
    return s.repeat_interleave(128, 1)[:, :k]


def meaning(op):
    """The float64 values that an operand stands for."""
    v = op.values.float().cpu().double()
    return v * spread(op.scales, *v.shape, op.block)


def definition(x, fp8, block, transpose, pow2):
    """(values, scales) of lpd_block_quantize in float32 on the CPU, block by block."""
    kind, most, _, _ = FP8[fp8]
    x = (x.t() if transpose else x).float().cpu()
    rows, k = x.shape
    tall = 128 if block else 1
    scales = torch.empty(-(-rows // tall), -(-k // 128))
    values = torch.empty(rows, k)
    for i in range(scales.shape[0]):
        for j in range(scales.shape[1]):
            part = (slice(i * tall, (i + 1) * tall), slice(j * 128, (j + 1) * 128))
            top = x[part].abs().max().clamp(min=2.0 ** -64)
            s = top / most
            if pow2:
                s = torch.tensor(2.0 ** int(np.ceil(np.log2(float(s)))), dtype=torch.float32)
                inv = 1 / s
            else:
                inv = torch.tensor(most) / top  # one rounding (a Python number over a tensor takes two)
            scales[i, j] = s
            values[part] = x[part] * inv
    return values.clamp(-most, most).to(kind), scales


def make(rng, rows, cols, kind, pad=0):
    x = rng.normal(0, 1, (rows, cols)) * np.exp(rng.normal(0, 2, (rows, 1)))
    t = torch.from_numpy(x.astype(np.float32)).to(KINDS[kind]).to(DEV)
    if pad:
        wide = torch.full((rows, cols + pad), float("nan"), dtype=t.dtype, device=DEV)
        wide[:, :cols] = t
        t = wide[:, :cols]
    return t


@pytest.mark.parametrize("rows,cols,pad", [(1, 1, 0), (1, 128, 0), (3, 130, 6), (128, 128, 0), (129, 257, 0), (200, 1000, 8),
                                           (37, 640, 3), (300, 72, 0)])
@pytest.mark.parametrize("block", [False, True])
@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("kind,fp8,pow2", [("bf16", "e4m3", False), ("bf16", "e5m2", True), ("f32", "e4m3", True), ("f32", "e5m2", False)])
def test_quantize(rows, cols, pad, block, transpose, kind, fp8, pow2):
    rng = np.random.default_rng(rows + cols)
    x = make(rng, rows, cols, kind, pad)
    out = B.block_quantize(x, FP8[fp8][0], block, transpose, pow2)
    values, scales = definition(x, fp8, block, transpose, pow2)
    assert torch.equal(out.scales.cpu(), scales)
    assert torch.equal(out.values.cpu().view(torch.uint8), values.view(torch.uint8))
    want = (x.t() if transpose else x).double().cpu()
    _, _, step, least = FP8[fp8]
    err = (meaning(out) - want).abs()
    tol = (step + 2.0 ** -22) * want.abs() + least * spread(out.scales, *want.shape, block)
    assert bool((err <= tol).all())


def test_quantize_zeros_tiny_and_non_finite():
    x = torch.zeros(4, 640, device=DEV)
    x[0, 200] = 2.0 ** -100
    x[1, 130] = float("inf")
    x[2, 300] = float("nan")
    x[3, 400] = -float("inf")
    x[1:, 500] = 3.0e38
    for transpose in (False, True):
        q = B.block_quantize(x if not transpose else x.t().contiguous(), transpose=transpose)
        v = meaning(q)
        assert bool((v[0] == 0).all()) and bool((q.scales[0] > 0).all())
        for r, j in ((1, 1), (2, 2), (3, 3)):
            assert bool(torch.isnan(v[r, 128 * j:128 * j + 128]).all())
            rest = torch.cat([v[r, :128 * j], v[r, 128 * j + 128:]])
            assert bool(torch.isfinite(rest).all())
        assert abs(float(v[1, 500]) - 3.0e38) <= 3.0e38 * 2.0 ** -22
    blk = B.block_quantize(x, block=True)
    assert bool(torch.isnan(meaning(blk)[:, 128:512]).all()) and bool(torch.isfinite(meaning(blk)[:, :128]).all())


def test_quantize_leaves_the_padding():
    x = make(np.random.default_rng(1), 70, 150, "bf16")
    for transpose in (False, True):
        rows, k = (150, 70) if transpose else (70, 150)
        room = torch.full((rows + 1, 208), 77, dtype=torch.uint8, device=DEV)
        wide = torch.full((rows + 1, 5), -3.0, device=DEV)
        out = B.BlockScaled(room.view(torch.float8_e4m3fn)[:rows, :k], wide[:rows, :-(-k // 128)])
        B.lpd_block_quantize(x, out, transpose)
        assert bool((room[:, k:] == 77).all()) and bool((room[rows] == 77).all())
        assert bool((wide[:, -(-k // 128):] == -3).all()) and bool((wide[rows] == -3).all())
        assert torch.equal(out.values.view(torch.uint8), B.block_quantize(x, transpose=transpose).values.view(torch.uint8))


def operand(rng, rows, k, fp8, block, pad=0):
    """Random 8-bit values and scales; the bytes behind each row are NaN patterns."""
    kind, most, _, _ = FP8[fp8]
    v = torch.from_numpy((rng.normal(0, 0.3, (rows, k)) * most / 4).astype(np.float32)).clamp(-most, most).to(kind)
    wide = torch.full((rows, -(-k // 16) * 16 + pad), 0x7F, dtype=torch.uint8)
    wide[:, :k] = v.view(torch.uint8)
    shape = (-(-rows // 128) if block else rows, -(-k // 128))
    scales = torch.from_numpy(np.exp(rng.normal(0, 1, shape)).astype(np.float32) / most)
    return B.BlockScaled(wide.to(DEV).view(kind)[:, :k], scales.to(DEV), block)


def check_product(a, b, out, kind):
    x, y = meaning(a), meaning(b)
    want, size = x @ y.t(), x.abs() @ y.abs().t()
    kb = -(-x.shape[1] // 128)
    err = (out.double().cpu() - want).abs()
    tol = (2.0 ** -20 + kb * 2.0 ** -23) * size + HALF[kind] * want.abs()
    assert bool((err <= tol).all()), float((err / (tol + 1e-300)).max())


SIZES = [(1, 1, 1), (1, 128, 128), (5, 300, 129), (127, 256, 16), (128, 257, 520), (129, 513, 1000), (300, 1000, 1031),
         (16, 5000, 256), (2, 256, 4096), (40, 300, 9000), (257, 40, 2100)]


@pytest.mark.parametrize("m,n,k", SIZES)
@pytest.mark.parametrize("a_block,b_block", [(False, True), (False, False), (True, True), (True, False)])
@pytest.mark.parametrize("a8,b8,kind", [("e4m3", "e4m3", "bf16"), ("e5m2", "e4m3", "f32")])
def test_product(m, n, k, a_block, b_block, a8, b8, kind):
    rng = np.random.default_rng(m + n + k)
    a, b = operand(rng, m, k, a8, a_block, 16), operand(rng, n, k, b8, b_block)
    check_product(a, b, B.block_matmul(a, b, KINDS[kind]), kind)


@pytest.mark.parametrize("a8,b8", [("e4m3", "e5m2"), ("e5m2", "e5m2")])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_product_types_and_strides(a8, b8, kind):
    """Every type pair; output rows on no 16-byte boundary, rows and columns around it untouched."""
    rng = np.random.default_rng(2)
    for m, n, k, pad in ((130, 270, 300, 1), (64, 264, 1024, 8), (9, 31, 4000, 3)):
        a, b = operand(rng, m, k, a8, False, 32), operand(rng, n, k, b8, True, 48)
        wide = torch.full((m + 2, n + pad), 9.0, dtype=KINDS[kind], device=DEV)
        ws = torch.zeros(B.lpd_block_workspace_size(m, n, k), dtype=torch.uint8, device=DEV)
        B.lpd_block_matmul(a, b, wide[:m, :n], ws)
        check_product(a, b, wide[:m, :n], kind)
        assert bool((wide[:, n:] == 9).all()) and bool((wide[m:] == 9).all())
        assert int(ws[:4].view(torch.int32)) == 0


def test_product_zero_sizes_and_nan():
    rng = np.random.default_rng(3)
    a, b = operand(rng, 70, 300, "e4m3", False), operand(rng, 90, 300, "e4m3", True)
    assert B.block_matmul(operand(rng, 0, 300, "e4m3", False), b).shape == (0, 90)
    assert B.block_matmul(a, operand(rng, 0, 300, "e4m3", True)).shape == (70, 0)
    wide = torch.full((70, 100), 5.0, device=DEV)
    ws = torch.empty(B.lpd_block_workspace_size(70, 90, 0), dtype=torch.uint8, device=DEV)
    B.lpd_block_matmul(operand(rng, 70, 0, "e4m3", False), operand(rng, 90, 0, "e4m3", True), wide[:, :90], ws)
    assert bool((wide[:, :90] == 0).all()) and bool((wide[:, 90:] == 5).all())
    # a NaN value or scale reaches its own row or column, and no other
    clean = B.block_matmul(a, b, torch.float32)
    a.values.view(torch.uint8)[3, 17] = 0x7F
    b.scales[0, 1] = float("nan")
    dirty = B.block_matmul(a, b, torch.float32)
    hit = torch.isnan(dirty)
    assert bool(hit[3].all()) and bool(hit.all()), "column scales of the first 128 columns cover all 90"
    b.scales[0, 1] = 1.0
    only = torch.isnan(B.block_matmul(a, b, torch.float32))
    assert bool(only[3].all()) and int(only.sum()) == 90
    assert bool(torch.isfinite(clean).all())


def test_product_rows_do_not_depend_on_the_batch():
    """Many columns: no split, so any subset of rows gives the same bits."""
    rng = np.random.default_rng(4)
    n, k = 39100, 700
    a, b = operand(rng, 300, k, "e4m3", False), operand(rng, n, k, "e4m3", True)
    full = B.block_matmul(a, b, torch.float32)
    for lo, hi in ((0, 1), (17, 90), (128, 300)):
        part = B.BlockScaled(a.values[lo:hi], a.scales[lo:hi])
        if hi - lo == 1:
            assert part.values.data_ptr() % 16 == 0
        assert torch.equal(B.block_matmul(part, b, torch.float32), full[lo:hi])


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("m,n,k,b_block", [(2000, 4099, 300, True), (2000, 4099, 300, False), (130, 261, 900, False), (70, 259, 9000, True)])
def test_product_leaves_aligned_padding(m, n, k, b_block, kind):
    """Output rows on 16-byte boundaries with columns behind them: several tiles a
    multiprocessor, an odd last column, no split of k and one."""
    rng = np.random.default_rng(7)
    a, b = operand(rng, m, k, "e5m2", False), operand(rng, n, k, "e4m3", b_block)
    wide = torch.full((m + 3, -(-n // 8) * 8 + 8), 9.0, dtype=KINDS[kind], device=DEV)
    ws = torch.zeros(B.lpd_block_workspace_size(m, n, k), dtype=torch.uint8, device=DEV)
    B.lpd_block_matmul(a, b, wide[:m, :n], ws)
    check_product(a, b, wide[:m, :n], kind)
    assert bool((wide[:, n:] == 9).all()) and bool((wide[m:] == 9).all())
    again = torch.empty(m, n, dtype=KINDS[kind], device=DEV)  # rows on no boundary: the other way out
    B.lpd_block_matmul(a, b, again, ws)
    assert torch.equal(again, wide[:m, :n])


def test_product_one_row_of_any_stride():
    """A single row's strides are never used, whatever they are."""
    rng = np.random.default_rng(8)
    a, b = operand(rng, 1, 700, "e4m3", False), operand(rng, 500, 700, "e4m3", True)
    room = torch.full((508,), 9.0, device=DEV)
    ws = torch.empty(B.lpd_block_workspace_size(1, 500, 700), dtype=torch.uint8, device=DEV)
    B.lpd_block_matmul(a, b, room.as_strided((1, 500), (2 ** 41, 1)), ws)
    check_product(a, b, room[None, :500], "f32")
    assert bool((room[500:] == 9).all())


def test_two_products_at_once():
    rng = np.random.default_rng(9)
    pairs = [(operand(rng, 300, 2000, "e4m3", False), operand(rng, 5000, 2000, "e4m3", True)) for _ in range(2)]
    want = [B.block_matmul(a, b) for a, b in pairs]
    streams = [torch.cuda.Stream() for _ in pairs]
    rooms = [(torch.empty_like(w), torch.empty(B.lpd_block_workspace_size(300, 5000, 2000), dtype=torch.uint8, device=DEV))
             for w in want]
    torch.cuda.synchronize()
    for _ in range(20):
        for (a, b), s, (out, ws) in zip(pairs, streams, rooms):
            B.lpd_block_matmul(a, b, out, ws, s)
    torch.cuda.synchronize()
    for w, (out, _) in zip(want, rooms):
        assert torch.equal(out, w)


def test_product_streams_graph_and_determinism():
    rng = np.random.default_rng(5)
    shapes = [(50, 700, 6000), (200, 2000, 512)]  # one splits the k axis, one does not
    cases = []
    for m, n, k in shapes:
        x = make(rng, m, k, "bf16")
        w = B.block_quantize(make(rng, n, k, "bf16"), block=True)
        cases.append((x, w, B.block_empty(m, k, torch.float8_e4m3fn), torch.empty(m, n, device=DEV),
                      torch.empty(B.lpd_block_workspace_size(m, n, k), dtype=torch.uint8, device=DEV)))

    def step():
        for x, w, q, out, ws in cases:
            B.lpd_block_quantize(x, q)
            B.lpd_block_matmul(q, w, out, ws)

    step()
    torch.cuda.synchronize()
    want = [c[3].clone() for c in cases]
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        for _ in range(3):
            step()
    torch.cuda.synchronize()
    for c, w in zip(cases, want):
        assert torch.equal(c[3], w)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for c in cases:
        c[0].mul_(1.5)
        c[3].zero_()
    g.replay()
    torch.cuda.synchronize()
    got = [c[3].clone() for c in cases]
    step()
    torch.cuda.synchronize()
    for c, v, w in zip(cases, got, want):
        assert torch.equal(c[3], v) and not torch.equal(v, w)


def test_eight_bit_head_to_gradients():
    """The pieces as they are used: the rollout's 8-bit head, both sides scored
    under the rollout's controls, the logprob's gradient, and the head's two
    gradients; each stage against float64 on the stage's own inputs."""
    rng = np.random.default_rng(6)
    rows, hidden, vocab = 200, 320, 2500
    h = torch.from_numpy(rng.normal(0, 1, (rows, hidden)).astype(np.float32)).to(DEV).to(torch.bfloat16)
    w = torch.from_numpy((rng.normal(0, 3, (vocab, hidden)) / np.sqrt(hidden)).astype(np.float32)).to(DEV).to(torch.bfloat16)
    hq, wq = B.block_quantize(h), B.block_quantize(w, block=True, pow2=True)
    rollout = B.block_matmul(hq, wq)
    check_product(hq, wq, rollout, "bf16")
    train = (h.float() @ w.float().t()).to(torch.bfloat16)
    ids = rng.integers(0, vocab, rows).astype(np.int32)
    c = ref.random_controls(rng, rows, vocab, keep=ids, history=rows)
    handle = B.Controls(**{k: torch.from_numpy(np.ascontiguousarray(v)).to(DEV) for k, v in c.items()})
    idt, act = torch.from_numpy(ids).to(DEV), torch.ones(rows, dtype=torch.uint8, device=DEV)
    res = B.score_controlled(train, rollout, idt, act, handle, handle)
    assert res.metrics["status"] == 0 and res.metrics["n_active"] == rows
    th, rh = (t.double().cpu().numpy() for t in (train, rollout))
    for r in range(rows):
        a, b = (ref.logp(ref.row(c, v[r], r)[0], ids[r]) for v in (th, rh))
        assert abs(float(res.logp_train[r]) - a) <= 1e-5 + 2.0 ** -23 * abs(a)
        assert abs(float(res.dlogp[r]) - (a - b)) <= 2e-5 + 2.0 ** -23 * abs(a - b)
    g = torch.randn(rows, device=DEV)
    d = torch.empty(rows, vocab, dtype=torch.bfloat16, device=DEV)
    B.lpd_logprob_backward_controlled(train, handle, idt, act, res.logp_train, g, d)
    # data gradient: dY (vocab inside) times W^T; weight gradient: dY^T times X^T (rows inside)
    dq = B.block_quantize(d, torch.float8_e5m2)
    wt = B.block_quantize(w, block=True, transpose=True, pow2=True)
    dh = B.block_matmul(dq, wt)
    check_product(dq, wt, dh, "bf16")
    dt, ht = B.block_quantize(d, torch.float8_e5m2, transpose=True), B.block_quantize(h, transpose=True)
    dw = B.block_matmul(dt, ht, torch.float32)
    check_product(dt, ht, dw, "f32")
    # the transposed weight holds the same values as the plain one (128 x 128 scales of powers of two)
    assert torch.equal(meaning(wt), meaning(wq).t())
    # against the unquantised gradients: half a step of each operand on the sum of magnitudes
    dd, ww, hh = d.double().cpu(), w.double().cpu(), h.double().cpu()
    for got, x, y, sx, sy in ((dh, dd, ww.t(), 2.0 ** -3, 2.0 ** -4), (dw, dd.t(), hh.t(), 2.0 ** -3, 2.0 ** -4)):
        want, size = x @ y.t(), x.abs() @ y.abs().t()
        # values far below a block's largest fall among the subnormals: half a subnormal step of the block's scale
        low = x.abs().amax(1, keepdim=True) * 2.0 ** -32 * y.abs().sum(1)[None] + x.abs().sum(1, keepdim=True) * y.abs().max() * 2.0 ** -18
        tol = (sx + sy + sx * sy + 2.0 ** -7) * size + low + 1e-30
        assert bool(((got.double().cpu() - want).abs() <= tol).all())
