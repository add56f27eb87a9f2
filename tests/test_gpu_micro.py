"""4-bit microscaled operands on the GPU (needs a GPU): quantisation bit for bit
against the definition in micro_ref.py, the product against float64.

Bound of the product.  Terms are exact (two 2-bit significands and two scales of 4
bits); an MMA adds 64 of them and the running sum with at least float32's 24 bits,
each of the ceil(k / 64) sums off by at most 2^-22 of the terms' absolute sum S (two
truncations of 2^-23), a split's join adds as many float32 additions as there are
parts (at most 152, 2^-24 each), the tensor scales two roundings and the output its half step.
"""
import subprocess
import sys
from pathlib import Path

import numpy as np
import pytest
import torch

from tests import micro_ref as ref
from tests import sample_ref
from logprob_drift_scoring_gb300 import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda"
ROOT = Path(__file__).resolve().parent.parent
KINDS = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


def rand(rng, rows, cols, kind):
    x = rng.normal(0, 1, (rows, cols)) * rng.uniform(0.2, 3, (rows, 1))
    return torch.from_numpy(x.astype(np.float32)).to(DEV).to(KINDS[kind])


def f32(t):
    return t.float().cpu().numpy()


def one(v):
    return torch.tensor([v], dtype=torch.float32, device=DEV)


def check_quantize(x, block, transpose=False, ts=None, vkind=None, pad=0):
    """The call's codes, scales, values and what it leaves alone."""
    rows, k = tuple(x.shape)[::-1] if transpose else tuple(x.shape)
    kb = -(-k // 2)
    room = torch.full((rows, kb + pad), 0xA5, dtype=torch.uint8, device=DEV)
    scales = torch.full((B.lpd_micro_scale_bytes(block, rows, k),), 0xA5, dtype=torch.uint8, device=DEV)
    out = B.MicroScaled(room[:, :kb], scales, k, block, None if ts is None else one(ts))
    values = None
    if vkind:
        wide = torch.full((rows, k + pad), 77.0, dtype=KINDS[vkind], device=DEV)
        values = wide[:, :k]
    B.lpd_micro_quantize(x, out, transpose, values)
    torch.cuda.synchronize()
    xh = f32(x).T if transpose else f32(x)
    codes, byte, want = ref.quantize(np.ascontiguousarray(xh), block, 1.0 if ts is None else ts)
    got = ref.unpacked(room[:, :kb].cpu().numpy(), k)
    fine = np.isfinite(want)
    assert np.array_equal(got[fine], codes[fine]), np.argwhere((got != codes) & fine)[:5]
    assert np.array_equal(scales.cpu().numpy(), ref.tiled(byte))
    if k % 2:
        assert not (room[:, kb - 1].cpu().numpy() >> 4).any() or not fine.all()
    assert bool((room[:, kb:] == 0xA5).all())
    if vkind:
        w = torch.from_numpy(want).to(KINDS[vkind]).float().numpy()
        assert np.array_equal(f32(values), w, equal_nan=True)
        assert bool((wide[:, k:] == 77.0).all())
    return out


@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("kind,vkind", [("bf16", "bf16"), ("f32", "f32"), ("bf16", None), ("f32", "bf16")])
@pytest.mark.parametrize("rows,cols,pad", [(1, 1, 0), (1, 16, 0), (3, 17, 3), (2, 31, 0), (5, 33, 16), (128, 128, 0), (129, 127, 1),
                                           (64, 200, 16), (131, 300, 8), (300, 65, 7), (256, 512, 0)])
def test_quantize(rows, cols, pad, kind, vkind, block, transpose):
    rng = np.random.default_rng(rows * 1000 + cols)
    check_quantize(rand(rng, rows, cols, kind), block, transpose, None if block == 32 else 0.003, vkind, pad)


@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("block", [16, 32])
def test_quantize_extremes(block, transpose):
    """Zeros of both signs, ties, denormals, huge values, NaN, infinities, odd strides."""
    rng = np.random.default_rng(1)
    x = rng.normal(0, 1, (70, 140)).astype(np.float32)
    x[0], x[1], x[2] = 0.0, -0.0, 1e-40
    x[3], x[4], x[5] = 3e38, 1e-30, rng.choice([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0], 140) * rng.choice([-1, 1], 140)
    x[6, 5], x[7, 64], x[8, 139], x[9, 0] = np.nan, np.inf, -np.inf, np.nan
    x[10:20] *= 1e4
    x[20:30] *= 1e-4
    wide = torch.zeros(70, 147, device=DEV)
    wide[:, 3:143] = torch.from_numpy(x).to(DEV)
    for ts in (None, 1.0, 0.0123, 1e-20, 1e20):
        check_quantize(wide[:, 3:143], block, transpose, ts, "f32")
    for ts in (0.0, -1.0, float("nan"), float("inf")):
        out = check_quantize(wide[:, 3:143], block, transpose, ts, "f32")
        assert out is not None


@pytest.mark.parametrize("block", [16, 32])
def test_quantize_larger(block):
    rng = np.random.default_rng(2)
    for transpose in (False, True):
        check_quantize(rand(rng, 1111, 2051, "bf16"), block, transpose, 0.002 if block == 16 else None, "bf16")


def operand(rng, rows, k, block, ts=None, pad=0):
    """Random codes and scales, laid out as the product takes them."""
    codes = rng.integers(0, 16, (rows, k)).astype(np.uint8)
    nb = -(-k // block)
    scales = rng.integers(0x20, 0x48, (rows, nb)).astype(np.uint8) if block == 16 else rng.integers(120, 131, (rows, nb)).astype(np.uint8)
    kb = -(-k // 2)
    room = torch.full((rows, -(-kb // 16) * 16 + pad), 0xFF, dtype=torch.uint8, device=DEV)
    room[:, :kb] = torch.from_numpy(ref.packed(codes)).to(DEV)
    t = torch.from_numpy(ref.tiled(scales)).to(DEV)
    op = B.MicroScaled(room[:, :kb], t, k, block, None if ts is None else one(ts))
    return op, ref.stands_for(codes, scales, block, 1.0 if ts is None else np.float32(ts))


def check_product(a, b, va, vb, kind, out=None):
    m, n, k = len(va), len(vb), va.shape[1]
    if out is None:
        out = torch.full((m, n), float("nan"), dtype=KINDS[kind], device=DEV)
    ws = torch.empty(B.lpd_micro_workspace_size(m, n, k), dtype=torch.uint8, device=DEV)
    ws[:4] = 0
    B.lpd_micro_matmul(a, b, out, ws)
    torch.cuda.synchronize()
    assert int(ws[:4].view(torch.int32)[0]) == 0
    ta, tb = torch.from_numpy(va).to(DEV), torch.from_numpy(vb).to(DEV)
    want, size = ta @ tb.T, ta.abs() @ tb.abs().T
    err = (out.double() - want).abs()
    bound = (-(-k // 64) * 2.0 ** -22 + 156 * 2.0 ** -24) * size + (2.0 ** -23 + HALF[kind]) * want.abs()
    assert bool((err <= bound).all()), (float((err / bound.clamp(min=1e-300)).max()), float((err / size.clamp(min=1e-300)).max()))
    return out


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("m,n,k", [(128, 256, 256), (1, 1, 1), (1, 1, 64), (5, 7, 33), (128, 256, 64), (128, 256, 128), (128, 256, 192),
                                   (16, 1000, 512), (129, 257, 300), (200, 130, 1030), (300, 600, 97), (1, 5000, 2048), (257, 64, 4111)])
def test_product(m, n, k, block, kind):
    rng = np.random.default_rng(m + n + k)
    a, va = operand(rng, m, k, block, 0.37)
    b, vb = operand(rng, n, k, block, 1.9 if m % 2 else None)
    check_product(a, b, va, vb, kind)


@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("m,n,k", [(2500, 4000, 512), (64, 512, 40000), (700, 8200, 1000)])
def test_product_many_tiles_and_splits(m, n, k, block):
    rng = np.random.default_rng(m)
    a, va = operand(rng, m, k, block)
    b, vb = operand(rng, n, k, block)
    check_product(a, b, va, vb, "bf16")


def test_every_place_has_its_own_scale_and_code():
    """One value of A and of B at a time: the output is that product alone."""
    rng = np.random.default_rng(4)
    for block in (16, 32):
        m, n, k = 130, 260, 520
        a, va = operand(rng, m, k, block)
        vb = np.zeros((n, k))
        codes = np.zeros((n, k), dtype=np.uint8)
        at = rng.permutation(k)[:n]
        codes[np.arange(n), at] = 3
        scales = rng.integers(0x30, 0x40, (n, -(-k // block))).astype(np.uint8) if block == 16 else rng.integers(125, 130, (n, -(-k // block))).astype(np.uint8)
        vb = ref.stands_for(codes, scales, block)
        b = B.MicroScaled(torch.from_numpy(ref.packed(codes)).to(DEV).contiguous(), torch.from_numpy(ref.tiled(scales)).to(DEV), k, block) \
            if -(-k // 2) % 16 == 0 else None
        if b is None:
            room = torch.zeros(n, -(-k // 32) * 16, dtype=torch.uint8, device=DEV)
            room[:, :-(-k // 2)] = torch.from_numpy(ref.packed(codes)).to(DEV)
            b = B.MicroScaled(room, torch.from_numpy(ref.tiled(scales)).to(DEV), k, block)
        out = B.micro_matmul(a, b, torch.float32)
        assert np.array_equal(f32(out), (va @ vb.T).astype(np.float32))


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_output_strides_and_columns_behind(kind):
    """Rows on and off 16-byte boundaries; what lies behind n and m stays as it was."""
    rng = np.random.default_rng(5)
    for m, n, stride, shift in ((37, 259, 264, 0), (140, 300, 301, 0), (37, 259, 280, 8), (33, 100, 333, 3), (130, 511, 512, 0)):
        a, va = operand(rng, m, 320, 16)
        b, vb = operand(rng, n, 320, 16)
        room = torch.full((m + 2, stride), 5.0, dtype=KINDS[kind], device=DEV)
        out = room[1:m + 1, shift:shift + n]
        check_product(a, b, va, vb, kind, out)
        keep = room.clone()
        keep[1:m + 1, shift:shift + n] = 5.0
        assert bool((keep == 5.0).all())


def test_zero_k_and_nan_blocks():
    rng = np.random.default_rng(6)
    e = B.micro_empty(5, 0, 16)
    out = torch.full((5, 5), 3.0, device=DEV)
    B.lpd_micro_matmul(e, e, out, torch.empty(B.lpd_micro_workspace_size(5, 5, 0), dtype=torch.uint8, device=DEV))
    assert not out.any()
    x = rand(rng, 20, 200, "bf16")
    x[7, 150] = float("inf")
    for block in (16, 32):
        q, w = B.micro_quantize(x, block), B.micro_quantize(rand(rng, 30, 200, "bf16"), block)
        y = B.micro_matmul(q, w, torch.float32)
        assert bool(torch.isnan(y[7]).all()) and bool(torch.isfinite(y[torch.arange(20, device=DEV) != 7]).all())


@pytest.mark.parametrize("block", [16, 32])
def test_linear_layer_and_its_gradients(block):
    """Forward, data gradient and weight gradient of Y = X W^T on quantised operands,
    each against the product of the values that the operands stand for."""
    rng = np.random.default_rng(7)
    tokens, hidden, vocab = 75, 384, 1030
    x, w, dy = rand(rng, tokens, hidden, "bf16"), rand(rng, vocab, hidden, "bf16"), rand(rng, tokens, vocab, "bf16")
    ts = {k: (v.abs().max().float() / 2688).reshape(1) if block == 16 else None for k, v in (("x", x), ("w", w), ("dy", dy))}

    def both(t, name, transpose):
        rows, k = tuple(t.shape)[::-1] if transpose else tuple(t.shape)
        q = B.micro_empty(rows, k, block, ts[name])
        v = torch.empty(rows, k, device=DEV)
        B.lpd_micro_quantize(t, q, transpose, v)
        return q, v

    for left, right in ((("x", x, False), ("w", w, False)), (("dy", dy, False), ("w", w, True)), (("dy", dy, True), ("x", x, True))):
        (qa, a), (qb, b) = both(left[1], left[0], left[2]), both(right[1], right[0], right[2])
        y = B.micro_matmul(qa, qb, torch.float32)
        a, b = a.double(), b.double()
        want, size = a @ b.T, a.abs() @ b.abs().T
        # (the values carry one more rounding of float32 each)
        bound = (-(-a.shape[1] // 64) * 2.0 ** -22 + 160 * 2.0 ** -24) * size + 2.0 ** -22 * want.abs()
        assert bool(((y.double() - want).abs() <= bound).all())


def test_head_of_a_rollout_from_hidden_rows_to_drift():
    """A run: hidden rows and head in 4 bits, logits, a filtered draw, its kept sets,
    and the drift of the 4-bit rollout against the bf16 head."""
    rng = np.random.default_rng(8)
    rows, hidden, vocab = 40, 256, 3001
    h, w = rand(rng, rows, hidden, "bf16"), (rand(rng, vocab, hidden, "f32") * 0.2).to(torch.bfloat16)
    train = h.float() @ w.float().T
    t = lambda v: (v.abs().max().float() / 2688).reshape(1)  # noqa: E731
    logits = B.micro_matmul(B.micro_quantize(h, 16, t(h)), B.micro_quantize(w, 16, t(w)), torch.float32)
    filt = B.Filter(scale=torch.full((rows,), 0.9, device=DEV), top_k=torch.full((rows,), 50, dtype=torch.int32, device=DEV),
                    top_p=torch.full((rows,), 0.95, device=DEV))
    ids, logp, kept = B.sample(logits, torch.rand(rows, device=DEV), filt)
    mask, lse, mkept = B.filter_mask(logits, filt, ids)
    assert torch.equal(kept, mkept) and bool((ids >= 0).all()) and bool((kept >= 1).all()) and bool((kept <= 50).all())
    c = B.Controls(scale=filt.scale, mask=mask)
    act = torch.ones(rows, dtype=torch.uint8, device=DEV)
    res = B.score_controlled(train, logits, ids, act, train_controls=c, rollout_controls=c)
    assert res.metrics["status"] == 0
    assert bool(((res.logp_rollout - logp).abs() <= 1.1e-5 + 2.0 ** -23 * logp.abs()).all())
    z = torch.where(torch.from_numpy(sample_ref.bits(mask.cpu().numpy(), vocab)).to(DEV), train.double() * filt.scale.double()[:, None], -float("inf"))
    want = torch.log_softmax(z, 1).gather(1, ids.long()[:, None])[:, 0]
    assert bool(((res.logp_train.double() - want).abs() <= 1.1e-5 + 2.0 ** -22 * want.abs()).all())


@pytest.mark.parametrize("block", [16, 32])
def test_a_row_does_not_depend_on_the_other_rows(block):
    """One row tile, whose CTAs are alone, and several, whose are pairs: the same bits (the k axis
    is not split where a row of tiles fills half of the multiprocessors)."""
    rng = np.random.default_rng(21)
    n, k = 256 * 100, 1000
    w = B.micro_quantize(rand(rng, n, k, "bf16"), block)
    x = rand(rng, 300, k, "bf16")
    whole = B.micro_matmul(B.micro_quantize(x, block), w, torch.float32)
    for m in (1, 100, 128, 129):
        assert torch.equal(B.micro_matmul(B.micro_quantize(x[:m].contiguous(), block), w, torch.float32), whole[:m]), m


@pytest.mark.parametrize("transpose", [False, True])
def test_rows_far_apart(transpose):
    """Offsets beyond 32 bits of what is read, of the values and of the product."""
    rng = np.random.default_rng(22)
    rows, k = 3, 70
    x = rand(rng, rows, k, "bf16")
    far = 2 ** 30 + 2 ** 20
    y = torch.empty(2 * far + k, dtype=x.dtype, device=DEV).as_strided((rows, k), (far, 1))
    y.copy_(x)
    out_rows = k if transpose else rows
    far_values = 2 ** 31 // (out_rows - 1) // 8 * 8 + 8
    cols = rows if transpose else k
    values = torch.empty(far_values * (out_rows - 1) + cols, dtype=x.dtype, device=DEV).as_strided((out_rows, cols), (far_values, 1))
    plain = torch.empty(out_rows, cols, dtype=x.dtype, device=DEV)
    a, b = (B.micro_empty(out_rows, cols, 16) for _ in range(2))
    B.lpd_micro_quantize(x, a, transpose, plain)
    B.lpd_micro_quantize(y, b, transpose, values)
    assert torch.equal(a.codes, b.codes) and torch.equal(a.scales, b.scales) and torch.equal(values, plain)
    del y, values
    far = 2 ** 31 // (out_rows - 1) // 8 * 8 + 8
    out = torch.empty(far * (out_rows - 1) + out_rows, dtype=x.dtype, device=DEV).as_strided((out_rows, out_rows), (far, 1))
    B.lpd_micro_matmul(a, a, out, torch.empty(B.lpd_micro_workspace_size(out_rows, out_rows, cols), dtype=torch.uint8, device=DEV))
    assert torch.equal(out, B.micro_matmul(a, a))


def test_first_call_is_captured():
    """In a process that has called nothing yet."""
    code = """
import torch
from logprob_drift_scoring_gb300 import binding as B
x = torch.randn(200, 320, device="cuda").bfloat16()
q = B.micro_empty(200, 320, 16)
out = torch.empty(200, 200, device="cuda")
ws = torch.empty(1 << 24, dtype=torch.uint8, device="cuda")
g, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
torch.cuda.synchronize()
with torch.cuda.stream(side), torch.cuda.graph(g, stream=side):
    B.lpd_micro_quantize(x, q)
    B.lpd_micro_matmul(q, q, out, ws)
g.replay()
torch.cuda.synchronize()
assert torch.equal(out, B.micro_matmul(q, q, torch.float32))
"""
    done = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert done.returncode == 0, done.stderr[-2000:]


def test_repeated_streams_and_graph():
    rng = np.random.default_rng(9)
    x, w = rand(rng, 200, 640, "bf16"), rand(rng, 900, 640, "bf16")
    qw = B.micro_quantize(w, 32)
    q = B.micro_empty(200, 640, 32)
    out = torch.empty(200, 900, device=DEV)
    ws = torch.empty(B.lpd_micro_workspace_size(200, 900, 640), dtype=torch.uint8, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        B.lpd_micro_quantize(x, q)
        B.lpd_micro_matmul(q, qw, out, ws)
        with torch.cuda.graph(g, stream=side):
            B.lpd_micro_quantize(x, q)
            B.lpd_micro_matmul(q, qw, out, ws)
    torch.cuda.synchronize()
    for seed in range(3):
        x.copy_(rand(np.random.default_rng(seed), 200, 640, "bf16"))
        g.replay()
        want = B.micro_matmul(B.micro_quantize(x, 32), qw, torch.float32)
        other = torch.cuda.Stream()
        other.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(other):
            again = B.micro_matmul(B.micro_quantize(x, 32), qw, torch.float32)
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(out, again)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("m,n,k", [(5, 300, 320), (200, 300, 320), (3, 40, 9000)])  # a tile, a pair, a split k axis
@pytest.mark.parametrize("ta,tb", [(1e-20, 1e-20), (1e-23, 1e-23), (1e20, 1e-20), (1e20, 1e20), (3e38, 2e-38), (1e-44, 1e30), (3e38, 3e38),
                                   (1e-45, 1e-45), (0.0, 3e38), (1e-30, 1e-8)])
def test_tensor_scales_whose_product_leaves_float32(ta, tb, m, n, k, block, kind):
    """The scaled sums count, not the scales' product: a row of zeros stays zero, and what
    float32 (or bf16) holds has its digits.  The bound of check_product, whose sums are those
    without the scales, and a step of float32's denormal numbers for each of two roundings; a
    result past the type's range may be infinite from half a step (and the sums' error) below."""
    rng = np.random.default_rng(30)
    a, va = operand(rng, m, k, block)
    b, vb = operand(rng, n, k, block)
    a.codes[1] = 0
    va[1] = 0.0
    t = np.float32([ta, tb]).astype(np.float64)
    a, b = (B.MicroScaled(o.codes, o.scales, k, block, one(s)) for o, s in ((a, ta), (b, tb)))
    out = B.micro_matmul(a, b, KINDS[kind])
    torch.cuda.synchronize()
    got = out.double().cpu().numpy()
    assert (got[1] == 0).all()
    sums, size = va @ vb.T, np.abs(va) @ np.abs(vb).T
    want = sums * (t[0] * t[1])
    bound = (-(-k // 64) * 2.0 ** -22 + 156 * 2.0 ** -24) * size * (t[0] * t[1]) + (2.0 ** -23 + HALF[kind]) * np.abs(want) + 2 * 2.0 ** -149
    if kind == "bf16":
        bound += 2.0 ** -134  # (half a step of bf16's denormal numbers)
    most = float(torch.finfo(KINDS[kind]).max)
    inside = np.abs(want) + bound <= most
    assert (np.abs(got - want)[inside] <= bound[inside]).all()
    assert np.isinf(got[np.abs(want) - bound > most * (1 + HALF[kind])]).all() and not np.isnan(got).any()


@pytest.mark.parametrize("block", [16, 32])
def test_every_scale_byte(block):
    """Each scale that a byte can say, on one value: the denormal e4m3 scales and the powers of
    two down to 2^-127 among them, against a partner that keeps the product in float32's range."""
    bytes_ = np.arange(1, 0x7F) if block == 16 else np.arange(0, 255)
    m, n = len(bytes_), 8
    codes = np.zeros((m, block), dtype=np.uint8)
    codes[:, 3] = 1 + np.arange(m) % 7
    scales = bytes_.astype(np.uint8)[:, None]
    for other in ((0x38,) if block == 16 else (127, 200, 60)):
        vb = np.zeros((n, block), dtype=np.uint8)
        vb[:, 3] = np.arange(n)
        sb = np.full((n, 1), other, dtype=np.uint8)
        a, b = (B.MicroScaled(torch.from_numpy(np.pad(ref.packed(c), ((0, 0), (0, 16 - block // 2)))).to(DEV), torch.from_numpy(ref.tiled(s)).to(DEV), block, block)
                for c, s in ((codes, scales), (vb, sb)))
        out = B.micro_matmul(a, b, torch.float32).cpu().numpy()
        with np.errstate(over="ignore"):
            want = (ref.stands_for(codes, scales, block) @ ref.stands_for(vb, sb, block).T)
        fits = (np.abs(want) >= 2.0 ** -126) & (np.abs(want) < 2.0 ** 127) | (want == 0)
        assert np.array_equal(out[fits], want[fits].astype(np.float32))
