"""4-bit microscaled operands from the definition (include/lpd.h, lpd_micro_scaled):
their quantisation step by step in float32, and what they stand for in float64."""
import numpy as np
import torch

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=np.float32)


def e4m3(v):
    """float32 -> (bytes, values), to nearest even, saturating."""
    t = torch.from_numpy(np.minimum(v, np.float32(448.0))).to(torch.float8_e4m3fn)
    return t.view(torch.uint8).numpy(), t.to(torch.float32).numpy()


def e2m1(v):
    """float32 -> codes, to nearest with ties to the even code, saturating."""
    a = np.abs(v)
    c = np.zeros(v.shape, dtype=np.uint8)
    for i in range(7):
        mid = (E2M1[i] + E2M1[i + 1]) / 2
        c[a >= mid if i % 2 else a > mid] = i + 1  # (a tie goes up where the upper code is even)
    return c | np.where(np.signbit(v), 8, 0).astype(np.uint8)


def quantize(x, block, tensor_scale=1.0):
    """x float32 [rows, k] -> (codes [rows, k], scale bytes [rows, blocks], values float32)."""
    rows, k = x.shape
    nb = -(-k // block)
    wide = np.zeros((rows, nb * block), dtype=np.float32)
    wide[:, :k] = x
    tiles = wide.reshape(rows, nb, block)
    t = np.float32(tensor_scale)
    with np.errstate(all="ignore"):
        top = np.abs(tiles).max(2)
        bad = ~np.isfinite(tiles).all(2) | ~(np.isfinite(t) and t > 0)
        top = np.where(bad, np.float32(1), top)
        if block == 16:
            byte, unit = e4m3(top / (np.float32(6) * t))
            byte = np.where(bad, 0x7F, byte)
        else:
            b = (np.clip(top / t, np.float32(2.0 ** -64), np.finfo(np.float32).max) / np.float32(6)).view(np.uint32)
            byte = ((b + 0x7FFFFF) >> 23).astype(np.uint8)
            unit = (byte.astype(np.uint32) << 23).view(np.float32)
            byte = np.where(bad, 0xFF, byte)
        back = np.float32(1) / (unit * t)
        inv = np.where(np.isfinite(back), back, np.float32(0))
        codes = e2m1(np.where(bad[:, :, None], np.float32(0), tiles) * inv[:, :, None])
        sign = np.where(codes & 8, np.float32(-1), np.float32(1))
        values = (sign * E2M1[codes & 7] * unit[:, :, None]) * t
        values = np.where(bad[:, :, None], np.float32(np.nan), values)
    flat = lambda a: a.reshape(rows, nb * block)[:, :k]  # noqa: E731
    return flat(codes), byte.astype(np.uint8), flat(values).astype(np.float32)


def packed(codes):
    """Codes two to a byte, the even column in the low half."""
    rows, k = codes.shape
    wide = np.zeros((rows, -(-k // 2) * 2), dtype=np.uint8)
    wide[:, :k] = codes
    return wide[:, 0::2] | wide[:, 1::2] << 4


def unpacked(p, k):
    return np.stack([p & 15, p >> 4], 2).reshape(p.shape[0], -1)[:, :k]


def at(rows, blocks):
    """[rows, blocks] places of the scale bytes."""
    r, b = np.arange(rows)[:, None], np.arange(blocks)[None]
    return ((r // 128) * -(-blocks // 4) + b // 4) * 512 + r % 32 * 16 + r // 32 % 4 * 4 + b % 4


def tiled(scales):
    rows, blocks = scales.shape
    out = np.zeros(-(-rows // 128) * -(-blocks // 4) * 512, dtype=np.uint8)
    out[at(rows, blocks)] = scales
    return out


def stands_for(codes, scales, block, tensor_scale=1.0):
    """float64 values of codes [rows, k] under scale bytes [rows, blocks]."""
    if block == 16:
        unit = torch.from_numpy(np.ascontiguousarray(scales)).view(torch.float8_e4m3fn).to(torch.float64).numpy()
    else:
        unit = np.where(scales == 255, np.nan, np.exp2(scales.astype(np.float64) - 127))
    v = E2M1[codes & 7].astype(np.float64) * np.where(codes & 8, -1.0, 1.0)
    return v * np.repeat(unit, block, 1)[:, :codes.shape[1]] * float(tensor_scale)
