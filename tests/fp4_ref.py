"""Microscaled 4-bit floating point in plain numpy, apart from the library:
the codes and scales of a matrix by the formats' definitions, the values they
stand for, and products in 64 bits."""
from __future__ import annotations

import numpy as np

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
BLOCK = {"mxfp4": 32, "nvfp4": 16}


def half_even(y, fraction_bits, e_min, top):
    """y to the nearest number with `fraction_bits` fraction bits and exponents
    from e_min, halves to even, at most `top`."""
    y = np.asarray(y, dtype=np.float64)
    _, e = np.frexp(np.abs(y))
    step = np.ldexp(1.0, np.maximum(e - 1, e_min) - fraction_bits)
    return np.clip(np.rint(y / step) * step, -top, top)


def e4m3_byte(v):
    """Bytes of values that E4M3 holds exactly (v >= 0)."""
    v = np.asarray(v, dtype=np.float64)
    m, e = np.frexp(v)
    normal = v >= 2.0 ** -6
    b = np.where(normal, ((e - 1 + 7) << 3) + np.rint((2 * m - 1) * 8).astype(int), np.rint(v * 512).astype(int))
    return b.astype(np.uint8)


def e4m3_value(b):
    b = np.asarray(b).astype(int)
    e, f = (b >> 3) & 15, b & 7
    v = np.where(e > 0, (1 + f / 8.0) * np.ldexp(1.0, e - 7), f * 2.0 ** -9)
    v = np.where((b & 0x7F) == 0x7F, np.nan, v)
    return np.where(b & 0x80, -v, v)


def scale_value(b, fmt):
    if fmt == "mxfp4":
        return np.where(b == 255, np.nan, np.ldexp(1.0, b.astype(int) - 127))
    return e4m3_value(b)


def quantize(x, fmt, g=None):
    """(codes [R, K] of 0..15, scale bytes [R, blocks]) of float32 x."""
    x = np.asarray(x, dtype=np.float32)
    R, K = x.shape
    blk = BLOCK[fmt]
    xb = np.pad(x, ((0, 0), (0, -K % blk))).reshape(R, -1, blk)
    bad = ~np.isfinite(xb).all(-1)
    xb = np.where(bad[..., None], np.float32(0), xb)
    amax = np.abs(xb).max(-1)
    if fmt == "mxfp4":
        _, e = np.frexp(amax.astype(np.float64))
        E = np.where(amax > 0, np.maximum(e - 1 - 2, -127), -127)
        byte = (E + 127).astype(np.uint8)
        y = xb.astype(np.float64) * np.ldexp(1.0, -E)[..., None]
        byte = np.where(bad, 255, byte).astype(np.uint8)
    else:
        g = np.float32(1.0 if g is None else g)
        with np.errstate(over="ignore", divide="ignore"):
            s = half_even((amax / (np.float32(6) * g)).astype(np.float32), 3, -6, 448.0)
            d = (s.astype(np.float32) * g).astype(np.float32)
            r = np.where(d > 0, np.float32(1) / np.where(d > 0, d, np.float32(1)), np.float32(0)).astype(np.float32)
        y = (xb * r[..., None]).astype(np.float32).astype(np.float64)
        byte = np.where(bad, 0x7F, e4m3_byte(s)).astype(np.uint8)
    q = half_even(y, 1, 0, 6.0)
    code = np.searchsorted(GRID, np.abs(q)) + 8 * np.signbit(xb)
    code = np.where(bad[..., None], 0, code).reshape(R, -1)[:, :K]
    return code.astype(np.uint8), byte


def values(code, byte, fmt, g=None):
    """The values in 64 bits."""
    R, K = code.shape
    v = GRID[code & 7] * np.where(code & 8, -1.0, 1.0)
    s = scale_value(byte, fmt)
    if g is not None:
        s = s * np.float64(np.float32(g))
    return v * np.repeat(s, BLOCK[fmt], axis=1)[:, :K]


def pack(code):
    """uint8 [R, ceil(K / 32) * 16], the even column in the low half."""
    R, K = code.shape
    c = np.pad(code, ((0, 0), (0, -K % 32)))
    return (c[:, 0::2] | (c[:, 1::2] << 4)).astype(np.uint8)


def tile_scales(byte, K, fmt):
    """Scale bytes [R, blocks] in tiles of 128 rows × 4 blocks, padding 0."""
    R = byte.shape[0]
    nb = -(-K // 256) * (256 // BLOCK[fmt])
    out = np.zeros(-(-R // 128) * 128 * nb, dtype=np.uint8)
    r = np.arange(R)[:, None]
    b = np.arange(byte.shape[1])[None, :]
    out[((r // 128) * (nb // 4) + b // 4) * 512 + (r % 32) * 16 + (r % 128 // 32) * 4 + b % 4] = byte
    return out
