"""The paged 8-bit cache in plain numpy, apart from the library: appends by
their definition, token by token and page by page, and attention in 64 bits."""
from __future__ import annotations

import numpy as np

from fp4_ref import e4m3_byte, e4m3_value, half_even


def encode(x):
    """float64 values to E4M3 bytes: nearest, halves to even, at most 448; NaN 0x7F."""
    x = np.asarray(x, dtype=np.float64)
    nan = np.isnan(x)
    v = half_even(np.where(nan, 0.0, np.clip(x, -448.0, 448.0)), 3, -6, 448.0)
    return np.where(nan, 0x7F, e4m3_byte(np.abs(v)) | (np.signbit(x).astype(np.uint8) << 7)).astype(np.uint8)


def page_scale(amax):
    """The smallest power of two s >= 2^-126 with amax <= 448 s."""
    e = -126
    while amax > 448.0 * 2.0 ** e:
        e += 1
    return 2.0 ** e


def append(codes, scale, new, table, starts, counts):
    """codes uint8 [P, H, page, D], scale float32 [P, H] in place; new float64 [B, T, H, D]."""
    page = codes.shape[2]
    for b in range(new.shape[0]):
        lo, hi = int(starts[b]), int(starts[b]) + int(counts[b])
        for slot in range(lo // page, (hi + page - 1) // page if hi > lo else lo // page):
            a, z = max(lo, slot * page), min(hi, (slot + 1) * page)
            p, old = int(table[b][slot]), a - slot * page
            for h in range(codes.shape[1]):
                x = new[b, a - lo:z - lo, h]
                finite = np.abs(x[np.isfinite(x)])
                s = page_scale(finite.max() if finite.size else 0.0)
                if old:
                    had = float(scale[p, h])
                    s = max(s, had)
                    if s > had:
                        codes[p, h, :old] = encode(e4m3_value(codes[p, h, :old]) * (had / s))
                codes[p, h, old:old + z - a] = encode(x / s)
                scale[p, h] = s


def values(codes, scale, table_row, length):
    """float64 [H, length, D] of one sequence."""
    page = codes.shape[2]
    n = -(-length // page)
    ids = np.asarray(table_row[:n], dtype=np.int64)
    x = e4m3_value(codes[ids]) * scale[ids].astype(np.float64)[:, :, None, None]
    return x.transpose(1, 0, 2, 3).reshape(codes.shape[1], n * page, -1)[:, :length]


def attention(q, codes_k, scale_k, codes_v, scale_v, table, lengths, counts, causal, scale):
    """(o, lse, Σ p|v|) in float64 for q [B, T, Hq, D]."""
    B, T, Hq, D = q.shape
    o, mag = np.zeros(q.shape), np.zeros(q.shape)
    lse = np.full((B, T, Hq), -np.inf)
    H = codes_k.shape[1]
    for b in range(B):
        n = int(lengths[b])
        if n == 0:
            continue
        k, v = values(codes_k, scale_k, table[b], n), values(codes_v, scale_v, table[b], n)
        for t in range(int(counts[b])):
            seen = max(0, n - int(counts[b]) + t + 1) if causal else n
            if seen == 0:
                continue
            for h in range(Hq):
                g = h // (Hq // H)
                s = (k[g, :seen] @ q[b, t, h]) * scale
                m = s.max()
                p = np.exp(s - m)
                l = p.sum()
                o[b, t, h] = p @ v[g, :seen] / l
                mag[b, t, h] = p @ np.abs(v[g, :seen]) / l
                lse[b, t, h] = m + np.log(l)
    return o, lse, mag
