"""The 4-bit cache's format, one sixteen at a time: e2m1 codes under an e4m3 scale, and a head's page byte by byte."""
from __future__ import annotations

import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def _e4m3_values():
    codes = np.arange(127)                                   # 0x7F is NaN
    e, m = codes >> 3, codes & 7
    return np.where(e > 0, (1 + m / 8) * 2.0 ** (e - 7), m / 8 * 2.0 ** -6)


E4M3 = _e4m3_values()


def nearest_even(x, values):
    """Index of the value nearest to x >= 0, ties to the even index, the largest for all above."""
    i = int(np.searchsorted(values, x))
    if i == len(values):
        return i - 1
    if i == 0:
        return 0
    low, high = x - values[i - 1], values[i] - x
    return i - 1 if low < high or (low == high and (i - 1) % 2 == 0) else i


def quantise16(x, whole_scale):
    """(codes, scale byte) of sixteen float32 values; every operation in float32."""
    t = np.float32(x) * (np.float32(1) / np.float32(whole_scale))
    scale = nearest_even(float(min(np.abs(t).max() * np.float32(1 / 6), np.float32(448))), E4M3)
    by = np.float32(E4M3[scale])
    if by == 0:
        return np.zeros(16, int), scale
    r = t / by
    return np.array([nearest_even(float(abs(v)), E2M1) + 8 * bool(np.signbit(v)) for v in r]), scale


def places(D, slot, d, value):
    """(byte of a head's page, whether its high half) of an element's code, and its scale's byte."""
    base, i = slot // 8 * 9 * D, slot % 8
    if not value:
        return base + i * D // 2 + d // 2, d % 2, base + 4 * D + i * D // 16 + d // 16
    eighth = D // 8
    code = base + 4 * D + D // 2 + (d // eighth * 4 + i // 2) * eighth + i % 2 * (eighth // 2) + d % eighth // 2
    return code, d % 2, base + 8 * D + D // 2 + d // 16 * 8 + i


def write(page, D, slot, x, value, whole_scale):
    """Quantises a token's [D] into a head's page (bytes, changed in place)."""
    for d0 in range(0, D, 16):
        codes, scale = quantise16(x[d0:d0 + 16], whole_scale)
        for d, c in zip(range(d0, d0 + 16), codes):
            at, high, scale_at = places(D, slot, d, value)
            page[at] = (page[at] & 0x0F) | (int(c) << 4) if high else (page[at] & 0xF0) | int(c)
            page[scale_at] = scale


def read(pool, D, page_size, whole_scale, value):
    """[pages, page_size, heads, D] float64 of a layer's pool [pages, heads, bytes]; NaN scales give 0."""
    pages, heads, _ = pool.shape
    out = np.zeros((pages, page_size, heads, D))
    scales = np.append(E4M3, 0.0)
    for slot in range(page_size):
        at = np.array([places(D, slot, d, value) for d in range(D)])
        byte = pool[:, :, at[:, 0]].astype(int)
        code = (byte >> (4 * at[:, 1])) & 15
        out[:, slot] = E2M1[code & 7] * np.where(code >= 8, -1.0, 1.0) * scales[pool[:, :, at[:, 2]].astype(int) & 127]
    return out * whole_scale
