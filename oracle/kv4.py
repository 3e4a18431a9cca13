"""The 4-bit key/value cache in 64 bits: the format's two roundings, its bytes, and a step's norms and rotation.

Blocks of 16 elements, codes e2m1, scales e4m3, one power of two g for a pool; a page of one group holds its tokens'
codes (16 ceil(d / 32) bytes each, the low nibble first) and then the scales, [page_size / 4][2 ceil(d / 32)][4].
"""
from __future__ import annotations

import numpy as np

CODES = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
SCALES = np.array([m / 512 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7) for e in range(16) for m in range(8)][:127])
NAN_SCALE = 0x7F


def nearest(x, grid):
    """Index of the nearest value of a rising grid, ties to the even index; past the ends, the ends."""
    x = np.asarray(x, dtype=np.float64)
    up = np.clip(np.searchsorted(grid, x), 1, len(grid) - 1)
    lo, hi = grid[up - 1], grid[up]
    odd = (up - 1) % 2 == 1
    # distances by multiplication, so that a tie is exact: x against (lo + hi) / 2
    above = (x + x > lo + hi) | ((x + x == lo + hi) & odd)
    return np.where(above, up, up - 1)


def quantise(x, g):
    """(codes [..., d], scale bytes [..., d / 16]) of rows x [..., d]."""
    x = np.asarray(x, dtype=np.float64)
    b = x.reshape(x.shape[:-1] + (-1, 16))
    bad = ~np.isfinite(b).all(-1)
    b = np.where(bad[..., None], 0.0, b)
    s = nearest(np.abs(b).max(-1) / (6 * g), SCALES)
    # |x| against code * scale * g, without a quotient: both sides exact where x is
    step = SCALES[s][..., None] * g
    mid = (CODES[1:] + CODES[:-1]) / 2
    size = np.abs(b)
    codes = np.zeros(b.shape, dtype=np.int64)
    for i, m in enumerate(mid):
        codes = np.where((size > m * step) | ((size == m * step) & (i % 2 == 1)), i + 1, codes)
    codes = np.where(step > 0, codes, 0) + 8 * np.signbit(b)
    return codes.reshape(x.shape), np.where(bad, NAN_SCALE, s)


def values(codes, scales, g):
    codes, scales = np.asarray(codes), np.asarray(scales)
    v = np.where(codes & 8, -1.0, 1.0) * CODES[codes & 7]
    s = np.where(scales & 127 == NAN_SCALE, np.nan, np.append(SCALES, np.nan)[scales & 127])
    return (v.reshape(v.shape[:-1] + (-1, 16)) * s[..., None] * g).reshape(v.shape)


def page_bytes(page_size, d):
    return page_size * -(-d // 32) * 18


def put(page, token, page_size, codes, scales):
    """Writes one token's row into `page`, the uint8 bytes of a page of one group."""
    d, nc = len(codes), -(-len(codes) // 32)
    full = np.zeros(32 * nc, dtype=np.uint8)
    full[:d] = codes
    page[token * 16 * nc:(token + 1) * 16 * nc] = full[0::2] | full[1::2] << 4
    s = np.zeros(2 * nc, dtype=np.uint8)
    s[:d // 16] = scales
    at = page_size * 16 * nc + token // 4 * 8 * nc + token % 4
    page[at:at + 8 * nc:4] = s


def get(pages, page_size, d):
    """(codes, scales) of every token of pages [..., bytes]: [..., page_size, d] and [..., page_size, d / 16]."""
    nc = -(-d // 32)
    c = pages[..., :page_size * 16 * nc].reshape(pages.shape[:-1] + (page_size, 16 * nc))
    c = np.stack([c & 15, c >> 4], -1).reshape(c.shape[:-1] + (32 * nc,))[..., :d]
    s = pages[..., page_size * 16 * nc:].reshape(pages.shape[:-1] + (page_size // 4, 2 * nc, 4))
    s = np.moveaxis(s, -1, -2).reshape(pages.shape[:-1] + (page_size, 2 * nc))[..., :d // 16]
    return c, s


def turned(x, pos, cos, sin, gain=None, eps=0.0, interleaved=False):
    """Rows x [T, heads, d] normalised (with a gain) and rotated by positions pos [T]."""
    x = np.asarray(x, dtype=np.float64)
    if gain is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + float(np.float32(eps))) * np.asarray(gain, dtype=np.float64)
    half = cos.shape[1]
    a, b = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else (slice(0, half), slice(half, 2 * half))
    c, s = (np.asarray(t, dtype=np.float64)[pos][:, None] for t in (cos, sin))
    y = x.copy()
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., a] * s + x[..., b] * c
    return y
