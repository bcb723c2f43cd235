"""CPU oracle of caches of 8-bit rows: the codes and scales of a row, what they
stand for, the append that writes them.

TEST INFRASTRUCTURE ONLY: imported by tests/, never by the product path.
Shares no code with the HIP library. Codes and scales are defined by float32
arithmetic, each operation rounded by itself, so the oracle does those steps in
numpy's float32 and its answers are exact; what a row stands for, and all that
is done with it (oracle/verify.py), is float64. Codes are held as the 256 byte
values (uint8).
"""

from __future__ import annotations

import numpy as np

from oracle import verify as O

MOST = {"e4m3": 448.0, "i8": 127.0}


def decode(kind: str) -> np.ndarray:
    """The value of each of the 256 codes (float64; e4m3's two NaN codes: NaN)."""
    c = np.arange(256)
    if kind == "i8":
        return np.where(c < 128, c, c - 256).astype(np.float64)
    e, f = c >> 3 & 15, c & 7
    v = np.where(e == 0, f / 8 * 2.0 ** -6, (1 + f / 8) * 2.0 ** (e - 7.0))
    v[(e == 15) & (f == 7)] = np.nan
    return np.where(c < 128, v, -v)


def nearest(y: np.ndarray, kind: str) -> np.ndarray:
    """Code (uint8) of the value nearest to each y, between two the one whose code is even; beyond
    the largest, the largest. (A zero keeps its sign in e4m3.)"""
    y = np.asarray(y, np.float64)
    value = decode(kind)
    most = MOST[kind]
    codes = np.array([c for c in range(128) if 0 <= value[c] <= most])  # ascending by value
    grid = value[codes]
    a = np.minimum(np.abs(y), most)
    hi = np.clip(np.searchsorted(grid, a), 1, len(grid) - 1)
    lo = hi - 1
    up, down = grid[hi] - a, a - grid[lo]  # exact: float64, few bits
    take = np.where(up < down, hi, np.where(down < up, lo, np.where(codes[lo] % 2 == 0, lo, hi)))
    c = codes[take]
    neg = np.signbit(y)
    return (np.where(neg, c | 128, c) if kind == "e4m3" else np.where(neg, -c, c) & 255).astype(np.uint8)


def quantise(x: np.ndarray, kind: str):
    """(codes, scales) of float32 rows x [..., n]."""
    assert x.dtype == np.float32
    inverse = np.float32(1.0 / MOST[kind])
    with np.errstate(all="ignore"):
        fine = np.isfinite(x).all(-1)
        a = np.where(fine, np.abs(np.where(fine[..., None], x, 0)).max(-1), 0).astype(np.float32)
        scale = np.maximum(a * inverse, np.float32(2.0 ** -126))
        y = np.where(fine[..., None], x, np.float32(0)) * (np.float32(1) / scale)[..., None]
    assert y.dtype == np.float32
    codes = np.where(fine[..., None], nearest(y, kind), 0).astype(np.uint8)
    return codes, np.where(fine, scale, np.float32(np.nan)).astype(np.float32)


def values(codes: np.ndarray, scales: np.ndarray, kind: str) -> np.ndarray:
    with np.errstate(invalid="ignore"):
        return decode(kind)[codes] * scales.astype(np.float64)[..., None]


def rotate32(x: np.ndarray, cos: np.ndarray, sin: np.ndarray, interleaved: bool) -> np.ndarray:
    """float32 x [heads, dh] turned by the angles of one position, product by product."""
    half = len(cos)
    y = x.copy()
    i = np.arange(half) * 2 if interleaved else np.arange(half)
    j = i + 1 if interleaved else i + half
    with np.errstate(all="ignore"):
        y[:, i] = x[:, i] * cos - x[:, j] * sin
        y[:, j] = x[:, j] * cos + x[:, i] * sin
    return y


def append(k, v, k_cache, v_cache, k_scale, v_scale, kind, past_len, rope=None, interleaved=False,
           table=None, depths=None, num_nodes=None):
    """Returns (k codes, v codes, k scales, v scales); inputs unchanged. k, v [batch, T, heads, dh]
    float32; codes [pages, heads, page_size, dh] uint8; rope float32."""
    batch, T = k.shape[:2]
    pages, _, page_size, _ = k_cache.shape
    got = [a.copy() for a in (k_cache, v_cache, k_scale, v_scale)]
    for b in range(batch):
        past = int(past_len[b])
        n = T - 1 if num_nodes is None else min(max(int(num_nodes[b]), 0), T - 1)
        for j in range(n + 1 if past >= 0 else 0):
            pos = past + (0 if j == 0 else int(depths[b, j - 1]) if depths is not None else j)
            if rope is not None and not 0 <= pos < len(rope):
                continue
            at = O.slot(table, pages, page_size, b, past + j)
            if at is None:
                continue
            half = 0 if rope is None else rope.shape[1] // 2
            turned = k[b, j] if half == 0 else rotate32(k[b, j], rope[pos, :half], rope[pos, half:], interleaved)
            for x, c, s in ((turned, got[0], got[2]), (v[b, j], got[1], got[3])):
                c[at[0], :, at[1]], s[at[0], :, at[1]] = quantise(x, kind)
    return got


def read(codes, scales, kind, first, count, n, table=None):
    """Rows read back in float64 [batch, n, heads, dh], 0 where there is none."""
    pages, heads, page_size, dh = codes.shape
    out = np.zeros((len(first), n, heads, dh))
    for b in range(len(first)):
        m = n if count is None else min(int(count[b]), n)
        for i in range(m):
            at = O.slot(table, pages, page_size, b, int(first[b]) + i)
            if at is not None:
                out[b, i] = values(codes[at[0], :, at[1]], scales[at[0], :, at[1]], kind)
    return out
