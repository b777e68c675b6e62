"""Float64 definitions of the serving operators around the attention calls (test infrastructure):
rotary positions, and where and as what the cache append writes new tokens."""
from __future__ import annotations

from decimal import Decimal, getcontext

import numpy as np

from .attention import e4m3_to_f64

getcontext().prec = 60
_TWO_PI = Decimal("6.28318530717958647692528676655900576839433879875021164194988918461563281257")


def angles(positions, inv_freq) -> np.ndarray:
    """position * inv_freq reduced to [0, 2 pi) in 60-digit decimal arithmetic, then float64."""
    out = np.empty((len(positions), len(inv_freq)))
    freq = [Decimal(float(f)) for f in inv_freq]
    for i, p in enumerate(positions):
        for j, f in enumerate(freq):
            out[i, j] = float((Decimal(int(p)) * f) % _TWO_PI)
    return out


def pair_columns(layout: str, dim: int):
    """Columns (a, b) of every pair of a head's first ``dim`` values."""
    i = np.arange(dim // 2)
    return (2 * i, 2 * i + 1) if layout == "interleaved" else (i, i + dim // 2)


def rotate(x, positions, inv_freq, layout: str, mscale: float = 1.0, inverse: bool = False) -> np.ndarray:
    """x [T, H, D] with pair p of row t turned by positions[t] * inv_freq[p] (by its negative: inverse)."""
    out = np.array(x, dtype=np.float64)
    a, b = pair_columns(layout, 2 * len(inv_freq))
    t = angles(positions, inv_freq)[:, None, :] * (-1.0 if inverse else 1.0)
    xa, xb = out[..., a].copy(), out[..., b].copy()
    out[..., a] = mscale * (xa * np.cos(t) - xb * np.sin(t))
    out[..., b] = mscale * (xa * np.sin(t) + xb * np.cos(t))
    return out


def decode(codes, dtype: str) -> np.ndarray:
    """Values of 8-bit codes (uint8 bytes) before their scale."""
    codes = np.asarray(codes, dtype=np.uint8)
    return e4m3_to_f64(codes) if dtype == "e4m3" else codes.view(np.int8).astype(np.float64)


def append_rows(append_indptr, kv_indptr, kv_indices, last, page_size: int):
    """(request, position, page, slot) of every new row; the page table is the one after the append."""
    out = []
    for r in range(len(kv_indptr) - 1):
        n_pages = int(kv_indptr[r + 1] - kv_indptr[r])
        length = (n_pages - 1) * page_size + int(last[r]) if n_pages else 0
        n = int(append_indptr[r + 1] - append_indptr[r])
        for i in range(n):
            pos = length - n + i
            out.append((r, pos, int(kv_indices[kv_indptr[r] + pos // page_size]), pos % page_size))
    return out


def append_blocks(x, values, scales, rows, block: int, qmax: float):
    """Block-scaled append of rows x [T, Hk, D] into a cache of real values [pages, P, Hk, D] with
    scales [pages, P / block, Hk]: the new scales, and the values the cache would hold without
    rounding.  ``rows``: append_rows; a block whose first slot is new starts from scale 0."""
    values, scales = values.copy(), scales.copy()
    groups = {}
    for t, (r, pos, page, slot) in enumerate(rows):
        groups.setdefault((page, slot // block), []).append((t, slot))
    for (page, b), members in groups.items():
        first = min(slot for _, slot in members)
        idx = [t for t, _ in members]
        want = np.abs(x[idx]).max(axis=(0, 2)) / qmax
        if first % block:
            want = np.maximum(want, scales[page, b])
        scales[page, b] = want
        for t, slot in members:
            values[page, slot] = x[t]
    return values, scales
