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


def attend(q, k, v, limits, sm_scale: float):
    """One KV head's rows q [R, D] over keys k [L, D], values v [L, D]; row i sees the first limits[i] keys.
    Returns O, LSE, sum_t p_t |v_t| (what rounding the weights acts on) and max_t sm_scale |q| . |k_t|."""
    if not len(k):
        z = np.zeros_like(q)
        return z, np.full(len(q), -np.inf), z.copy(), np.zeros(len(q))
    s = sm_scale * (q @ k.T)
    s[np.arange(len(k))[None, :] >= np.asarray(limits)[:, None]] = -np.inf
    m = s.max(axis=1)
    base = np.where(np.isneginf(m), 0.0, m)
    p = np.exp(s - base[:, None])
    l = p.sum(axis=1)
    p /= np.where(l > 0, l, 1.0)[:, None]
    with np.errstate(divide="ignore"):
        lse = np.where(l > 0, base + np.log(l), -np.inf)
    return p @ v, lse, p @ np.abs(v), sm_scale * (np.abs(q) @ np.abs(k).T).max(axis=1)


def packed_attention(q, k_of, v_of, qo_indptr, lengths, hk: int, causal: bool, sm_scale: float, requests=None):
    """Attention of packed queries q [T, Hq, D]; k_of(r) / v_of(r) give request r's keys [L_r, Hk, D].  With
    ``causal`` the n query tokens of a request are its last n positions.  Returns O, LSE, weight scale
    and score scale of ``attend`` for every row (NaN where a request is not asked for)."""
    T, hq, d = q.shape
    g = hq // hk
    o, a = np.full((T, hq, d), np.nan), np.full((T, hq, d), np.nan)
    lse, mag = np.full((T, hq), np.nan), np.full((T, hq), np.nan)
    for r in range(len(lengths)) if requests is None else requests:
        q0, q1, L = int(qo_indptr[r]), int(qo_indptr[r + 1]), int(lengths[r])
        if q1 == q0:
            continue
        k, v, n = k_of(r), v_of(r), q1 - q0
        limits = L - n + 1 + np.arange(n) if causal else np.full(n, L)
        for h in range(hq):
            o[q0:q1, h], lse[q0:q1, h], a[q0:q1, h], mag[q0:q1, h] = attend(q[q0:q1, h], k[:, h // g], v[:, h // g],
                                                                            limits, sm_scale)
    return o, lse, a, mag
