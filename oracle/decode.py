"""fp64 oracle of the operators around the projections of a decode step.

Test infrastructure only (see the package docstring). Each function is the definition written
out, one token, head or row at a time, and returns fp64 values that are not rounded to a storage
type unless it says so.
"""

from __future__ import annotations

import numpy as np

from .embedding import _f64, _i64


def w4_weight(codes, scales, zero_points=None) -> np.ndarray:
    """W [N][K] of 4-bit codes (uint8 [N][K/2], even k in the low half), scales [N][K/group] and zero
    points (None: 8): W = scale * (code - zero point)."""
    c = _i64(codes)
    N, half = c.shape
    q = np.empty((N, 2 * half), dtype=np.float64)
    q[:, 0::2], q[:, 1::2] = c & 15, c >> 4
    s = _f64(scales)
    g = 2 * half // s.shape[1]
    z = np.full(s.shape, 8.0) if zero_points is None else _f64(_i64(zero_points) & 15)
    return (q - np.repeat(z, g, axis=1)) * np.repeat(s, g, axis=1)


def linear_w4(x, codes, scales, zero_points=None) -> np.ndarray:
    """y = x W^T."""
    return _f64(x) @ w4_weight(codes, scales, zero_points).T


def rope_head(x, cos, sin, w=None, eps: float = 1e-6, interleaved: bool = False) -> np.ndarray:
    """One head x [D]: the norm (w not None), then the rotation of its first 2 * len(cos) elements."""
    u = _f64(x).copy()
    if w is not None:
        u = u * _f64(w) / np.sqrt(np.mean(u * u) + eps)
    half = len(cos)
    out = u.copy()
    for p in range(half):
        a, b = (2 * p, 2 * p + 1) if interleaved else (p, p + half)
        out[a] = u[a] * cos[p] - u[b] * sin[p]
        out[b] = u[b] * cos[p] + u[a] * sin[p]
    return out


def rope_append(q, k, v, table, positions, slots, k_cache, v_cache, q_norm=None, k_norm=None,
                eps: float = 1e-6, interleaved: bool = False):
    """(q_out [T][Hq*D], k_cache, v_cache) after the append; rows left out are NaN in q_out and keep
    the caches' values. The caches are [pages][page size][Hkv][D]."""
    q, k, v, table = _f64(q), _f64(k), _f64(v), _f64(table)
    pos, slots = _i64(positions), _i64(slots)
    kc, vc = _f64(k_cache).copy(), _f64(v_cache).copy()
    pages, page, Hkv, D = kc.shape
    T, Hq, half = q.shape[0], q.shape[1] // D, table.shape[1] // 2
    q_out = np.full(q.shape, np.nan)
    for t in range(T):
        if not 0 <= pos[t] < table.shape[0]:
            continue
        cos, sin = table[pos[t], :half], table[pos[t], half:]
        for h in range(Hq):
            c = slice(h * D, h * D + D)
            q_out[t, c] = rope_head(q[t, c], cos, sin, q_norm, eps, interleaved)
        if not 0 <= slots[t] < pages * page:
            continue
        pg, place = divmod(int(slots[t]), page)
        for h in range(Hkv):
            c = slice(h * D, h * D + D)
            kc[pg, place, h] = rope_head(k[t, c], cos, sin, k_norm, eps, interleaved)
            vc[pg, place, h] = v[t, c]
    return q_out, kc, vc


def _places(pages, length: int, page: int, num_pages: int):
    """(page, offset) of the visible places of a list: those whose page id lies in the cache."""
    out = []
    length = min(max(int(length), 0), len(pages) * page)
    for j in range(length):
        pid = int(pages[j // page])
        if 0 <= pid < num_pages:
            out.append((pid, j % page))
    return out


def prefix_attention(q, k_cache, v_cache, seg_indptr, permutation, prefix_pages, prefix_lens,
                     own_pages, own_lens, scale: float):
    """(out [T][Hq*D], lse [T][Hq], spread [T][Hq*D]); rows no segment covers are NaN. spread is
    sum_j p_j |v_j|, the magnitude that roundings of the weights p act on."""
    q, kc, vc = _f64(q), _f64(k_cache), _f64(v_cache)
    num_pages, page, Hkv, D = kc.shape
    T, Hq = q.shape[0], q.shape[1] // D
    indptr = _i64(seg_indptr)
    perm = np.arange(T) if permutation is None else _i64(permutation)
    out, lse = np.full((T, Hq * D), np.nan), np.full((T, Hq), np.nan)
    spread = np.full((T, Hq * D), np.nan)
    for g in range(len(indptr) - 1):
        shared = [] if prefix_pages is None else _places(_i64(prefix_pages)[g], _i64(prefix_lens)[g], page, num_pages)
        for t in perm[int(indptr[g]):int(indptr[g + 1])]:
            mine = [] if own_pages is None else _places(_i64(own_pages)[t], _i64(own_lens)[t], page, num_pages)
            at = shared + mine
            if not at:
                out[t], lse[t], spread[t] = 0.0, -np.inf, 0.0
                continue
            pg, pl = np.array(at).T
            for h in range(Hq):
                c = slice(h * D, h * D + D)
                kh, vh = kc[pg, pl, h // (Hq // Hkv)], vc[pg, pl, h // (Hq // Hkv)]
                s = scale * (kh @ q[t, c])
                e = np.exp(s - s.max())
                out[t, c] = (e @ vh) / e.sum()
                spread[t, c] = (e @ np.abs(vh)) / e.sum()
                lse[t, h] = s.max() + np.log(e.sum())
    return out, lse, spread
