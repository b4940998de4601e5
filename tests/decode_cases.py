"""Seeded inputs and derived tolerances of the decode-step operators' tests.

Tolerances. u is the unit roundoff of the storage type (2^-8 bf16, 2^-11 fp16, 2^-24 fp32) and e the
one of fp32 (2^-24); every bound is a worst case over the roundings, none is fitted.

* linear_w4: products of 16-bit values are exact in fp32. A group of g codes is two sums of at
  most g terms, of magnitude s |x| (16 + c) <= 31 s |x| and s |x| (16 + z) <= 31 s |x|, then one
  multiplication and addition each; the groups and the 8 waves are added in turn. Each addition
  rounds by at most e times the magnitude summed so far, so with A = sum_k s |x_k|
      |y - exact| <= u |exact| + (g + K / g + 16) e 62 A.
* rope_append: r = 1 / sqrt(mean + eps) carries at most (D + 16) e (the sum of D squares, the
  division, the root), each rotated element two products and a sum of fp32 values; with |u_a|, |u_b|
  the pair's magnitudes |out - exact| <= u |exact| + (D + 24) e (|u_a| + |u_b|).
* prefix_attention: the score of a key is off by at most (D + 4) e S, S the largest
  scale sum_d |q_d| |k_d|, so its weight by that factor, the exponential's own error and the
  subtraction's (under 16 e + 4 e S) included; the weight is then rounded by u (fp16: or by 2^-25
  below 2^-14, where the largest weight is 1). The same weights stand in the sum, so with
  w = sum_j p_j |v_j| and d = u + ((2 D + 32) S + n + 64) e, n keys (n e: the additions),
      |out - exact| <= u |exact| + 2 d w + f n max|v|,   f = 2^-24 (fp16) or 0,
      |lse - exact| <= d + f n + 8 e (1 + |exact|).
"""

from __future__ import annotations

import numpy as np
import torch

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
U = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}
E = 2.0 ** -24


def f64(t) -> np.ndarray:
    return t.detach().cpu().double().numpy()


def normal(g, shape, dtype, std=1.0):
    return (torch.randn(shape, generator=g) * std).to(DT[dtype])


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def within(got, ref, tol, what):
    """|got - ref| <= tol, NaN exactly where ref has NaN."""
    got, ref = np.asarray(got), np.asarray(ref)
    bad = ~(np.abs(got - ref) <= tol) & ~(np.isnan(got) & np.isnan(ref)) & ~(got == ref)
    if bad.any():
        at = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} outside the bound; first at {at}: "
                             f"{got[at]} against {ref[at]}, bound {np.broadcast_to(tol, ref.shape)[at]}")


def w4_inputs(seed, dtype, M, K, N, group, zeros):
    g = gen(seed)
    codes = torch.randint(0, 256, (N, K // 2), generator=g, dtype=torch.uint8)
    scales = ((0.5 + torch.rand((N, K // group), generator=g)) * 0.05).to(DT[dtype])
    zp = torch.randint(0, 16, (N, K // group), generator=g, dtype=torch.uint8) if zeros else None
    return normal(g, (M, K), dtype), codes, scales, zp


def w4_bound(dtype, x, scales, ref, group):
    K = x.shape[1]
    a = np.abs(f64(x)) @ np.repeat(f64(scales), group, axis=1).T
    return U[dtype] * np.abs(ref) + (group + K / group + 16) * E * 62 * a


def table(rows, rot, base=1e4):
    inv = base ** (-np.arange(0, rot, 2) / rot)
    ang = np.arange(rows)[:, None] * inv
    return torch.from_numpy(np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32))


def rope_bound(dtype, ref, D, rot, interleaved):
    """ref [..., D]: the rotation keeps a pair's norm, so |u_a| + |u_b| <= sqrt(2) times it."""
    r = np.abs(ref)
    mag = r.copy()
    half = rot // 2
    p = np.arange(half)
    a, b = (2 * p, 2 * p + 1) if interleaved else (p, p + half)
    pair = np.sqrt(2.0) * np.hypot(r[..., a], r[..., b])
    mag[..., a], mag[..., b] = pair, pair
    return U[dtype] * r + (D + 24) * E * mag


class Attn:
    """Inputs of one prefix_attention call (CPU tensors). Every place that no list names within its
    length holds NaN; list entries beyond a length are wild."""

    def __init__(self, seed, dtype, T, lens_seg, Hq, Hkv, D, page, prefix_lens, own_lens,
                 indptr0=0, layout="phd", perm=True, std=1.0, extra_pages=3, q_pad=0):
        g = gen(seed)
        rng = np.random.default_rng(seed)
        G = len(lens_seg)
        self.dtype, self.T, self.G, self.Hq, self.Hkv, self.D, self.page = dtype, T, G, Hq, Hkv, D, page
        need = lambda n: (max(n, 0) + page - 1) // page
        wp, wo = max([1] + [need(n) for n in prefix_lens]), max([1] + [need(n) for n in own_lens])
        total = sum(map(need, prefix_lens)) + sum(map(need, own_lens)) + extra_pages
        ids = rng.permutation(total)
        at = 0
        wild = lambda shape: rng.integers(-2 ** 31, 2 ** 31 - 1, size=shape).astype(np.int32)
        self.prefix_pages, self.own_pages = wild((G, wp)), wild((T, wo))
        used = np.zeros((total, page), dtype=bool)
        for lists, lens in ((self.prefix_pages, prefix_lens), (self.own_pages, own_lens)):
            for row, n in zip(lists, lens):
                row[:need(n)] = ids[at:at + need(n)]
                for j in range(max(n, 0)):
                    used[row[j // page], j % page] = True
                at += need(n)
        i32 = lambda a: torch.from_numpy(np.ascontiguousarray(np.asarray(a, dtype=np.int32)))
        self.prefix_pages, self.own_pages = i32(self.prefix_pages), i32(self.own_pages)
        self.prefix_lens, self.own_lens = i32(prefix_lens), i32(own_lens)
        self.indptr = i32(np.concatenate([[indptr0], indptr0 + np.cumsum(lens_seg)]))
        self.perm = i32(rng.permutation(T)) if perm else None
        q = normal(g, (T, Hq * D + q_pad), dtype, std)
        self.q = q[:, :Hq * D]
        shape = (total, page, Hkv, D) if layout == "phd" else (total, Hkv, page, D)
        self.k, self.v = normal(g, shape, dtype, std), normal(g, shape, dtype)
        if layout != "phd":
            self.k, self.v = self.k.permute(0, 2, 1, 3), self.v.permute(0, 2, 1, 3)
        hole = torch.from_numpy(~used)
        self.k[hole] = float("nan")
        self.v[hole] = float("inf")
        self.scale = D ** -0.5

    def args(self, to=lambda t: t):
        m = lambda t: None if t is None else to(t)
        return (m(self.q), m(self.k), m(self.v), m(self.indptr), m(self.perm), m(self.prefix_pages),
                m(self.prefix_lens), m(self.own_pages), m(self.own_lens), self.scale)

    def bounds(self, ref, lse, spread):
        u, f = U[self.dtype], 2.0 ** -24 if self.dtype == "f16" else 0.0
        k = np.nan_to_num(f64(self.k))
        S = self.scale * np.linalg.norm(f64(self.q).reshape(self.T, self.Hq, self.D), axis=2).max() * \
            np.linalg.norm(k, axis=3).max()
        n = (self.prefix_pages.shape[1] + self.own_pages.shape[1]) * self.page
        d = u + ((2 * self.D + 32) * S + n + 64) * E
        v = f64(self.v)
        vmax = np.abs(v[np.isfinite(v)]).max() if np.isfinite(v).any() else 0.0
        return (u * np.abs(ref) + 2 * d * spread + f * n * vmax,
                d + f * n + 8 * E * (1 + np.abs(lse)))
