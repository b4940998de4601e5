"""Tensor-level helpers of the operators around the projections of a decode step: the 4-bit base
projection (``linear_w4``), the rotation and cache append (``rope_append``) and the attention over
a shared prefix (``prefix_attention``). The checks and the marshalling are native
(``csrc/binding.cpp``), as small calls are bound by them; wrong shapes, strides and devices raise
ValueError, wrong dtypes TypeError, and what the library refuses LoraError. The calls run on the
device of their operands (all on one) and its current stream. They compute no gradients.
"""

from __future__ import annotations

from dataclasses import dataclass

import torch

from . import _lib, ops

_native = None


def _load():
    """The native module. There is no fallback: without it every call raises."""
    global _native
    _lib.lib()  # says what to do if nothing is built
    from . import _binding

    _native = _binding
    return _binding


def _result(fn: str, r):
    if type(r) is int:
        raise _lib.LoraError(fn, r)
    return r


@dataclass(frozen=True)
class W4Weight:
    """A 4-bit weight as ``linear_w4`` reads it (from ``linear_w4_prepare``)."""

    data: torch.Tensor  # uint8, the library's layout
    dtype: torch.dtype  # of the scales, and so of x and y
    K: int
    N: int
    group: int
    zero_points: bool


def linear_w4_prepare(codes, scales, zero_points=None) -> W4Weight:
    """The weight W[n][k] = scales[n][k / group] (c[n][k] - z) in the layout the product reads
    (``lora_linear_w4_prepare``), once per layer. codes: uint8 [N][K/2], the code of an even k in the
    low half of its byte; scales: [N][K/group] bf16 or fp16, group 32, 64 or 128; zero_points: uint8
    [N][K/group] in 0..15, or None for 8 everywhere."""
    ops._dev(codes, scales, zero_points)
    if codes.dtype != torch.uint8 or (zero_points is not None and zero_points.dtype != torch.uint8):
        raise ValueError("codes and zero_points must be uint8")
    ldc, lds = ops._rows(codes, "codes"), ops._rows(scales, "scales")
    if scales.dtype not in (torch.bfloat16, torch.float16):
        raise TypeError("scales must be bf16 or fp16")
    N, K = codes.shape[0], 2 * codes.shape[1]
    groups = scales.shape[1]
    if scales.shape[0] != N or groups == 0 or K % groups != 0:
        raise ValueError("scales must be [N][K / group]")
    if zero_points is not None and zero_points.shape != scales.shape:
        raise ValueError("zero_points must have the shape of scales")
    if any(t is not None and t.device != codes.device for t in (scales, zero_points)):
        raise ValueError("all tensors must be on one GPU")
    ldz = 0 if zero_points is None else ops._rows(zero_points, "zero_points")
    dt, group = ops.dtype_code(scales), K // groups
    nbytes = _lib.lora_linear_w4_prepared_size(dt, K, N, group, zero_points is not None)
    if nbytes == 0:
        raise ValueError(f"unsupported weight: K {K}, N {N}, group {group} (32, 64 or 128)")
    with torch.cuda.device(codes.device):
        data = codes.new_empty(nbytes)
        _lib.lora_linear_w4_prepare(dt, K, N, group, codes, ldc, scales, lds, zero_points, ldz, data,
                                    nbytes, ops._stream())
    return W4Weight(data, scales.dtype, K, N, group, zero_points is not None)


def linear_w4(x, w: W4Weight, out: torch.Tensor | None = None) -> torch.Tensor:
    """y = x W^T with a 4-bit weight (``lora_linear_w4``), for few rows of x: the base product of
    a quantised layer, which ``shrink_expand`` then updates. x: [M][K] of the weight's dtype;
    returns [M][N] (out, which must not overlap x)."""
    return _result("lora_linear_w4", (_native or _load()).linear_w4(
        x, w.data, ops._DT[w.dtype], w.K, w.N, w.group, w.zero_points, out))


def rope_append(q, k, v, table, positions, slots, k_cache, v_cache, q_norm=None, k_norm=None,
                eps: float = 1e-6, interleaved: bool = False,
                q_out: torch.Tensor | None = None) -> torch.Tensor:
    """Rotates q and k (after an optional norm of each head) and appends k and v to a paged cache
    (``lora_rope_append``). q: [T][Hq*D], k, v: [T][Hkv*D] (column views of one projection do);
    table: float32 [rows][rot], rot / 2 cosines then rot / 2 sines a row; positions: int32 [T], rows of
    the table; slots: int64 [T], place page * page_size + offset, -1: not appended; caches
    [pages][page_size][Hkv][D], written in place; q_norm, k_norm: [D]. Pairs are (p, p + rot / 2), or
    (2p, 2p + 1) when interleaved. Returns the rotated q [T][Hq*D] (q_out, which may be q and
    must not overlap it otherwise)."""
    return _result("lora_rope_append", (_native or _load()).rope_append(
        q, k, v, table, positions, slots, k_cache, v_cache, q_norm, k_norm, eps, interleaved, q_out))


def prefix_attention_workspace(q, k_cache, seg_indptr, prefix_pages, own_pages) -> torch.Tensor:
    """A workspace for ``prefix_attention`` on operands of these shapes (for calls that do not overlap
    in time)."""
    ops._dev(q, k_cache)
    _, page, Hkv, D = k_cache.shape
    nbytes = _lib.lora_prefix_attention_workspace_size(
        ops.dtype_code(q), q.shape[0], seg_indptr.numel() - 1, q.shape[1] // D, Hkv, D, page,
        0 if prefix_pages is None else prefix_pages.shape[1],
        0 if own_pages is None else own_pages.shape[1])
    return torch.empty(nbytes, dtype=torch.uint8, device=q.device)


def prefix_attention(q, k_cache, v_cache, seg_indptr, permutation, prefix_pages, prefix_lens,
                     own_pages, own_lens, scale: float, out: torch.Tensor | None = None,
                     return_lse: bool = False, workspace: torch.Tensor | None = None):
    """Attention of one query token per row over a paged cache, where a segment's tokens share a
    prefix (``lora_prefix_attention``). q: [T][Hq*D] in token order; caches [pages][page_size][Hkv][D];
    seg_indptr, permutation (None: identity) as for ``shrink``; prefix_pages int32 [G][width] and
    prefix_lens int32 [G] (None: no prefix); own_pages int32 [T][width] and own_lens int32 [T]: the
    keys of each token after the prefix. Returns out [T][Hq*D], with return_lse also the natural
    logarithm of the softmax sums, float32 [T][Hq]; rows no segment covers are not written.
    out must not overlap q. workspace: from ``prefix_attention_workspace`` (a fresh one otherwise)."""
    return _result("lora_prefix_attention", (_native or _load()).prefix_attention(
        q, k_cache, v_cache, seg_indptr, permutation, prefix_pages, prefix_lens, own_pages, own_lens,
        scale, out, return_lse, workspace))
