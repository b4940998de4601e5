"""Tensor-level helpers of the operators around the projections of a decode step: the 4-bit base
projection (``linear_w4``), the rotation and cache append (``rope_append``) and the attention over
a shared prefix (``prefix_attention``). As in ``ops``: marshalling only, the work is the library's.
The calls run on the device of their operands (all on one) and its current stream. They compute no
gradients.
"""

from __future__ import annotations

from dataclasses import dataclass

import torch

from . import _lib, ops

_HALF = (torch.bfloat16, torch.float16)


def _place(first, *rest) -> int:
    """The index of the one device of all operands."""
    dev = first.get_device()
    for t in rest:
        if t is not None and t.get_device() != dev:
            raise ValueError("all tensors must be on one GPU")
    if dev < 0:
        raise ValueError("all tensors must be on the GPU")
    return dev


def _launch(name: str, dev: int, *args) -> None:
    """Calls the entry point ``name`` on device ``dev`` and its current stream (the last argument).
    Small calls are bound by this path, so the stream and the current device are taken without
    wrapper objects."""
    fn = getattr(_lib.lib(), name)
    stream = torch._C._cuda_getCurrentRawStream(dev)
    if torch._C._cuda_getDevice() == dev:
        st = fn(*args, stream)
    else:
        with torch.cuda.device(dev):
            st = fn(*args, stream)
    if st != _lib.LORA_OK:
        raise _lib.LoraError(name, st)


def _ptr(t) -> int | None:
    return None if t is None else t.data_ptr()


def _pitch(t: torch.Tensor, name: str) -> int:
    """Row pitch of a matrix whose rows are contiguous (the pitch of a single row does not matter)."""
    if t.dim() != 2:
        raise ValueError(f"{name} must be a 2-D tensor")
    rows, cols = t.shape
    ld, unit = t.stride()
    if unit != 1 and cols > 1:
        raise ValueError(f"{name} must have a unit column stride")
    return ld if rows > 1 else cols


def _half(t: torch.Tensor, name: str) -> int:
    if t.dtype not in _HALF:
        raise TypeError(f"{name} must be bf16 or fp16")
    return ops.dtype_code(t)


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
    dev = _place(codes, scales, zero_points)
    if codes.dtype != torch.uint8 or (zero_points is not None and zero_points.dtype != torch.uint8):
        raise ValueError("codes and zero_points must be uint8")
    ldc, lds = _pitch(codes, "codes"), _pitch(scales, "scales")
    N, K = codes.shape[0], 2 * codes.shape[1]
    groups = scales.shape[1]
    if scales.shape[0] != N or groups == 0 or K % groups != 0:
        raise ValueError("scales must be [N][K / group]")
    if zero_points is not None and zero_points.shape != scales.shape:
        raise ValueError("zero_points must have the shape of scales")
    ldz = 0 if zero_points is None else _pitch(zero_points, "zero_points")
    dt, group = _half(scales, "scales"), K // groups
    nbytes = _lib.lora_linear_w4_prepared_size(dt, K, N, group, zero_points is not None)
    if nbytes == 0:
        raise ValueError(f"unsupported weight: K {K}, N {N}, group {group} (32, 64 or 128)")
    data = codes.new_empty(nbytes)
    _launch("lora_linear_w4_prepare", dev, dt, K, N, group, codes.data_ptr(), ldc, scales.data_ptr(), lds,
            _ptr(zero_points), ldz, data.data_ptr(), nbytes)
    return W4Weight(data, scales.dtype, K, N, group, zero_points is not None)


def linear_w4(x, w: W4Weight, out: torch.Tensor | None = None) -> torch.Tensor:
    """y = x W^T with a 4-bit weight (``lora_linear_w4``), for few rows of x: the base product of
    a quantised layer, which ``shrink_expand`` then updates. x: [M][K] of the weight's dtype;
    returns [M][N]."""
    dev = _place(x, w.data, out)
    if x.dtype != w.dtype:
        raise TypeError(f"x must have the dtype {w.dtype} of the weight's scales")
    ldx = _pitch(x, "x")
    M, K = x.shape
    if K != w.K:
        raise ValueError(f"x must be [M][{w.K}]")
    if out is None:
        out, ldy = x.new_empty((M, w.N)), w.N
    else:
        ops._out(out, (M, w.N), x.dtype, x.device, "out")
        ldy = _pitch(out, "out")
    _launch("lora_linear_w4", dev, ops._DT[x.dtype], M, K, w.N, w.group, w.zero_points, x.data_ptr(), ldx,
            w.data.data_ptr(), out.data_ptr(), ldy)
    return out


def _cache(k_cache, v_cache, ref) -> tuple[int, int, int, int, int, int, int]:
    """(pages, page size, heads, head size, page, token and head strides) of a pair of caches."""
    if k_cache.dim() != 4 or k_cache.shape != v_cache.shape:
        raise ValueError("k_cache and v_cache must be [pages][page size][heads][D], of one shape")
    if k_cache.dtype != ref.dtype or v_cache.dtype != ref.dtype:
        raise TypeError(f"the caches must have the dtype {ref.dtype}")
    shape, stride = k_cache.shape, k_cache.stride()
    if stride != v_cache.stride():
        raise ValueError("k_cache and v_cache must have the same strides")
    pages, page, heads, D = shape
    if stride[3] != 1 and D > 1:
        raise ValueError("the caches must have a unit stride along D")
    # a stride of an extent of one place is never used
    return (pages, page, heads, D, stride[0] if pages > 1 else 0, stride[1] if page > 1 else 0,
            stride[2] if heads > 1 else 0)


def rope_append(q, k, v, table, positions, slots, k_cache, v_cache, q_norm=None, k_norm=None,
                eps: float = 1e-6, interleaved: bool = False,
                q_out: torch.Tensor | None = None) -> torch.Tensor:
    """Rotates q and k (after an optional norm of each head) and appends k and v to a paged cache
    (``lora_rope_append``). q: [T][Hq*D], k, v: [T][Hkv*D] (column views of one projection do);
    table: float32 [rows][rot], rot / 2 cosines then rot / 2 sines a row; positions: int32 [T], rows of
    the table; slots: int64 [T], place page * page_size + offset, -1: not appended; caches
    [pages][page_size][Hkv][D], written in place; q_norm, k_norm: [D]. Pairs are (p, p + rot / 2), or
    (2p, 2p + 1) when interleaved. Returns the rotated q [T][Hq*D] (q_out, which may be q)."""
    dev = _place(q, k, v, table, positions, slots, k_cache, v_cache, q_norm, k_norm, q_out)
    pages, page, Hkv, D, ps, ts, hs = _cache(k_cache, v_cache, q)
    ldq, ldk, ldv = _pitch(q, "q"), _pitch(k, "k"), _pitch(v, "v")
    T, nq = q.shape
    if D == 0 or nq % D != 0:
        raise ValueError("q must be [T][Hq * D]")
    nkv = (T, Hkv * D)
    if k.shape != nkv or v.shape != nkv:
        raise ValueError(f"k and v must be [T][{Hkv * D}]")
    if k.dtype != q.dtype or v.dtype != q.dtype:
        raise TypeError(f"k and v must have the dtype {q.dtype}")
    for t, name in ((q_norm, "q_norm"), (k_norm, "k_norm")):
        if t is not None and (t.dtype != q.dtype or t.shape != (D,) or not t.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous {q.dtype} vector of {D}")
    if table.dtype != torch.float32 or table.dim() != 2 or not table.is_contiguous():
        raise ValueError("table must be a contiguous float32 [rows][rot]")
    if positions.dtype != torch.int32 or positions.shape != (T,) or not positions.is_contiguous():
        raise ValueError(f"positions must be a contiguous int32 vector of {T}")
    if slots.dtype != torch.int64 or slots.shape != (T,) or not slots.is_contiguous():
        raise ValueError(f"slots must be a contiguous int64 vector of {T}")
    dt = ops.dtype_code(q)
    if q_out is None:
        q_out, ldqo = q.new_empty((T, nq)), nq
    else:
        ops._out(q_out, q.shape, q.dtype, q.device, "q_out")
        ldqo = _pitch(q_out, "q_out")
    rows, rot = table.shape
    _launch("lora_rope_append", dev, dt, T, nq // D, Hkv, D, rot, interleaved, pages, page, rows, q.data_ptr(),
            ldq, k.data_ptr(), ldk, v.data_ptr(), ldv, table.data_ptr(), positions.data_ptr(),
            slots.data_ptr(), _ptr(q_norm), _ptr(k_norm), eps, q_out.data_ptr(), ldqo, k_cache.data_ptr(),
            v_cache.data_ptr(), ps, ts, hs)
    return q_out


def _page_list(pages, lens, n: int, name: str) -> int:
    """Width of a page list (0 for None)."""
    if pages is None:
        if lens is not None:
            raise ValueError(f"{name}_lens without {name}_pages")
        return 0
    if pages.dtype != torch.int32 or pages.dim() != 2 or not pages.is_contiguous() or pages.shape[0] != n:
        raise ValueError(f"{name}_pages must be a contiguous int32 [{n}][width]")
    if lens is None:
        raise ValueError(f"{name}_pages without {name}_lens")
    ops._meta(lens, n, f"{name}_lens")
    return pages.shape[1]


def prefix_attention_workspace(q, k_cache, seg_indptr, prefix_pages, own_pages) -> torch.Tensor:
    """A workspace for ``prefix_attention`` on operands of these shapes (for calls that do not overlap
    in time)."""
    _place(q, k_cache, seg_indptr, prefix_pages, own_pages)
    _, page, Hkv, D = k_cache.shape
    nbytes = _lib.lora_prefix_attention_workspace_size(
        _half(q, "q"), q.shape[0], seg_indptr.numel() - 1, q.shape[1] // D, Hkv, D, page,
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
    workspace: from ``prefix_attention_workspace`` (a fresh one otherwise)."""
    dev = _place(q, k_cache, v_cache, seg_indptr, permutation, prefix_pages, prefix_lens, own_pages,
                 own_lens, out, workspace)
    dt = _half(q, "q")
    pages, page, Hkv, D, ps, ts, hs = _cache(k_cache, v_cache, q)
    ldq = _pitch(q, "q")
    T, nq = q.shape
    if D == 0 or nq % D != 0:
        raise ValueError("q must be [T][Hq * D]")
    Hq = nq // D
    ops._meta(seg_indptr, None, "seg_indptr")
    G = seg_indptr.numel() - 1
    if G < 0:
        raise ValueError("seg_indptr must have at least one entry")
    if permutation is not None:
        ops._meta(permutation, T, "permutation")
    wp = _page_list(prefix_pages, prefix_lens, G, "prefix")
    wo = _page_list(own_pages, own_lens, T, "own")
    if out is None:
        out, ldo = q.new_empty((T, nq)), nq
    else:
        ops._out(out, q.shape, q.dtype, q.device, "out")
        ldo = _pitch(out, "out")
    lse = q.new_empty((T, Hq), dtype=torch.float32) if return_lse else None
    if workspace is None:
        nbytes = _lib.lora_prefix_attention_workspace_size(dt, T, G, Hq, Hkv, D, page, wp, wo)
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=q.device)
    elif workspace.dtype != torch.uint8 or workspace.dim() != 1 or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous uint8 vector")
    _launch("lora_prefix_attention", dev, dt, T, G, Hq, Hkv, D, pages, page, q.data_ptr(), ldq,
            k_cache.data_ptr(), v_cache.data_ptr(), ps, ts, hs, seg_indptr.data_ptr(), _ptr(permutation),
            _ptr(prefix_pages), wp, _ptr(prefix_lens), _ptr(own_pages), wo, _ptr(own_lens), scale,
            out.data_ptr(), ldo, _ptr(lse), workspace.data_ptr(), workspace.numel())
    return (out, lse) if return_lse else out
