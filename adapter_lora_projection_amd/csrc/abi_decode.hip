// C ABI of the operators around the projections of a decode step: the 4-bit base projection, the
// rotation and cache append, and the attention over a shared prefix. Every check here runs on the
// host before anything is enqueued; nothing reads device memory.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>
#include <utility>

#include "../../include/lora_mi355x.h"
#include "linear_w4.hpp"
#include "prefix_attention.hpp"
#include "rope_append.hpp"

namespace {

bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

lora_status hip_status(hipError_t e) { return e == hipSuccess ? LORA_OK : LORA_EHIP; }

bool is_16bit(int d) { return d == LORA_BF16 || d == LORA_F16; }

// Whether places of a cache with these element strides can share elements: sorted by stride, each
// stride has to cover the extents below it.
bool places_overlap(int64_t pages, int64_t ps, int64_t page, int64_t ts, int64_t heads, int64_t hs,
                    int64_t D) {
  int64_t n[3] = {pages, page, heads}, s[3] = {ps, ts, hs};
  for (int i = 0; i < 2; ++i)
    for (int j = i + 1; j < 3; ++j)
      if (s[j] < s[i]) { std::swap(s[i], s[j]); std::swap(n[i], n[j]); }
  __int128 span = D;
  for (int i = 0; i < 3; ++i) {
    if (n[i] <= 1) continue;
    if (s[i] < span) return true;
    span += __int128(s[i]) * (n[i] - 1);
  }
  return false;
}

constexpr int64_t kMaxW4Rows = int64_t(1) << 19;  // 16 rows per workgroup in a 16-bit grid dimension

// Sizes of a 4-bit weight: LORA_OK, or the error of the first one that is wrong.
lora_status w4_sizes(lora_dtype dtype, int64_t K, int64_t N, int32_t group) {
  if (!is_16bit(dtype)) return LORA_EUNSUPPORTED;
  if (K < 1 || N < 1 || group < 1) return LORA_EINVAL;
  if (group != 32 && group != 64 && group != 128) return LORA_EUNSUPPORTED;
  if (K % group != 0) return LORA_EINVAL;
  if (K > (int64_t(1) << 24) || N > (int64_t(1) << 24)) return LORA_EUNSUPPORTED;
  return LORA_OK;
}

}  // namespace

extern "C" {

size_t lora_linear_w4_prepared_size(lora_dtype dtype, int64_t K, int64_t N, int32_t group,
                                    int32_t zero_points) {
  if (w4_sizes(dtype, K, N, group) != LORA_OK) return 0;
  return lmx::w4_layout(K, N, group, zero_points != 0).total;
}

lora_status lora_linear_w4_prepare(lora_dtype dtype, int64_t K, int64_t N, int32_t group,
                                   const uint8_t* codes, int64_t ldc, const void* scales,
                                   int64_t lds, const uint8_t* zero_points, int64_t ldz,
                                   void* prepared, size_t prepared_bytes, void* stream) {
  const lora_status st = w4_sizes(dtype, K, N, group);
  if (st != LORA_OK) return st;
  if (!codes || !scales || !prepared) return LORA_EINVAL;
  if (ldc < K / 2 || lds < K / group || (zero_points && ldz < K / group)) return LORA_EINVAL;
  if (!al16(prepared)) return LORA_EUNSUPPORTED;
  if (prepared_bytes < lmx::w4_layout(K, N, group, zero_points != nullptr).total) return LORA_EWORKSPACE;
  lmx::W4PrepareArgs a{};
  a.codes = codes; a.scales = static_cast<const uint16_t*>(scales); a.zeros = zero_points;
  a.out = static_cast<uint8_t*>(prepared);
  a.ldc = ldc; a.lds = lds; a.ldz = ldz;
  a.K = int(K); a.N = int(N); a.group = group;
  return hip_status(lmx::launch_w4_prepare(a, reinterpret_cast<hipStream_t>(stream)));
}

size_t lora_linear_w4_workspace_size(lora_dtype dtype, int64_t M, int64_t K, int64_t N, int32_t group) {
  if (w4_sizes(dtype, K, N, group) != LORA_OK || M < 1 || M > kMaxW4Rows) return 0;
  return lmx::w4_plan(M, K, N, group).workspace;
}

lora_status lora_linear_w4(lora_dtype dtype, int64_t M, int64_t K, int64_t N, int32_t group,
                           int32_t zero_points, const void* x, int64_t ldx, const void* prepared,
                           void* y, int64_t ldy, void* workspace, size_t workspace_bytes,
                           void* stream) {
  const lora_status st = w4_sizes(dtype, K, N, group);
  if (st != LORA_OK) return st;
  if (M < 0) return LORA_EINVAL;
  if (M > kMaxW4Rows) return LORA_EUNSUPPORTED;
  if (M == 0) return LORA_OK;
  if (!x || !prepared || !y || ldx < K || ldy < N) return LORA_EINVAL;
  if (!al16(x) || ldx % 8 != 0 || !al16(prepared)) return LORA_EUNSUPPORTED;
  const lmx::W4Plan p = lmx::w4_plan(M, K, N, group);
  if (p.workspace > 0 && (workspace == nullptr || workspace_bytes < p.workspace || !al16(workspace)))
    return LORA_EWORKSPACE;
  lmx::W4Args a{};
  a.part = static_cast<float*>(workspace);
  a.x = static_cast<const uint16_t*>(x); a.w = static_cast<const uint8_t*>(prepared);
  a.y = static_cast<uint16_t*>(y);
  a.ldx = ldx; a.ldy = ldy;
  a.M = int(M); a.K = int(K); a.N = int(N); a.group = group;
  return hip_status(lmx::launch_linear_w4(a, p, dtype, zero_points != 0, reinterpret_cast<hipStream_t>(stream)));
}

lora_status lora_rope_append(lora_dtype dtype, int64_t T, int32_t Hq, int32_t Hkv, int32_t D,
                             int32_t rot, int32_t interleaved, int64_t num_pages,
                             int32_t page_size, int64_t table_rows, const void* q, int64_t ldq,
                             const void* k, int64_t ldk, const void* v, int64_t ldv,
                             const float* table, const int32_t* positions, const int64_t* slots,
                             const void* q_norm, const void* k_norm, float eps, void* q_out,
                             int64_t ldqo, void* k_cache, void* v_cache, int64_t page_stride,
                             int64_t token_stride, int64_t head_stride, void* stream) {
  if (dtype != LORA_F32 && !is_16bit(dtype)) return LORA_EUNSUPPORTED;
  if (T < 0 || Hq < 0 || Hkv < 1 || D < 1 || rot < 2 || rot % 2 != 0 || rot > D || num_pages < 0 ||
      page_size < 1 || table_rows < 1)
    return LORA_EINVAL;
  if (!std::isfinite(eps) || eps < 0.f) return LORA_EINVAL;
  if (D > 1024 || Hq > 65536 || Hkv > 65536 || table_rows >= INT_MAX) return LORA_EUNSUPPORTED;
  // up to 64 lanes a head in a launch of less than 2^32 threads; slots are 64-bit
  if (T >= (int64_t(1) << 26) || T * (int64_t(Hq) + 2 * Hkv) >= (int64_t(1) << 26)) return LORA_EUNSUPPORTED;
  if (num_pages > INT64_MAX / page_size) return LORA_EUNSUPPORTED;
  if (T == 0) return LORA_OK;
  if ((Hq > 0 && (!q || !q_out)) || !k || !v || !table || !positions || !slots) return LORA_EINVAL;
  if (num_pages > 0 && (!k_cache || !v_cache)) return LORA_EINVAL;
  if ((Hq > 0 && (ldq < int64_t(Hq) * D || ldqo < int64_t(Hq) * D)) || ldk < int64_t(Hkv) * D ||
      ldv < int64_t(Hkv) * D || page_stride < 0 || token_stride < 0 || head_stride < 0 ||
      places_overlap(num_pages, page_stride, page_size, token_stride, Hkv, head_stride, D))
    return LORA_EINVAL;
  lmx::RopeArgs a{};
  a.q = q; a.k = k; a.v = v; a.table = table; a.positions = positions; a.slots = slots;
  a.q_norm = q_norm; a.k_norm = k_norm; a.q_out = q_out; a.k_cache = k_cache; a.v_cache = v_cache;
  a.ldq = ldq; a.ldk = ldk; a.ldv = ldv; a.ldqo = ldqo;
  a.page_stride = page_stride; a.token_stride = token_stride; a.head_stride = head_stride;
  a.num_slots = num_pages * page_size;
  a.T = int(T); a.Hq = Hq; a.Hkv = Hkv; a.D = D; a.rot = rot; a.page_size = page_size;
  a.table_rows = int(table_rows); a.eps = eps;
  const int64_t ve = dtype == LORA_F32 ? 4 : 8;
  const bool vec = D % 8 == 0 && rot % 16 == 0 && al16(q) && al16(k) && al16(v) && al16(table) &&
                   al16(q_norm) && al16(k_norm) && al16(q_out) && al16(k_cache) && al16(v_cache) &&
                   (Hq == 0 || (ldq % ve == 0 && ldqo % ve == 0)) && ldk % ve == 0 &&
                   ldv % ve == 0 && page_stride % ve == 0 && token_stride % ve == 0 &&
                   head_stride % ve == 0;
  return hip_status(lmx::launch_rope_append(a, dtype, interleaved != 0, vec, reinterpret_cast<hipStream_t>(stream)));
}

}  // extern "C"

namespace {

// Sizes of the attention: LORA_OK, or the error of the first one that is wrong.
lora_status attn_sizes(lora_dtype dtype, int64_t T, int32_t G, int32_t Hq, int32_t Hkv, int32_t D,
                       int32_t page_size, int64_t prefix_width, int64_t own_width) {
  if (!is_16bit(dtype)) return LORA_EUNSUPPORTED;
  if (T < 0 || G < 0 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || D < 1 || page_size < 1 ||
      prefix_width < 0 || own_width < 0)
    return LORA_EINVAL;
  if (D > 256 || D % 8 != 0) return LORA_EUNSUPPORTED;
  // 32-bit key indexes and row counts in the kernels
  constexpr int64_t kMaxKeys = int64_t(1) << 30;
  if (prefix_width > kMaxKeys / page_size || own_width > kMaxKeys / page_size) return LORA_EUNSUPPORTED;
  if (T > (int64_t(1) << 24) || G > (1 << 24) || T * Hq >= (int64_t(1) << 26)) return LORA_EUNSUPPORTED;
  return LORA_OK;
}

}  // namespace

extern "C" {

size_t lora_prefix_attention_workspace_size(lora_dtype dtype, int64_t T, int32_t G, int32_t Hq,
                                            int32_t Hkv, int32_t D, int32_t page_size,
                                            int64_t prefix_width, int64_t own_width) {
  if (attn_sizes(dtype, T, G, Hq, Hkv, D, page_size, prefix_width, own_width) != LORA_OK) return 0;
  if (T == 0 || G == 0) return 0;
  return lmx::prefix_attention_plan(T, G, Hq, Hkv, D, page_size, prefix_width, own_width).total;
}

lora_status lora_prefix_attention(lora_dtype dtype, int64_t T, int32_t G, int32_t Hq, int32_t Hkv,
                                  int32_t D, int64_t num_pages, int32_t page_size, const void* q,
                                  int64_t ldq, const void* k_cache, const void* v_cache,
                                  int64_t page_stride, int64_t token_stride, int64_t head_stride,
                                  const int32_t* seg_indptr, const int32_t* permutation,
                                  const int32_t* prefix_pages, int64_t prefix_width,
                                  const int32_t* prefix_lens, const int32_t* own_pages,
                                  int64_t own_width, const int32_t* own_lens, float scale,
                                  void* out, int64_t ldo, float* lse, void* workspace,
                                  size_t workspace_bytes, void* stream) {
  const lora_status s = attn_sizes(dtype, T, G, Hq, Hkv, D, page_size, prefix_width, own_width);
  if (s != LORA_OK) return s;
  if (num_pages < 0 || !std::isfinite(scale)) return LORA_EINVAL;
  if (num_pages >= INT_MAX) return LORA_EUNSUPPORTED;
  if (T == 0 || G == 0) return LORA_OK;
  if (!q || !out || !seg_indptr) return LORA_EINVAL;
  if (prefix_width > 0 && (!prefix_pages || !prefix_lens)) return LORA_EINVAL;
  if (own_width > 0 && (!own_pages || !own_lens)) return LORA_EINVAL;
  if (num_pages > 0 && (!k_cache || !v_cache)) return LORA_EINVAL;
  if (ldq < int64_t(Hq) * D || ldo < int64_t(Hq) * D || page_stride < 0 || token_stride < 0 ||
      head_stride < 0)
    return LORA_EINVAL;
  if (!al16(q) || ldq % 8 != 0 || !al16(k_cache) || !al16(v_cache) ||
      (num_pages > 1 && page_stride % 8 != 0) || (page_size > 1 && token_stride % 8 != 0) ||
      (Hkv > 1 && head_stride % 8 != 0))
    return LORA_EUNSUPPORTED;
  const lmx::PrefixAttnPlan p = lmx::prefix_attention_plan(T, G, Hq, Hkv, D, page_size, prefix_width, own_width);
  if (p.total > 0 && (workspace == nullptr || workspace_bytes < p.total || !al16(workspace)))
    return LORA_EWORKSPACE;
  const int64_t wgs = int64_t(Hkv) * (int64_t(p.prefix_tiles) * p.prefix_splits + T * p.own_tiles * p.own_splits);
  if (wgs >= (int64_t(1) << 24)) return LORA_EUNSUPPORTED;  // of 256 threads, of which a launch takes under 2^32
  lmx::PrefixAttnArgs a{};
  a.q = q; a.k_cache = k_cache; a.v_cache = v_cache; a.seg_indptr = seg_indptr;
  a.permutation = permutation; a.prefix_pages = prefix_pages; a.prefix_lens = prefix_lens;
  a.own_pages = own_pages; a.own_lens = own_lens; a.out = out; a.lse = lse;
  a.part_o = static_cast<float*>(workspace);
  a.part_ml = reinterpret_cast<float2*>(static_cast<char*>(workspace) + p.part_ml);
  a.ldq = ldq; a.ldo = ldo; a.page_stride = page_stride; a.token_stride = token_stride;
  a.head_stride = head_stride;
  a.T = int(T); a.G = G; a.Hq = Hq; a.Hkv = Hkv; a.grp = Hq / Hkv; a.D = D;
  a.page_size = page_size; a.num_pages = int(num_pages);
  a.prefix_width = int(prefix_width); a.own_width = int(own_width);
  a.prefix_tiles = p.prefix_tiles; a.prefix_splits = p.prefix_splits;
  a.own_tiles = p.own_tiles; a.own_splits = p.own_splits;
  a.by_kvh = lmx::FastDiv::of(Hkv); a.by_grp = lmx::FastDiv::of(a.grp);
  a.by_page = lmx::FastDiv::of(page_size); a.by_hq = lmx::FastDiv::of(Hq);
  a.by_prefix_splits = lmx::FastDiv::of(p.prefix_splits);
  a.by_own_tiles = lmx::FastDiv::of(p.own_tiles); a.by_own_splits = lmx::FastDiv::of(p.own_splits);
  a.out8 = (reinterpret_cast<uintptr_t>(out) & 7u) == 0 && ldo % 4 == 0;
  a.direct = p.direct; a.shared = p.shared; a.prefix_unit = p.prefix_unit; a.own_unit = p.own_unit;
  // the kernels multiply masked scores (-inf) by it: above 0, with the sign in the queries (a scale of
  // 0 gives equal weights, and so does 2^-100)
  a.negate = scale < 0.f;
  a.scale_log2 = std::max(std::fabs(scale) * 1.44269504f, 0x1p-100f);
  return hip_status(lmx::launch_prefix_attention(dtype, p, a, reinterpret_cast<hipStream_t>(stream)));
}

}  // extern "C"
