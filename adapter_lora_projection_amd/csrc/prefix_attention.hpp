// Internal launch interface of the shared-prefix attention kernels (not part of the public C ABI).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace lmx {

// n / d for 0 <= n < 2^31 as one high product: m = floor(2^(32 + s) / d) + 1 with s = floor(log2 d) is off
// by at most d <= 2^(s + 1) parts in 2^(32 + s), which n does not carry over. m = 0 stands for d = 1; a
// power of two takes 2^31 and one shift less.
struct FastDiv {
  uint32_t m, s;
  int d;
  static FastDiv of(int64_t d) {
    FastDiv f{0u, 0u, int(d)};
    if (d <= 1) return f;
    while ((int64_t(2) << f.s) <= d) ++f.s;
    if ((int64_t(1) << f.s) == d) {
      f.m = 0x80000000u;
      f.s -= 1;
    } else {
      f.m = uint32_t((uint64_t(1) << (32 + f.s)) / uint64_t(d)) + 1u;
    }
    return f;
  }
  __host__ __device__ int div(int n) const {
    return m == 0 ? n : int(uint32_t((uint64_t(uint32_t(n)) * m) >> 32) >> s);
  }
};

struct PrefixAttnArgs {
  const void* q;        // [T][ldq], head h of token t at t * ldq + h * D
  const void* k_cache;  // element (page, place, head, d) at page * page_stride + place *
  const void* v_cache;  //   token_stride + head * head_stride + d, the same for both
  const int* seg_indptr;
  const int* permutation;   // null: identity
  const int* prefix_pages;  // [G][prefix_width]
  const int* prefix_lens;   // [G] (null: no prefixes)
  const int* own_pages;     // [T][own_width]
  const int* own_lens;      // [T] (null: no keys of their own)
  void* out;                // [T][ldo]
  float* lse;               // [T][Hq] or null
  float* part_o;            // [slots][T * Hq][D]: unnormalised outputs of each key range
  float2* part_ml;          // [slots][T * Hq]: running maximum (base 2) and sum of each
  int64_t ldq, ldo, page_stride, token_stride, head_stride;
  int T, G, Hq, Hkv, grp, D, page_size, num_pages, prefix_width, own_width;
  FastDiv by_kvh, by_grp, by_page, by_prefix_splits, by_own_tiles, by_own_splits, by_hq;
  int prefix_tiles, prefix_splits;  // row-tile bound and key ranges of the prefix part
  int own_tiles, own_splits;        // row tiles per token and key ranges of the own part
  int prefix_unit, own_unit;        // keys that a range is a multiple of
  int shared;                       // prefix tiles of 128 rows, else 16
  int direct;                       // one key range a row: no partials, no join
  int out8;                         // output rows are 8-byte aligned
  int negate;                       // scale < 0: the queries' signs are flipped
  float scale_log2;                 // |scale| * log2(e), above 0
};

// Launch plan from host-known sizes only (lengths live on the device; the page lists' widths bound
// them).
struct PrefixAttnPlan {
  int dp;  // head size rounded up to 64, 128 or 256
  bool shared;  // prefix tiles of 128 rows sharing their key blocks (else 16 rows)
  bool direct;  // one key range per row, written to the output at once
  int prefix_tiles, prefix_splits, prefix_unit, own_tiles, own_splits, own_unit;
  size_t part_ml, total;  // workspace: byte offset of part_ml, total bytes
};
PrefixAttnPlan prefix_attention_plan(int64_t T, int G, int Hq, int Hkv, int D, int page_size,
                                     int64_t prefix_width, int64_t own_width);

hipError_t launch_prefix_attention(int dtype, const PrefixAttnPlan& plan, const PrefixAttnArgs& a,
                                   hipStream_t st);

}  // namespace lmx
