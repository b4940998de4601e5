// Internal launch interface of the rotation and cache-append kernel (not part of the public C ABI).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace lmx {

struct RopeArgs {
  const void *q, *k, *v;  // rows of Hq * D, Hkv * D and Hkv * D elements
  const float* table;     // [table_rows][rot]: rot / 2 cosines, then rot / 2 sines
  const int* positions;   // [T]
  const int64_t* slots;   // [T]
  const void *q_norm, *k_norm;  // [D] or null
  void *q_out, *k_cache, *v_cache;
  int64_t ldq, ldk, ldv, ldqo, page_stride, token_stride, head_stride, num_slots;
  int T, Hq, Hkv, D, rot, page_size, table_rows;
  float eps;
};

// vec: every row, weight and cache row is 16-byte aligned, D % 8 == 0 and rot % 16 == 0 (the caller
// checks).
hipError_t launch_rope_append(const RopeArgs& a, int dtype, bool interleaved, bool vec,
                              hipStream_t st);

}  // namespace lmx
