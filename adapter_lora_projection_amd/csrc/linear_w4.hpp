// Internal launch interface of the 4-bit-weight projection (not part of the public C ABI).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace lmx {

// The prepared weight: byte offsets of its two parts (256-byte aligned).
//   codes  [ceil(N / 16)][ceil(K / 128)][64 lanes][16 bytes]: lane n + 16 g of tile (tn, tk) holds
//          W[16 tn + n][128 tk + 32 s + 8 g + e] (s < 4 its dwords, e < 8), element e in bits
//          4 (e / 2) of the dword's half e % 2. Entries beyond N or K are 0.
//   meta   [ceil(N / 16)][K / group][16]: the scale of (n, group), 16 bits; with zero points a dword,
//          the zero point in its upper half.
struct W4Layout {
  int64_t ntiles, ktiles, groups;
  size_t meta, total;
};
__host__ __device__ inline W4Layout w4_layout(int64_t K, int64_t N, int group, bool zeros) {
  W4Layout l{};
  l.ntiles = (N + 15) / 16;
  l.ktiles = (K + 127) / 128;
  l.groups = K / group;
  l.meta = size_t(l.ntiles) * l.ktiles * 1024;
  l.total = l.meta + size_t(l.ntiles) * l.groups * 16 * (zeros ? 4 : 2);
  l.total = (l.total + 255) & ~size_t(255);
  return l;
}

struct W4PrepareArgs {
  const uint8_t* codes;    // [N][ldc], two codes a byte, even k low
  const uint16_t* scales;  // [N][lds]
  const uint8_t* zeros;    // [N][ldz] or null
  uint8_t* out;
  int64_t ldc, lds, ldz;
  int K, N, group;
};
hipError_t launch_w4_prepare(const W4PrepareArgs& a, hipStream_t st);

struct W4Args {
  const uint16_t* x;  // [M][ldx]
  const uint8_t* w;   // prepared
  uint16_t* y;        // [M][ldy]
  float* part;        // planes of W4Plan
  int64_t ldx, ldy;
  int M, K, N, group;
};
// How a product is shared out, from its sizes alone.
struct W4Plan {
  int ranges;        // 0: column kernel; else slab kernel over this many ranges of K
  bool wide;         // column kernel with 16 waves (else 8)
  size_t workspace;  // bytes: fp32 planes [ranges][M][ceil(N / 16) * 16] of more than one range
};
W4Plan w4_plan(int64_t M, int64_t K, int64_t N, int group);

hipError_t launch_linear_w4(const W4Args& a, const W4Plan& p, int dtype, bool zeros, hipStream_t st);

}  // namespace lmx
