// Matrix-vector products with 4-bit weights: y = x W^T for few rows of x, where
//     W[n][k] = s[n][k / group] (c[n][k] - z[n][k / group]),   c in 0..15, z in 0..15 (8 if not given).
//
// A code becomes a 16-bit float without any conversion: placed in the top mantissa bits under the
// exponent of 16 it reads 16 + c exactly, in bf16 (0x4180 | c << 3) and in fp16 (0x4c00 | c << 6). The
// matrix step runs on 16 + c, and the offset and the zero point leave once per group in fp32:
//     y[m][n] = sum_groups s (sum_k x (16 + c)) - s (16 + z) (sum_k x),
// with both sums in fp32 and the second one a matrix step against ones, which lands in the same lanes
// and registers as the first. The subtraction costs at most 5 bits of the fp32 sums.
//
// Bound by the bytes of the weight. One workgroup per 16 NT output columns and 16 MT rows of x;
// its waves share out the K tiles (16 x 128 codes = 1 KiB, one 16-byte load a lane) and are added in
// LDS in a fixed order. Rows of x beyond M repeat row M - 1 and are not stored (a row of the product
// depends on its own row of x only).
#include "device_common.hpp"
#include "linear_w4.hpp"

namespace lmx {

namespace {

// The 8 codes of a dword as a fragment of 16 + c.
template <int DT>
__device__ __forceinline__ uint4 w4_frag(uint32_t w) {
  if constexpr (DT == DT_BF16) {
    return make_uint4(((w << 3) & 0x00780078u) | 0x41804180u, ((w >> 1) & 0x00780078u) | 0x41804180u,
                      ((w >> 5) & 0x00780078u) | 0x41804180u, ((w >> 9) & 0x00780078u) | 0x41804180u);
  } else {
    return make_uint4(((w << 6) & 0x03c003c0u) | 0x4c004c00u, ((w << 2) & 0x03c003c0u) | 0x4c004c00u,
                      ((w >> 2) & 0x03c003c0u) | 0x4c004c00u, ((w >> 6) & 0x03c003c0u) | 0x4c004c00u);
  }
}

template <int DT>
constexpr uint32_t ones2() { return DT == DT_BF16 ? 0x3f803f80u : 0x3c003c00u; }

constexpr int kWaves = 8;

// GS: steps of 32 per group (1, 2 or 4).
template <int DT, int MT, int NT, int GS, bool ZP>
__global__ __launch_bounds__(64 * kWaves) void linear_w4_kernel(W4Args a) {
  __shared__ float s_acc[kWaves][MT * NT * 256];
  const int lane = int(threadIdx.x) & 63, wave = wave_id();
  const int col = lane & 15, lg = lane >> 4;
  const int tn0 = int(blockIdx.x) * NT, m0 = int(blockIdx.y) * 16 * MT;
  const W4Layout L = w4_layout(a.K, a.N, a.group, ZP);
  const int ntiles = int(L.ntiles), ktiles = int(L.ktiles), groups = int(L.groups);
  const uint16_t* xr[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) xr[i] = a.x + int64_t(min(m0 + i * 16 + col, a.M - 1)) * a.ldx + lg * 8;
  f32x4_t acc[NT][MT];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int i = 0; i < MT; ++i) acc[n][i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  const uint4 ones = make_uint4(ones2<DT>(), ones2<DT>(), ones2<DT>(), ones2<DT>());

  for (int tk = wave; tk < ktiles; tk += kWaves) {
    uint4 code[NT];
    uint32_t meta[NT][4 / GS];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int tn = min(tn0 + n, ntiles - 1);
      code[n] = gload16(a.w + (int64_t(tn) * ktiles + tk) * 1024 + lane * 16);
#pragma unroll
      for (int g = 0; g < 4 / GS; ++g) {
        const int64_t at = (int64_t(tn) * groups + min(tk * (4 / GS) + g, groups - 1)) * 16 + col;
        if constexpr (ZP) meta[n][g] = reinterpret_cast<const uint32_t*>(a.w + L.meta)[at];
        else meta[n][g] = reinterpret_cast<const uint16_t*>(a.w + L.meta)[at];
      }
    }
    uint4 xf[4][MT];
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const int k = tk * 128 + s * 32;  // K is a multiple of 32: a step is whole or absent
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        xf[s][i] = make_uint4(0u, 0u, 0u, 0u);
        if (k < a.K) xf[s][i] = gload16(xr[i] + k);
      }
    }
#pragma unroll
    for (int g = 0; g < 4 / GS; ++g) {
      f32x4_t xs[MT];
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        xs[i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = 0; s < GS; ++s) xs[i] = mma_step<DT>(xf[g * GS + s][i], ones, xs[i]);
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        f32x4_t t[MT];
#pragma unroll
        for (int i = 0; i < MT; ++i) t[i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = 0; s < GS; ++s) {
          const uint32_t c[4] = {code[n].x, code[n].y, code[n].z, code[n].w};
          const uint4 wf = w4_frag<DT>(c[g * GS + s]);
#pragma unroll
          for (int i = 0; i < MT; ++i) t[i] = mma_step<DT>(xf[g * GS + s][i], wf, t[i]);
        }
        const float sc = Traits<DT>::to_f32(uint16_t(meta[n][g]));
        const float off = ZP ? sc * float(16 + int(meta[n][g] >> 16)) : sc * 24.f;
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[n][i][e] += sc * t[i][e] - off * xs[i][e];
      }
    }
  }
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        s_acc[wave][(i * 16 + lg * 4 + e) * (16 * NT) + n * 16 + col] = acc[n][i][e];
  __syncthreads();
  for (int e = int(threadIdx.x); e < MT * NT * 256; e += 64 * kWaves) {
    const int r = e / (16 * NT), c = e - r * (16 * NT);
    const int m = m0 + r, n = tn0 * 16 + c;
    if (m >= a.M || n >= a.N) continue;
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) v += s_acc[w][e];
    a.y[int64_t(m) * a.ldy + n] = Traits<DT>::from_f32(v);
  }
}

// One thread per (16-row tile, K tile, lane) dword, then one per (tile, group, row) scale.
__global__ __launch_bounds__(256) void w4_prepare_kernel(W4PrepareArgs a) {
  const W4Layout L = w4_layout(a.K, a.N, a.group, a.zeros != nullptr);
  const int64_t ncode = L.ntiles * L.ktiles * 256, nmeta = L.ntiles * L.groups * 16;
  const int64_t step = int64_t(gridDim.x) * 256;
  for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < ncode; i += step) {
    const int s = int(i & 3), lane = int(i >> 2) & 63;
    const int64_t tile = i >> 8;
    const int64_t n = tile / L.ktiles * 16 + (lane & 15);
    const int64_t k = tile % L.ktiles * 128 + s * 32 + (lane >> 4) * 8;
    uint32_t w = 0;
    if (n < a.N && k < a.K) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t b = a.codes[n * a.ldc + (k >> 1) + e];
        w |= ((b & 15u) << (4 * e)) | ((b >> 4) << (16 + 4 * e));
      }
    }
    reinterpret_cast<uint32_t*>(a.out)[i] = w;
  }
  for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < nmeta; i += step) {
    const int64_t n = i / 16 / L.groups * 16 + (i & 15), g = i / 16 % L.groups;
    const bool ok = n < a.N;
    const uint16_t sc = ok ? a.scales[n * a.lds + g] : uint16_t(0);
    if (a.zeros != nullptr) {
      const uint32_t z = ok ? uint32_t(a.zeros[n * a.ldz + g]) & 15u : 0u;
      reinterpret_cast<uint32_t*>(a.out + L.meta)[i] = sc | (z << 16);
    } else {
      reinterpret_cast<uint16_t*>(a.out + L.meta)[i] = sc;
    }
  }
}

template <int DT, int MT, int GS, bool ZP>
hipError_t launch_mt(const W4Args& a, hipStream_t st) {
  const dim3 grid(unsigned((a.N + 15) / 16), unsigned((a.M + 16 * MT - 1) / (16 * MT)));
  hipLaunchKernelGGL((linear_w4_kernel<DT, MT, 1, GS, ZP>), grid, dim3(64 * kWaves), 0, st, a);
  return hipGetLastError();
}

template <int DT, int GS, bool ZP>
hipError_t launch_gs(const W4Args& a, hipStream_t st) {
  if (a.M <= 16) return launch_mt<DT, 1, GS, ZP>(a, st);
  if (a.M <= 32) return launch_mt<DT, 2, GS, ZP>(a, st);
  return launch_mt<DT, 4, GS, ZP>(a, st);
}

template <int DT, bool ZP>
hipError_t launch_group(const W4Args& a, hipStream_t st) {
  if (a.group == 32) return launch_gs<DT, 1, ZP>(a, st);
  if (a.group == 64) return launch_gs<DT, 2, ZP>(a, st);
  return launch_gs<DT, 4, ZP>(a, st);
}

}  // namespace

hipError_t launch_w4_prepare(const W4PrepareArgs& a, hipStream_t st) {
  const W4Layout L = w4_layout(a.K, a.N, a.group, a.zeros != nullptr);
  const int64_t blocks = (L.ntiles * L.ktiles * 256 + 255) / 256;
  hipLaunchKernelGGL(w4_prepare_kernel, dim3(unsigned(blocks < 65536 ? blocks : 65536)), dim3(256), 0, st, a);
  return hipGetLastError();
}

hipError_t launch_linear_w4(const W4Args& a, int dtype, bool zeros, hipStream_t st) {
  if (dtype == DT_BF16)
    return zeros ? launch_group<DT_BF16, true>(a, st) : launch_group<DT_BF16, false>(a, st);
  return zeros ? launch_group<DT_F16, true>(a, st) : launch_group<DT_F16, false>(a, st);
}

}  // namespace lmx
