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
// Bound by the bytes of the weight and, from a few rows on, of x: the two kernels below share them
// out differently. Rows of x beyond M repeat row M - 1 and are not stored (a row of the product depends
// on its own row of x only). Sums are added in a fixed order.
#include <algorithm>

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

// acc += the K tile's part: its 128 codes per column (`code`, a dword per step of 32) against the fragments
// frag(s, i) of the 4 steps. GS: steps per group (1, 2 or 4).
template <int DT, int MT, int NT, int GS, bool ZP, typename F>
__device__ __forceinline__ void w4_tile(const uint4 (&code)[NT], const uint32_t (&meta)[NT][4 / GS],
                                        F frag, f32x4_t (&acc)[NT][MT]) {
  const uint4 ones = make_uint4(ones2<DT>(), ones2<DT>(), ones2<DT>(), ones2<DT>());
#pragma unroll
  for (int g = 0; g < 4 / GS; ++g) {
    uint4 xf[GS][MT];
#pragma unroll
    for (int s = 0; s < GS; ++s)
#pragma unroll
      for (int i = 0; i < MT; ++i) xf[s][i] = frag(g * GS + s, i);
    f32x4_t xs[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      xs[i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int s = 0; s < GS; ++s) xs[i] = mma_step<DT>(xf[s][i], ones, xs[i]);
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      f32x4_t t[MT];
#pragma unroll
      for (int i = 0; i < MT; ++i) t[i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
      const uint32_t c[4] = {code[n].x, code[n].y, code[n].z, code[n].w};
#pragma unroll
      for (int s = 0; s < GS; ++s) {
        const uint4 wf = w4_frag<DT>(c[g * GS + s]);
#pragma unroll
        for (int i = 0; i < MT; ++i) t[i] = mma_step<DT>(xf[s][i], wf, t[i]);
      }
      uint32_t mt = meta[n][g];
      asm volatile("" : "+v"(mt));  // converted here: at the load it would wait for the load
      const float sc = Traits<DT>::to_f32(uint16_t(mt));
      const float off = ZP ? sc * float(16 + int(mt >> 16)) : sc * 24.f;
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[n][i][e] += sc * t[i][e] - off * xs[i][e];
    }
    if constexpr (MT > 2) __builtin_amdgcn_sched_barrier(0);  // one group's fragments at a time: 64 rows fill the registers
  }
}

// Codes and scales of K tile tk (clamped into the weight) for the 16-column tiles tn0 ...
template <int NT, int GS, bool ZP>
__device__ __forceinline__ void w4_load(const W4Args& a, const W4Layout& L, int tn0, int tk, uint4 (&code)[NT],
                                        uint32_t (&meta)[NT][4 / GS]) {
  constexpr int G = 4 / GS;
  const int lane = int(threadIdx.x) & 63, groups = int(L.groups);
  tk = min(tk, int(L.ktiles) - 1);
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int tn = min(tn0 + n, int(L.ntiles) - 1);
    code[n] = gload16(a.w + (int64_t(tn) * L.ktiles + tk) * 1024 + lane * 16);
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const int64_t at = (int64_t(tn) * groups + min(tk * G + g, groups - 1)) * 16 + (lane & 15);
      if constexpr (ZP) meta[n][g] = reinterpret_cast<const uint32_t*>(a.w + L.meta)[at];
      else meta[n][g] = reinterpret_cast<const uint16_t*>(a.w + L.meta)[at];
    }
  }
}

// Column kernel, up to 16 rows of x per workgroup: W waves share out the K tiles of 16 columns and are added
// in LDS. One launch and no workspace; x is read once per 16 columns, so its bytes count from a few
// rows on. Latency is hidden by the workgroups of a compute unit (4 of them), not by a ring of tiles per
// wave: one row x 4096 x 24576, 10.8 us; with 3 tiles in flight 13.2 (2 workgroups fit), with 4 18.5.
template <int DT, int W, int GS, bool ZP>
__global__ __launch_bounds__(64 * W, 4) void linear_w4_kernel(W4Args a) {
  __shared__ float s_acc[W][256];
  const int lane = int(threadIdx.x) & 63, wave = wave_id();
  const int col = lane & 15, lg = lane >> 4;
  const int tn = int(blockIdx.x), m0 = int(blockIdx.y) * 16;
  const W4Layout L = w4_layout(a.K, a.N, a.group, ZP);
  const int ktiles = int(L.ktiles);
  const uint16_t* xr = a.x + int64_t(min(m0 + col, a.M - 1)) * a.ldx + lg * 8;
  f32x4_t acc[1][1] = {{f32x4_t{0.f, 0.f, 0.f, 0.f}}};
  for (int tk = wave; tk < ktiles; tk += W) {
    uint4 code[1], xf[4];
    uint32_t meta[1][4 / GS];
    w4_load<1, GS, ZP>(a, L, tn, tk, code, meta);
#pragma unroll
    for (int s = 0; s < 4; ++s) xf[s] = gload16(xr + min(tk * 128 + s * 32, a.K - 32));
    if (tk * 128 + 128 > a.K) {  // K is a multiple of 32: a step is whole, or repeats the last one as zeros
#pragma unroll
      for (int s = 1; s < 4; ++s)
        if (tk * 128 + s * 32 >= a.K) xf[s] = make_uint4(0u, 0u, 0u, 0u);
    }
    w4_tile<DT, 1, 1, GS, ZP>(code, meta, [&](int s, int) { return xf[s]; }, acc);
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) s_acc[wave][(lg * 4 + e) * 16 + col] = acc[0][0][e];
  __syncthreads();
  const int e = int(threadIdx.x), m = m0 + (e >> 4), n = tn * 16 + (e & 15);
  if (e >= 256 || m >= a.M || n >= a.N) return;
  float v = 0.f;
#pragma unroll
  for (int w = 0; w < W; ++w) v += s_acc[w][e];
  a.y[int64_t(m) * a.ldy + n] = Traits<DT>::from_f32(v);
}

// Workgroup barrier after this wave's LDS operations, for loops with global loads in flight.
__device__ __forceinline__ void lds_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// Slab kernel: a workgroup takes 128 NT columns (its 8 waves 16 NT each), 16 MT rows of x and a range of K
// tiles. The x tile is staged in LDS once for all waves (double buffered, one barrier a tile; 16-byte
// chunks XOR-swizzled by the row, so that 16 rows at one chunk spread over the banks). A compute unit
// takes in about 25 bytes/ns whatever their source, so what counts is the sum of the weight's and x's
// bytes per unit: few columns over all of K would read x N / 16 times. With several ranges
// (gridDim.y > 1) the sums go to fp32 planes, which w4_sum_kernel adds in order.
constexpr int kSlabWaves = 8;
template <int DT, int MT, int NT, int GS, bool ZP>
__global__ __launch_bounds__(64 * kSlabWaves) void linear_w4_slab_kernel(W4Args a) {
  constexpr int PD = MT > 2 ? 2 : 3;  // tiles in flight (64 rows leave registers for two)
  constexpr int XL = (MT + 1) / 2;  // 16-byte pieces of the x tile per thread: 256 MT pieces, 512 threads
  __shared__ __align__(16) uint16_t s_x[2][16 * MT * 128];
  const int lane = int(threadIdx.x) & 63, wave = wave_id(), tid = int(threadIdx.x);
  const int col = lane & 15, lg = lane >> 4;
  const int tn0 = (int(blockIdx.x) * kSlabWaves + wave) * NT, m0 = int(blockIdx.z) * 16 * MT;
  const W4Layout L = w4_layout(a.K, a.N, a.group, ZP);
  const int ktiles = int(L.ktiles), per = ceil_div(ktiles, int(gridDim.y));
  const int t0 = int(blockIdx.y) * per, t1 = min(t0 + per, ktiles);

  uint4 xv[PD][XL];
  // x tile t into registers: piece p = row p / 16, chunk p % 16; row M - 1 beyond M, zeroed beyond K when
  // it is stored
  auto load_x = [&](int u, int t) {
#pragma unroll
    for (int i = 0; i < XL; ++i) {
      const int p = tid + i * 512, r = p >> 4, k = t * 128 + (p & 15) * 8;
      if (p < 256 * MT) xv[u][i] = gload16(a.x + int64_t(min(m0 + r, a.M - 1)) * a.ldx + min(k, a.K - 8));
    }
  };
  auto store_x = [&](int u, int t, int buf) {
#pragma unroll
    for (int i = 0; i < XL; ++i) {
      const int p = tid + i * 512, r = p >> 4, c = (p & 15) ^ (r & 15);
      const uint4 v = t * 128 + (p & 15) * 8 < a.K ? xv[u][i] : make_uint4(0u, 0u, 0u, 0u);
      if (p < 256 * MT) *reinterpret_cast<uint4*>(&s_x[buf][r * 128 + c * 8]) = v;
    }
  };
  f32x4_t acc[NT][MT];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int i = 0; i < MT; ++i) acc[n][i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  uint4 code[PD][NT];
  uint32_t meta[PD][NT][4 / GS];
#pragma unroll
  for (int u = 0; u < PD; ++u) {
    if (t0 + u < t1) {
      load_x(u, t0 + u);
      w4_load<NT, GS, ZP>(a, L, tn0, t0 + u, code[u], meta[u]);
    }
  }
  store_x(0, t0, 0);
  if (t0 + PD < t1) load_x(0, t0 + PD);
  // tile t in slot u; more_x, more_w: tiles t + 1 + PD and t + PD are there
  auto step = [&](int t, int u, bool more_x, bool more_w) {
    const int buf = (t - t0) & 1;
    lds_barrier();  // tile t is in s_x[buf], and nobody reads the other buffer any more
    if (t + 1 < t1) store_x((u + 1) % PD, t + 1, buf ^ 1);
    if (more_x) load_x((u + 1) % PD, t + 1 + PD);
    w4_tile<DT, MT, NT, GS, ZP>(code[u], meta[u], [&](int s, int i) {
      return *reinterpret_cast<const uint4*>(&s_x[buf][(i * 16 + col) * 128 + ((s * 4 + lg) ^ col) * 8]);
    }, acc);
    if (more_w) w4_load<NT, GS, ZP>(a, L, tn0, t + PD, code[u], meta[u]);
  };
  // whole rounds of the ring, every load unconditional (a branch around one would make the next wait one
  // for all of them), then what is left
  int tb = t0;
  for (; tb + 2 * PD < t1; tb += PD) {
#pragma unroll
    for (int u = 0; u < PD; ++u) step(tb + u, u, true, true);
  }
  for (; tb < t1; tb += PD) {
#pragma unroll
    for (int u = 0; u < PD; ++u)
      if (tb + u < t1) step(tb + u, u, tb + u + 1 + PD < t1, tb + u + PD < t1);
  }
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int m = m0 + i * 16 + lg * 4 + e, c = (tn0 + n) * 16 + col;
        if (m >= a.M) continue;
        if (gridDim.y > 1) {
          if (tn0 + n < int(L.ntiles)) a.part[(int64_t(blockIdx.y) * a.M + m) * (L.ntiles * 16) + c] = acc[n][i][e];
        } else if (c < a.N) {
          a.y[int64_t(m) * a.ldy + c] = Traits<DT>::from_f32(acc[n][i][e]);
        }
      }
}

// y = the sum of `planes` fp32 planes [M][pitch] in order; four columns a thread.
template <int DT>
__global__ __launch_bounds__(256) void w4_sum_kernel(W4Args a, int planes, int pitch) {
  const int q = pitch / 4;
  const int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x;
  if (i >= int64_t(a.M) * q) return;
  const int m = int(i / q), n = int(i - int64_t(m) * q) * 4;
  const float* p = a.part + int64_t(m) * pitch + n;
  const int64_t plane = int64_t(a.M) * pitch;
  float4 v = *reinterpret_cast<const float4*>(p);
#pragma unroll 8
  for (int s = 1; s < planes; ++s) {
    const float4 u = *reinterpret_cast<const float4*>(p + s * plane);
    v.x += u.x; v.y += u.y; v.z += u.z; v.w += u.w;
  }
  const float r[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (n + e < a.N) a.y[int64_t(m) * a.ldy + n + e] = Traits<DT>::from_f32(r[e]);
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

template <int DT, int W, int GS, bool ZP>
hipError_t launch_columns(const W4Args& a, hipStream_t st) {
  const dim3 grid(unsigned((a.N + 15) / 16), unsigned((a.M + 15) / 16));
  hipLaunchKernelGGL((linear_w4_kernel<DT, W, GS, ZP>), grid, dim3(64 * W), 0, st, a);
  return hipGetLastError();
}

template <int DT, int MT, int NT, int GS, bool ZP>
hipError_t launch_slab(const W4Args& a, const W4Plan& p, hipStream_t st) {
  const dim3 grid(unsigned((a.N + 128 * NT - 1) / (128 * NT)), unsigned(p.ranges), unsigned((a.M + 16 * MT - 1) / (16 * MT)));
  hipLaunchKernelGGL((linear_w4_slab_kernel<DT, MT, NT, GS, ZP>), grid, dim3(64 * kSlabWaves), 0, st, a);
  if (p.ranges > 1) {
    const int pitch = (a.N + 15) / 16 * 16;
    const int64_t n = int64_t(a.M) * (pitch / 4);
    hipLaunchKernelGGL((w4_sum_kernel<DT>), dim3(unsigned((n + 255) / 256)), dim3(256), 0, st, a, p.ranges, pitch);
  }
  return hipGetLastError();
}

template <int DT, int GS, bool ZP>
hipError_t launch_gs(const W4Args& a, const W4Plan& p, hipStream_t st) {
  if (p.ranges > 0) {
    if (a.M <= 16) return launch_slab<DT, 1, 1, GS, ZP>(a, p, st);
    // groups of 32 hold too many sums at once for the larger shapes
    if constexpr (GS == 1) return launch_slab<DT, 2, 1, GS, ZP>(a, p, st);
    else if (a.M <= 32) return launch_slab<DT, 2, 2, GS, ZP>(a, p, st);
    else return launch_slab<DT, 4, 2, GS, ZP>(a, p, st);
  }
  if (p.wide) return launch_columns<DT, 16, GS, ZP>(a, st);
  return launch_columns<DT, 8, GS, ZP>(a, st);
}

template <int DT, bool ZP>
hipError_t launch_group(const W4Args& a, const W4Plan& p, hipStream_t st) {
  if (a.group == 32) return launch_gs<DT, 1, ZP>(a, p, st);
  if (a.group == 64) return launch_gs<DT, 2, ZP>(a, p, st);
  return launch_gs<DT, 4, ZP>(a, p, st);
}

}  // namespace

hipError_t launch_w4_prepare(const W4PrepareArgs& a, hipStream_t st) {
  const W4Layout L = w4_layout(a.K, a.N, a.group, a.zeros != nullptr);
  const int64_t blocks = (L.ntiles * L.ktiles * 256 + 255) / 256;
  hipLaunchKernelGGL(w4_prepare_kernel, dim3(unsigned(blocks < 65536 ? blocks : 65536)), dim3(256), 0, st, a);
  return hipGetLastError();
}

// Time of either kernel in ns, from the bytes its busiest compute unit takes in: about 34 a ns in the
// column kernel and 25 in the slab kernel, and 6.5 us for planes and the second launch. Measured on
// weights that are not in the caches, column kernel against the best slab: 16 rows x 4096 x 4096 6.5 /
// 10.7 us, 16 x 4096 x 24576 27 / 20, 16 x 16384 x 1024 18 / 12, 32 x 8192 x 8192 35 / 19, 64 x 12288 x
// 4096 49 / 23, 64 x 16384 x 28672 429 / 119, 24 x 768 x 3426 3.8 / 8.5.
W4Plan w4_plan(int64_t M, int64_t K, int64_t N, int group) {
  W4Plan best{};
  const int64_t ntiles = (N + 15) / 16, kt = (K + 127) / 128;
  auto rounds = [](int64_t wgs) { return double((wgs + 255) / 256); };
  best.wide = ntiles * ((M + 15) / 16) <= 128 && kt >= 16;
  double least = rounds(ntiles * ((M + 15) / 16)) * double(kt) * double(1088 + 256 * std::min<int64_t>(M, 16)) / 34;
  // the shapes of launch_gs
  const int64_t mt = M <= 16 ? 1 : M <= 32 || group == 32 ? 2 : 4, nt = M <= 16 || group == 32 ? 1 : 2;
  const int64_t slabs = (N + 128 * nt - 1) / (128 * nt), mb = (M + 16 * mt - 1) / (16 * mt);
  for (int64_t want = 1; want <= std::min<int64_t>(kt, 64); want *= 2) {
    const int64_t per = (kt + want - 1) / want, r = (kt + per - 1) / per;  // no empty ranges at the end
    if (r > 1 && M * ntiles >= int64_t(1) << 29) break;  // four columns a thread, under 2^31 threads in w4_sum_kernel
    double c = rounds(slabs * mb * r) * double(per) * double(8 * nt * 1088 + 4096 * mt);
    if (r > 1) c += rounds(slabs * mb * r) * 8192.0 * nt * mt + double(r * M * ntiles * 16 * 4) / 256;
    c = c / 25 + (r > 1 ? 6500 : 0);
    if (c < least) {
      least = c;
      best.ranges = int(r);
    }
  }
  if (best.ranges > 1) best.workspace = size_t(best.ranges) * size_t(M) * size_t(ntiles) * 64;
  return best;
}

hipError_t launch_linear_w4(const W4Args& a, const W4Plan& p, int dtype, bool zeros, hipStream_t st) {
  if (dtype == DT_BF16)
    return zeros ? launch_group<DT_BF16, true>(a, p, st) : launch_group<DT_BF16, false>(a, p, st);
  return zeros ? launch_group<DT_F16, true>(a, p, st) : launch_group<DT_F16, false>(a, p, st);
}

}  // namespace lmx
