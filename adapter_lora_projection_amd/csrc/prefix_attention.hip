// Attention of a batch of query tokens over a paged key/value cache, where the tokens of a segment
// (one adapter's tokens: keys and values depend on the adapter) share a prefix.
//
// For sorted position i (token t = perm[i], segment g) and query head h, over the keys j of the
// segment's prefix followed by the token's own:
//     s_j = scale q_t,h . k_j,   o = sum_j exp(s_j - m) v_j / sum_j exp(s_j - m),   m = max_j s_j.
// Every (row tile, key head, key range) is one workgroup; its waves take 32-key blocks of the range
// in turn, each with its own running maximum and sum (fp32, base 2), and are joined in LDS at the
// end. The ranges of a row are joined by a second kernel with the same rule. A prefix tile holds 16
// query rows (token, head of the group) of one segment, so the prefix is read once per 16 rows;
// an own tile holds the query heads of one token.
//
// Matrix steps (v_mfma_f32_16x16x32): scores transposed, S^T = K Q^T (K rows as the A operand, the
// queries as columns), so that a lane holds 4 + 4 scores of ONE query and the softmax needs two
// cross-lane steps per block; O^T = V^T P^T takes those 8 probabilities as its B operand as they
// lie (keys 4g + i and 16 + 4g + i of lane group g; the contraction order is free as long as V uses
// the same), and V^T is read from the row-major block by the transposing LDS read.
// P is rounded to the storage type for the second product, and the sum of a row adds the rounded
// values, so the weights applied are normalised exactly; scores, maxima, sums and outputs are fp32.
//
// Keys and values go straight from the cache to LDS (16 bytes a lane); the addresses come from a
// per-wave table of 256 key offsets in LDS, so that no page-list load sits in the way of the
// loads in flight. The 16-byte chunks of a key row are XOR-swizzled by the row (by the choice of
// the global chunk each lane fetches) so that 16 rows at one chunk spread over the banks.
// A key whose page id lies outside the cache, or beyond its list's length, is masked: its offset is
// -1, its row is filled from a zero vector and its score is -inf.
#include <algorithm>

#include "device_common.hpp"
#include "prefix_attention.hpp"

namespace lmx {

namespace {

typedef short s16x4_t __attribute__((ext_vector_type(4)));

__device__ const uint4 kZeroChunk = {0u, 0u, 0u, 0u};

constexpr int kBlk = 32;       // keys per block
constexpr int kTabBlocks = 8;  // blocks covered by one fill of the offset table

constexpr float kNegInf = -__builtin_huge_valf();

// Four 16-bit elements down a column: lane t of a 16-lane group passes the address of row t / 4,
// columns 4 (t % 4) .. + 3 of a 4 x 16 block and receives rows 0..3 of column t.
__device__ __forceinline__ s16x4_t lds_read_tr(uint32_t addr) {
  typedef __attribute__((address_space(3))) s16x4_t lds_t;
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16(reinterpret_cast<lds_t*>(addr));
}

__device__ __forceinline__ uint4 lds_read16(uint32_t addr) {
  typedef unsigned int u32x4_t __attribute__((ext_vector_type(4)));
  typedef __attribute__((address_space(3))) u32x4_t lds_t;
  const u32x4_t v = *reinterpret_cast<lds_t*>(addr);
  return make_uint4(v.x, v.y, v.z, v.w);
}

// What one workgroup computes: rows of one segment or token, one key head, one key range.
struct Work {
  const int* pages;  // page list of the keys
  int len;           // keys of the whole list
  int k0, k1;        // key range of this workgroup
  int row0, nrows;   // flattened rows (sorted position * grp + head of the group) of the tile
  int slot;          // partial slot
  int kvh;
  bool live;
};

__device__ __forceinline__ int clamp_len(int len, int width, int page) {
  const int64_t cap = int64_t(width) * page;
  return int(min(int64_t(max(len, 0)), cap));
}

// Key range of split `s` of `n`: equal shares rounded up to `unit` keys.
__device__ __forceinline__ void key_range(int len, int n, int s, int unit, int* k0, int* k1) {
  const int per = ((len + n - 1) / n + unit - 1) / unit * unit;
  const int64_t lo = int64_t(per) * s;
  *k0 = int(min(lo, int64_t(len)));
  *k1 = int(min(lo + per, int64_t(len)));
}

__device__ __forceinline__ int seg_lo(const PrefixAttnArgs& a, int g) {
  return min(max(a.seg_indptr[g], 0), a.T);
}

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// Decodes blockIdx into a Work. Prefix workgroups come first (they are the longest).
template <int ROWS, int UNIT>
__device__ __forceinline__ Work find_work(const PrefixAttnArgs& a, int b) {
  Work w{};
  const int np = a.prefix_tiles * a.prefix_splits * a.Hkv;
  if (b < np) {
    w.kvh = b % a.Hkv;
    const int rest = b / a.Hkv;
    w.slot = rest % a.prefix_splits;
    int tile = rest / a.prefix_splits;
    // segment-major search for the row tile (every lane walks 64 segments at a time)
    const int lane = int(threadIdx.x) & 63;
    for (int g0 = 0; g0 < a.G; g0 += 64) {
      const int g = g0 + lane;
      int lo = 0, n = 0;
      if (g < a.G) {
        lo = seg_lo(a, g);
        n = max(seg_lo(a, g + 1) - lo, 0);
      }
      const int nt = (n * a.grp + ROWS - 1) / ROWS;
      int incl = nt;
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const int o = __shfl_up(incl, d, 64);
        if (lane >= d) incl += o;
      }
      const int excl = incl - nt;
      const unsigned long long hit = __ballot(tile >= excl && tile < incl);
      if (hit != 0) {
        const int src = __ffsll(hit) - 1;
        const int lo_s = uniform(__shfl(lo, src, 64)), n_s = uniform(__shfl(n, src, 64));
        const int ex = uniform(__shfl(excl, src, 64));
        const int gs = g0 + src, r0 = (tile - ex) * ROWS;
        w.row0 = lo_s * a.grp + r0;
        w.nrows = min(ROWS, n_s * a.grp - r0);
        w.pages = a.prefix_pages + int64_t(gs) * a.prefix_width;
        w.len = clamp_len(a.prefix_lens[gs], a.prefix_width, a.page_size);
        key_range(w.len, a.prefix_splits, w.slot, UNIT, &w.k0, &w.k1);
        w.live = w.k1 > w.k0;
        return w;
      }
      tile -= uniform(__shfl(incl, 63, 64));
    }
    return w;
  }
  b -= np;
  w.kvh = b % a.Hkv;
  int rest = b / a.Hkv;
  const int tile = rest % a.own_tiles;
  rest /= a.own_tiles;
  const int split = rest % a.own_splits;
  const int i = rest / a.own_splits;  // sorted position
  if (i >= a.T || i < seg_lo(a, 0) || i >= seg_lo(a, a.G)) return w;
  const int tok = a.permutation != nullptr ? a.permutation[i] : i;
  if (tok < 0 || tok >= a.T) return w;
  w.slot = a.prefix_splits + split;
  w.row0 = i * a.grp + tile * ROWS;
  w.nrows = min(ROWS, a.grp - tile * ROWS);
  w.pages = a.own_pages + int64_t(tok) * a.own_width;
  w.len = clamp_len(a.own_lens[tok], a.own_width, a.page_size);
  key_range(w.len, a.own_splits, split, UNIT, &w.k0, &w.k1);
  w.live = w.k1 > w.k0;
  return w;
}

template <int DT>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  return uint32_t(Traits<DT>::from_f32(a)) | (uint32_t(Traits<DT>::from_f32(b)) << 16);
}

// LDS of one wave: two buffers of a K and a V block, the key offset table and the block masks.
template <int DP>
struct WaveLds {
  uint16_t kv[2][2][kBlk * DP];
  int64_t off[kTabBlocks * kBlk];
  uint32_t mask[kTabBlocks];
};

template <int DP>
constexpr int attn_waves() { return DP > 128 ? 2 : 4; }

template <int DT, int DP>
__global__ __launch_bounds__(64 * attn_waves<DP>()) void prefix_attn_kernel(PrefixAttnArgs a) {
  constexpr int NW = attn_waves<DP>();
  constexpr int CPR = DP / 8;         // 16-byte chunks per key row
  constexpr int RPI = 64 / CPR;       // key rows one DMA instruction covers
  constexpr int NI = kBlk / RPI;      // DMA instructions per block and operand
  constexpr int KS = DP / 32;         // reduction steps of the scores
  constexpr int DTILES = DP / 16;     // 16-row tiles of O^T
  __shared__ __align__(16) WaveLds<DP> s_wave[NW];
  __shared__ float2 s_ml[NW][16];

  const Work w = find_work<16, kBlk * NW>(a, int(blockIdx.x));
  if (!w.live) return;

  const int lane = int(threadIdx.x) & 63, wave = wave_id();
  const int col = lane & 15, grp = lane >> 4;
  WaveLds<DP>& L = s_wave[wave];
  const uint16_t* kc = static_cast<const uint16_t*>(a.k_cache);
  const uint16_t* vc = static_cast<const uint16_t*>(a.v_cache);

  // the query column of this lane
  const bool row_ok = col < w.nrows;
  const int row = w.row0 + min(col, w.nrows - 1);
  const int pos = row / a.grp, head = w.kvh * a.grp + row % a.grp;
  const int tok = a.permutation != nullptr ? a.permutation[pos] : pos;
  const bool tok_ok = row_ok && tok >= 0 && tok < a.T;
  uint4 qf[KS];
  {
    const uint16_t* qp = static_cast<const uint16_t*>(a.q) + int64_t(tok_ok ? tok : 0) * a.ldq +
                         int64_t(head) * a.D;
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      const int d = s * 32 + grp * 8;
      qf[s] = make_uint4(0u, 0u, 0u, 0u);
      if (tok_ok && d < a.D) qf[s] = gload16(qp + d);
    }
  }

  f32x4_t o[DTILES];
#pragma unroll
  for (int t = 0; t < DTILES; ++t) o[t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  float m = kNegInf, l = 0.f;

  const int nblk = (w.k1 - w.k0 + kBlk - 1) / kBlk;
  const int mine = (nblk - wave + NW - 1) / NW;  // blocks wave, wave + NW, ...

  // offsets and masks of this wave's blocks first .. first + kTabBlocks - 1
  auto fill_table = [&](int first) {
#pragma unroll
    for (int e = 0; e < kTabBlocks * kBlk / 64; ++e) {
      const int idx = e * 64 + lane;
      const int key = w.k0 + ((first + (idx >> 5)) * NW + wave) * kBlk + (idx & 31);
      int64_t off = -1;
      if (key < w.k1) {
        const int pg = key / a.page_size, place = key - pg * a.page_size;
        const int id = w.pages[pg];
        if (id >= 0 && id < a.num_pages)
          off = int64_t(id) * a.page_stride + int64_t(place) * a.token_stride +
                int64_t(w.kvh) * a.head_stride;
      }
      L.off[idx] = off;
      const unsigned long long bits = __ballot(off >= 0);
      if (lane == 0) {
        L.mask[2 * e] = uint32_t(bits);
        L.mask[2 * e + 1] = uint32_t(bits >> 32);
      }
    }
    // the reads below are other lanes' writes (LDS operations of one wave complete in order)
    __builtin_amdgcn_wave_barrier();
    asm volatile("" ::: "memory");
  };
  // issues the loads of table block `tb` into buffer `buf`
  auto issue = [&](int tb, int buf) {
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int r = i * RPI + lane / CPR;
      const int64_t off = L.off[tb * kBlk + r];
      const int cs = lane % CPR;
      const int ck = cs ^ (r & (CPR - 1)), cv = cs ^ ((r & 7) << 1 & (CPR - 1));
      const bool ok = off >= 0;
      const void* kp = ok && ck * 8 < a.D ? static_cast<const void*>(kc + off + ck * 8) : &kZeroChunk;
      const void* vp = ok && cv * 8 < a.D ? static_cast<const void*>(vc + off + cv * 8) : &kZeroChunk;
      dma16(kp, __builtin_amdgcn_readfirstlane(lds_addr(&L.kv[buf][0][i * 512])));
      dma16(vp, __builtin_amdgcn_readfirstlane(lds_addr(&L.kv[buf][1][i * 512])));
    }
  };

  if (mine > 0) {
    fill_table(0);
    issue(0, 0);
  }
  for (int j = 0; j < mine; ++j) {
    const int buf = j & 1;
    const uint32_t mask = __builtin_amdgcn_readfirstlane(L.mask[j % kTabBlocks]);
    if (j + 1 < mine) {
      if ((j + 1) % kTabBlocks == 0) fill_table(j + 1);
      issue((j + 1) % kTabBlocks, buf ^ 1);
      vm_wait<2 * NI>();
    } else {
      vm_wait<0>();
    }
    asm volatile("" ::: "memory");
    const uint32_t kb = lds_addr(&L.kv[buf][0][0]), vb = lds_addr(&L.kv[buf][1][0]);
    // scores of 2 x 16 keys
    f32x4_t sc[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      sc[t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
      const int r = t * 16 + col;
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        const int c = (s * 4 + grp) ^ (r & (CPR - 1));
        sc[t] = mma_step<DT>(lds_read16(kb + uint32_t(r * DP * 2 + c * 16)), qf[s], sc[t]);
      }
    }
    float p[8];
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) p[t * 4 + i] = sc[t][i] * a.scale_log2;
    if (mask != 0xffffffffu) {
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (!((mask >> (t * 16 + grp * 4 + i)) & 1u)) p[t * 4 + i] = kNegInf;
    }
    float mx = p[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) mx = fmaxf(mx, p[i]);
    mx = fmaxf(mx, __shfl_xor(mx, 16, 64));
    mx = fmaxf(mx, __shfl_xor(mx, 32, 64));
    const float mn = fmaxf(m, mx);
    const float base = mn == kNegInf ? 0.f : mn;  // nothing visible yet: every p is exp2(-inf) = 0
    const float alpha = __builtin_amdgcn_exp2f(m - base);
    m = mn;
    uint32_t pk[4];
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      pk[i] = pack2<DT>(__builtin_amdgcn_exp2f(p[2 * i] - base), __builtin_amdgcn_exp2f(p[2 * i + 1] - base));
      sum += Traits<DT>::to_f32(uint16_t(pk[i])) + Traits<DT>::to_f32(uint16_t(pk[i] >> 16));
    }
    l = l * alpha + sum;
    const uint4 pf = make_uint4(pk[0], pk[1], pk[2], pk[3]);
    if (!__all(alpha == 1.f)) {
#pragma unroll
      for (int t = 0; t < DTILES; ++t) o[t] *= alpha;
    }
#pragma unroll
    for (int t = 0; t < DTILES; ++t) {
      const int r0 = grp * 4 + (col >> 2), r1 = r0 + 16;
      const int c = t * 2 + ((col & 3) >> 1), sub = (col & 1) * 8;
      const int c0 = c ^ ((r0 & 7) << 1 & (CPR - 1)), c1 = c ^ ((r1 & 7) << 1 & (CPR - 1));
      const s16x4_t v0 = lds_read_tr(vb + uint32_t(r0 * DP * 2 + c0 * 16 + sub));
      const s16x4_t v1 = lds_read_tr(vb + uint32_t(r1 * DP * 2 + c1 * 16 + sub));
      const uint2 u0 = __builtin_bit_cast(uint2, v0), u1 = __builtin_bit_cast(uint2, v1);
      o[t] = mma_step<DT>(make_uint4(u0.x, u0.y, u1.x, u1.y), pf, o[t]);
    }
    // this block's LDS reads are done before the next iteration's loads may overwrite the buffer
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  }
  l += __shfl_xor(l, 16, 64);
  l += __shfl_xor(l, 32, 64);

  // join the waves: a common maximum, scaled outputs summed through LDS
  if (grp == 0) s_ml[wave][col] = make_float2(m, l);
  __syncthreads();
  float mm = kNegInf;
#pragma unroll
  for (int x = 0; x < NW; ++x) mm = fmaxf(mm, s_ml[x][col].x);
  const float base = mm == kNegInf ? 0.f : mm;
  float ll = 0.f;
#pragma unroll
  for (int x = 0; x < NW; ++x) ll += s_ml[x][col].y * __builtin_amdgcn_exp2f(s_ml[x][col].x - base);
  const float f = __builtin_amdgcn_exp2f(m - base);
  // [16 rows][DP + 4] fp32 per wave, over the wave's own (now idle) buffers
  float* ob = reinterpret_cast<float*>(&L.kv[0][0][0]);
  static_assert(sizeof(L.kv) >= sizeof(float) * 16 * (DP + 4), "join buffer");
#pragma unroll
  for (int t = 0; t < DTILES; ++t)
#pragma unroll
    for (int i = 0; i < 4; ++i) ob[col * (DP + 4) + t * 16 + grp * 4 + i] = o[t][i] * f;
  __syncthreads();
  const int64_t rows_all = int64_t(a.T) * a.Hq;
  for (int e = int(threadIdx.x); e < 16 * DP; e += 64 * NW) {
    const int r = e / DP, d = e - r * DP;
    if (r >= w.nrows || d >= a.D) continue;
    float v = 0.f;
#pragma unroll
    for (int x = 0; x < NW; ++x)
      v += reinterpret_cast<const float*>(&s_wave[x].kv[0][0][0])[r * (DP + 4) + d];
    const int rr = w.row0 + r;
    const int64_t prow = int64_t(rr / a.grp) * a.Hq + w.kvh * a.grp + rr % a.grp;
    a.part_o[(int64_t(w.slot) * rows_all + prow) * a.D + d] = v;
  }
  if (wave == 0 && grp == 0 && row_ok) {
    const int64_t prow = int64_t(pos) * a.Hq + head;
    a.part_ml[int64_t(w.slot) * rows_all + prow] = make_float2(mm, ll);
  }
}

// Joins the key ranges of every (sorted position, query head): one wave per row.
template <int DT, int UNIT>
__global__ __launch_bounds__(256) void prefix_attn_join_kernel(PrefixAttnArgs a) {
  const int64_t row = int64_t(blockIdx.x) * 4 + wave_id();
  const int64_t rows_all = int64_t(a.T) * a.Hq;
  if (row >= rows_all) return;
  const int lane = int(threadIdx.x) & 63;
  const int i = int(row / a.Hq), h = int(row - int64_t(i) * a.Hq);
  const int end = seg_lo(a, a.G);
  if (i < seg_lo(a, 0) || i >= end) return;
  const int tok = a.permutation != nullptr ? a.permutation[i] : i;
  if (tok < 0 || tok >= a.T) return;
  int plen = 0, olen = 0;
  if (a.prefix_splits > 0) {
    int lo = 0, hi = a.G - 1;  // last segment that starts at or before i
    while (lo < hi) {
      const int mid = lo + (hi - lo + 1) / 2;
      if (seg_lo(a, mid) <= i) lo = mid; else hi = mid - 1;
    }
    plen = clamp_len(a.prefix_lens[lo], a.prefix_width, a.page_size);
  }
  if (a.own_splits > 0) olen = clamp_len(a.own_lens[tok], a.own_width, a.page_size);
  const int slots = a.prefix_splits + a.own_splits;
  auto used = [&](int s) {
    int k0, k1;
    if (s < a.prefix_splits) key_range(plen, a.prefix_splits, s, UNIT, &k0, &k1);
    else key_range(olen, a.own_splits, s - a.prefix_splits, UNIT, &k0, &k1);
    return k1 > k0;
  };
  float mm = kNegInf;
  for (int s = 0; s < slots; ++s)
    if (used(s)) mm = fmaxf(mm, a.part_ml[s * rows_all + row].x);
  const float base = mm == kNegInf ? 0.f : mm;
  float ll = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
  for (int s = 0; s < slots; ++s) {
    if (!used(s)) continue;
    const float2 ml = a.part_ml[s * rows_all + row];
    const float f = __builtin_amdgcn_exp2f(ml.x - base);
    ll += ml.y * f;
    const float* po = a.part_o + (s * rows_all + row) * a.D;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int d = e * 64 + lane;
      if (d < a.D) acc[e] += po[d] * f;
    }
  }
  const float inv = ll == 0.f ? 0.f : 1.f / ll;  // no visible key: zeros (a NaN sum stays NaN)
  uint16_t* op = static_cast<uint16_t*>(a.out) + int64_t(tok) * a.ldo + int64_t(h) * a.D;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int d = e * 64 + lane;
    if (d < a.D) op[d] = Traits<DT>::from_f32(acc[e] * inv);
  }
  if (a.lse != nullptr && lane == 0)
    a.lse[int64_t(tok) * a.Hq + h] = ll == 0.f ? kNegInf : (mm + __log2f(ll)) * 0.6931471805599453f;
}

int64_t cdiv64(int64_t a, int64_t b) { return (a + b - 1) / b; }

template <int DT, int DP>
hipError_t launch_dp(const PrefixAttnArgs& a, hipStream_t st) {
  constexpr int NW = attn_waves<DP>();
  const int64_t grid = int64_t(a.Hkv) * (int64_t(a.prefix_tiles) * a.prefix_splits +
                                         int64_t(a.T) * a.own_tiles * a.own_splits);
  if (grid > 0)
    hipLaunchKernelGGL((prefix_attn_kernel<DT, DP>), dim3(unsigned(grid)), dim3(64 * NW), 0, st, a);
  hipLaunchKernelGGL((prefix_attn_join_kernel<DT, kBlk * NW>),
                     dim3(unsigned(cdiv64(int64_t(a.T) * a.Hq, 4))), dim3(256), 0, st, a);
  return hipGetLastError();
}

}  // namespace

PrefixAttnPlan prefix_attention_plan(int64_t T, int G, int Hq, int Hkv, int D, int page_size,
                                     int64_t prefix_width, int64_t own_width) {
  PrefixAttnPlan p{};
  p.dp = D <= 64 ? 64 : D <= 128 ? 128 : 256;
  const int grp = Hq / Hkv;
  const int64_t pmax = prefix_width * page_size, omax = own_width * page_size;
  // enough key ranges for about 1024 workgroups, none shorter than 256 keys
  p.prefix_tiles = int(cdiv64(T * grp, 16) + G);
  p.own_tiles = int(cdiv64(grp, 16));
  auto splits = [](int64_t keys, int64_t wgs) {
    if (keys <= 0) return int64_t(0);
    const int64_t want = std::max<int64_t>(1, 1024 / std::max<int64_t>(wgs, 1));
    return std::max<int64_t>(1, std::min(want, cdiv64(keys, 256)));
  };
  p.prefix_splits = int(splits(pmax, int64_t(p.prefix_tiles) * Hkv));
  p.own_splits = int(splits(omax, T * p.own_tiles * Hkv));
  const int64_t rows = T * Hq, slots = p.prefix_splits + p.own_splits;
  p.part_ml = size_t(slots * rows * D * 4 + 255) & ~size_t(255);
  p.total = p.part_ml + size_t(slots * rows * 8);
  return p;
}

hipError_t launch_prefix_attention(int dtype, const PrefixAttnPlan& plan, const PrefixAttnArgs& a,
                                   hipStream_t st) {
  if (dtype == DT_BF16) {
    if (plan.dp == 64) return launch_dp<DT_BF16, 64>(a, st);
    if (plan.dp == 128) return launch_dp<DT_BF16, 128>(a, st);
    return launch_dp<DT_BF16, 256>(a, st);
  }
  if (plan.dp == 64) return launch_dp<DT_F16, 64>(a, st);
  if (plan.dp == 128) return launch_dp<DT_F16, 128>(a, st);
  return launch_dp<DT_F16, 256>(a, st);
}

}  // namespace lmx
