// Attention of a batch of query tokens over a paged key/value cache, where the tokens of a segment
// (one adapter's tokens: keys and values depend on the adapter) share a prefix.
//
// For sorted position i (token t = perm[i], segment g) and query head h, over the keys j of the
// segment's prefix followed by the token's own:
//     s_j = scale q_t,h . k_j,   o = sum_j exp(s_j - m) v_j / sum_j exp(s_j - m),   m = max_j s_j.
// Every (row tile, key head, key range) is one workgroup; the ranges of a row are joined by a second
// kernel. Statistics and outputs are fp32, scores in base 2. Two kinds of tiles run in one launch:
//
//   shared (tile_body)  128 query rows (token, head of the group) of one segment against a range of
//     its prefix, when segments have more than 32 rows on average (37 tokens of 7 heads a key head in 5
//     segments: 14 us, 18.8 with 16-row tiles): 4 waves of 32 rows walk the same 64-key blocks (32
//     for D > 128), staged once in LDS. 256 tokens over one 16k prefix run at 663 TFLOP/s; the matrix
//     pipe is about a quarter busy, the LDS as much, and the rest are waits of a wave's own chain
//     (scores, softmax, outputs), of which one workgroup per unit hides little.
//   rows (rows_body)    at most 16 rows: the heads of one token against its own keys, or the rows of a
//     short prefix tile. Bound by the bytes of the keys: each wave takes 16-key blocks of the range
//     in turn, with its own statistics, and the waves are joined in LDS at the end. 256 tokens with 1024
//     keys of their own (8 key heads of 128): 5.7 TB/s.
//
// Prefix workgroups come first, about one per compute unit, and leave half of each unit's LDS to
// the memory-bound ones that follow, which then run beside them.
//
// Matrix steps: scores transposed, S^T = K Q^T (K rows as the A operand, the queries as columns),
// so that a lane holds scores of ONE query and the softmax needs one or two cross-lane steps per
// block; O^T = V^T P^T takes those probabilities as its B operand as they lie (the contraction
// order over the keys is free as long as V uses the same), and V^T is read from the row-major block
// by the transposing LDS read.
// P is rounded to the storage type for the second product, and the sum of a row adds the rounded
// values, so the weights applied are normalised exactly.
//
// Keys and values go straight from the cache to LDS (16 bytes a lane); the addresses come from a
// table of key offsets in LDS, so that no page-list load sits in the way of the loads in flight. The
// 16-byte chunks of a key row are XOR-swizzled by the row (by the choice of the global chunk each
// lane fetches) so that rows at one chunk spread over the banks.
// A key whose page id lies outside the cache, or beyond its list's length, is masked: its offset is
// -1, its row is filled from a zero vector and its score is -inf. A range without keys leaves only its
// statistics, so that the join reads no lengths.
#include <algorithm>
#include <utility>

#include "device_common.hpp"
#include "prefix_attention.hpp"

namespace lmx {

namespace {

typedef short s16x4_t __attribute__((ext_vector_type(4)));

__device__ const uint4 kZeroChunk = {0u, 0u, 0u, 0u};

// The base of the exponentials follows the running maximum only when it lags by more than 2^4: weights
// up to 16 cost nothing in a floating type, and the outputs are rescaled a few times per range.
constexpr float kLag = 4.f;

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

typedef float f32x16_t __attribute__((ext_vector_type(16)));

template <int DT>
__device__ __forceinline__ f32x16_t mma32(uint4 a, uint4 b, f32x16_t acc) {
  if constexpr (DT == DT_BF16)
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, a),
                                                   __builtin_bit_cast(bf16x8_t, b), acc, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8_t, a),
                                                  __builtin_bit_cast(f16x8_t, b), acc, 0, 0, 0);
}

// Two fp32 values rounded to nearest even to the storage type, one instruction.
template <int DT>
__device__ __forceinline__ uint32_t cvt2(float a, float b) {
  typedef float f2 __attribute__((ext_vector_type(2)));
  const f2 v = {a, b};
  if constexpr (DT == DT_BF16) {
    typedef __bf16 b2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, b2));
  } else {
    typedef _Float16 h2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, h2));
  }
}

// acc + lo + hi of a packed pair, in fp32.
template <int DT>
__device__ __forceinline__ float add2(uint32_t p, float acc) {
  if constexpr (DT == DT_BF16) {
    typedef __bf16 b2 __attribute__((ext_vector_type(2)));
    return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(b2, p), __builtin_bit_cast(b2, 0x3f803f80u), acc, false);
  } else {
    typedef _Float16 h2 __attribute__((ext_vector_type(2)));
    return __builtin_amdgcn_fdot2(__builtin_bit_cast(h2, p), __builtin_bit_cast(h2, 0x3c003c00u), acc, false);
  }
}

// Eight query elements, negated for a negative scale (the kernels use its magnitude).
__device__ __forceinline__ uint4 signed_chunk(uint4 v, int negate) {
  const uint32_t f = negate ? 0x80008000u : 0u;
  return make_uint4(v.x ^ f, v.y ^ f, v.z ^ f, v.w ^ f);
}

// Maximum over the two lanes l and l ^ 32.
__device__ __forceinline__ float max_halves(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float add_halves(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

constexpr int kTileRows = 128;  // query rows of a shared tile: 32 per wave
constexpr int kRows = 16;       // of the others

// What one workgroup computes: rows of one segment or token, one key head, one key range.
struct Work {
  const int* pages;  // page list of the keys
  int len;           // keys of the whole list
  int k0, k1;        // key range of this workgroup
  int row0, nrows;   // flattened rows (sorted position * grp + head of the group) of the tile
  int slot;          // partial slot
  int kvh;
  bool shared;
};

__device__ __forceinline__ int clamp_len(int len, int width, int page) {
  const int64_t cap = int64_t(width) * page;
  return int(min(int64_t(max(len, 0)), cap));
}

// Key range of split `s`: equal shares rounded up to `unit` keys (a power of two).
__device__ __forceinline__ void key_range(int len, const FastDiv& n, int s, int unit, int* k0, int* k1) {
  const int per = (n.div(len + n.d - 1) + unit - 1) & -unit;
  const int64_t lo = int64_t(per) * s;
  *k0 = int(min(lo, int64_t(len)));
  *k1 = int(min(lo + per, int64_t(len)));
}

__device__ __forceinline__ int seg_lo(const PrefixAttnArgs& a, int g) {
  return min(max(a.seg_indptr[g], 0), a.T);
}

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// Decodes blockIdx into a Work. Prefix workgroups come first (they are the longest). Loads that do not
// depend on each other are issued together: this chain stands before the first key load.
__device__ __forceinline__ Work find_work(const PrefixAttnArgs& a, int b) {
  Work w{};
  const int np = a.prefix_tiles * a.prefix_splits * a.Hkv;
  if (b < np) {
    const int rest = a.by_kvh.div(b);
    w.kvh = b - rest * a.Hkv;
    int tile = a.by_prefix_splits.div(rest);
    w.slot = rest - tile * a.prefix_splits;
    w.shared = a.shared != 0;
    const int rows = w.shared ? kTileRows : kRows;
    // segment-major search for the row tile (every wave walks 64 segments at a time)
    const int lane = int(threadIdx.x) & 63;
    for (int g0 = 0; g0 < a.G; g0 += 64) {
      const int g = g0 + lane;
      int lo = 0, n = 0, len = 0;
      if (g < a.G) {
        lo = seg_lo(a, g);
        n = max(seg_lo(a, g + 1) - lo, 0);
        len = a.prefix_lens[g];
      }
      const int nt = (n * a.grp + rows - 1) / rows;
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
        const int lo_s = __builtin_amdgcn_readlane(lo, src), n_s = __builtin_amdgcn_readlane(n, src);
        const int gs = g0 + src, r0 = (tile - __builtin_amdgcn_readlane(excl, src)) * rows;
        w.row0 = lo_s * a.grp + r0;
        w.nrows = min(rows, n_s * a.grp - r0);
        w.pages = a.prefix_pages + int64_t(gs) * a.prefix_width;
        w.len = clamp_len(__builtin_amdgcn_readlane(len, src), a.prefix_width, a.page_size);
        key_range(w.len, a.by_prefix_splits, w.slot, a.prefix_unit, &w.k0, &w.k1);
        return w;
      }
      tile -= __builtin_amdgcn_readlane(incl, 63);
    }
    return w;
  }
  b -= np;
  int rest = a.by_kvh.div(b);
  w.kvh = b - rest * a.Hkv;
  const int r1 = a.by_own_tiles.div(rest), tile = rest - r1 * a.own_tiles;
  const int i = a.by_own_splits.div(r1), split = r1 - i * a.own_splits;  // i: sorted position, < T
  const int first = a.seg_indptr[0], last = a.seg_indptr[a.G];
  const int tok = a.permutation != nullptr ? a.permutation[i] : i;
  if (i < first || i >= last || tok < 0 || tok >= a.T) return w;
  w.slot = a.prefix_splits + split;
  w.row0 = i * a.grp + tile * kRows;
  w.nrows = min(kRows, a.grp - tile * kRows);
  w.pages = a.own_pages + int64_t(tok) * a.own_width;
  w.len = clamp_len(a.own_lens[tok], a.own_width, a.page_size);
  key_range(w.len, a.by_own_splits, split, a.own_unit, &w.k0, &w.k1);
  return w;
}

template <int DT>
__device__ __forceinline__ f32x4_t mma16(uint2 a, uint2 b, f32x4_t acc) {
  if constexpr (DT == DT_BF16) {
    return __builtin_amdgcn_mfma_f32_16x16x16bf16_1k(__builtin_bit_cast(s16x4_t, a),
                                                     __builtin_bit_cast(s16x4_t, b), acc, 0, 0, 0);
  } else {
    typedef _Float16 f16x4_t __attribute__((ext_vector_type(4)));
    return __builtin_amdgcn_mfma_f32_16x16x16f16(__builtin_bit_cast(f16x4_t, a),
                                                 __builtin_bit_cast(f16x4_t, b), acc, 0, 0, 0);
  }
}

// Maximum over the lanes l ^ 16 k.
__device__ __forceinline__ float max_groups(float v) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return max_halves(fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1])));
}
__device__ __forceinline__ float add_groups(float v) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return add_halves(__uint_as_float(r[0]) + __uint_as_float(r[1]));
}

// Maximum and sum over the wave, in every lane.
__device__ __forceinline__ float max_wave(float v) {
#pragma unroll
  for (int d = 1; d < 16; d <<= 1) v = fmaxf(v, __shfl_xor(v, d, 64));
  return max_groups(v);
}
__device__ __forceinline__ float add_wave(float v) {
#pragma unroll
  for (int d = 1; d < 16; d <<= 1) v += __shfl_xor(v, d, 64);
  return add_groups(v);
}

// Four output elements of one row, to be followed by their row's other pieces.
template <int DT>
__device__ __forceinline__ void store_out(const PrefixAttnArgs& a, int tok, int head, int d, float4 v) {
  uint16_t* op = static_cast<uint16_t*>(a.out) + int64_t(tok) * a.ldo + int64_t(head) * a.D + d;
  const uint32_t lo = cvt2<DT>(v.x, v.y), hi = cvt2<DT>(v.z, v.w);
  if (a.out8) {
    *reinterpret_cast<uint2*>(op) = make_uint2(lo, hi);
  } else {
    op[0] = uint16_t(lo);
    op[1] = uint16_t(lo >> 16);
    op[2] = uint16_t(hi);
    op[3] = uint16_t(hi >> 16);
  }
}
__device__ __forceinline__ void store_lse(const PrefixAttnArgs& a, int tok, int head, float m, float l) {
  if (a.lse != nullptr)
    a.lse[int64_t(tok) * a.Hq + head] = l == 0.f ? kNegInf : (m + __log2f(l)) * 0.6931471805599453f;
}
// Of a row's sum: no visible key gives zeros (a NaN sum stays NaN).
__device__ __forceinline__ float inverse(float l) { return l == 0.f ? 0.f : 1.f / l; }

constexpr int kWaves = 4;
constexpr int kTabKeys = 256;  // keys covered by one fill of a wave's offset table

// Row tile of at most 16 query rows, its keys split over the waves in 16-key blocks. LDS of one wave:
// a ring of K and V blocks, the offsets of its next 256 keys and their validity.
template <int DP>
struct RowsWave {
  static constexpr int kBufs = DP > 64 ? 2 : 4;
  uint16_t kv[kBufs][2][16 * DP];
  int64_t off[kTabKeys];
  uint64_t mask[kTabKeys / 64];
};
template <int DP>
struct RowsLds {
  RowsWave<DP> wave[kWaves];
  float2 ml[kWaves][16];
  float inv[16];
};

template <int DT, int DP, bool DIRECT>
__device__ __forceinline__ void rows_body(const PrefixAttnArgs& a, const Work& w, RowsLds<DP>& S) {
  constexpr int NB = RowsWave<DP>::kBufs;
  constexpr int CPR = DP / 8;         // 16-byte chunks per key row
  constexpr int RPI = 64 / CPR;       // key rows one DMA instruction covers
  constexpr int NI = 16 / RPI;        // DMA instructions per block and operand
  constexpr int KS = DP / 32;         // reduction steps of the scores
  constexpr int DTILES = DP / 16;     // 16-row tiles of O^T
  constexpr int TB = kTabKeys / 16;

  const int lane = int(threadIdx.x) & 63, wave = wave_id();
  const int col = lane & 15, grp = lane >> 4;
  RowsWave<DP>& L = S.wave[wave];
  const uint16_t* kc = static_cast<const uint16_t*>(a.k_cache);
  const uint16_t* vc = static_cast<const uint16_t*>(a.v_cache);

  const int nblk = (w.k1 - w.k0 + 15) / 16;
  const int mine = (nblk - wave + kWaves - 1) / kWaves;  // blocks wave, wave + 4, ...

  // offsets and validity of this wave's blocks first .. first + TB - 1
  auto fill_table = [&](int first) {
#pragma unroll
    for (int e = 0; e < kTabKeys / 64; ++e) {
      const int idx = e * 64 + lane;
      const int key = w.k0 + ((first + (idx >> 4)) * kWaves + wave) * 16 + (idx & 15);
      int64_t off = -1;
      if (key < w.k1) {
        const int pg = a.by_page.div(key), place = key - pg * a.page_size;
        const int id = w.pages[pg];
        if (id >= 0 && id < a.num_pages)
          off = int64_t(id) * a.page_stride + int64_t(place) * a.token_stride +
                int64_t(w.kvh) * a.head_stride;
      }
      L.off[idx] = off;
      const unsigned long long bits = __ballot(off >= 0);
      if (lane == 0) L.mask[e] = bits;
    }
    // the reads below are other lanes' writes (LDS operations of one wave complete in order)
    __builtin_amdgcn_wave_barrier();
    asm volatile("" ::: "memory");
  };
  auto issue = [&](int j) {
    const int tb = j % TB, buf = j % NB;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int r = i * RPI + lane / CPR;
      const int64_t off = L.off[tb * 16 + r];
      const int cs = lane % CPR;
      const int ck = cs ^ (r & (CPR - 1)), cv = cs ^ (((r & 7) << 1) & (CPR - 1));
      const bool ok = off >= 0;
      const void* kp = ok && ck * 8 < a.D ? static_cast<const void*>(kc + off + ck * 8) : &kZeroChunk;
      const void* vp = ok && cv * 8 < a.D ? static_cast<const void*>(vc + off + cv * 8) : &kZeroChunk;
      dma16(kp, __builtin_amdgcn_readfirstlane(lds_addr(&L.kv[buf][0][i * 512])));
      dma16(vp, __builtin_amdgcn_readfirstlane(lds_addr(&L.kv[buf][1][i * 512])));
    }
  };
  // A block whose issue crosses into the next table fill finds the table free: the masks of earlier
  // blocks are read when they are issued.
  uint32_t masks[NB];
  auto start = [&](int j, uint32_t& mask) {
    if (j % TB == 0) fill_table(j);
    mask = uint32_t(uniform(int(uint32_t(L.mask[(j % TB) / 4] >> (16 * (j & 3)))))) & 0xffffu;
    issue(j);
  };

  // the query column of this lane
  const bool row_ok = col < w.nrows;
  const int row = w.row0 + min(col, w.nrows - 1);
  const int pos = a.by_grp.div(row), head = w.kvh * a.grp + row - pos * a.grp;
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
      if (tok_ok && d < a.D) qf[s] = signed_chunk(gload16(qp + d), a.negate);
    }
  }
  f32x4_t o[DTILES];
#pragma unroll
  for (int t = 0; t < DTILES; ++t) o[t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  float m = kNegInf, l = 0.f;

  auto compute = [&](int buf, uint32_t mask) {
    const uint32_t kb = lds_addr(&L.kv[buf][0][0]), vb = lds_addr(&L.kv[buf][1][0]);
    f32x4_t sc = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      const int c = (s * 4 + grp) ^ (col & (CPR - 1));
      sc = mma_step<DT>(lds_read16(kb + uint32_t(col * DP * 2 + c * 16)), qf[s], sc);
    }
    if (mask != 0xffffu) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (!((mask >> (grp * 4 + i)) & 1u)) sc[i] = kNegInf;
    }
    const float mx = max_groups(fmaxf(fmaxf(sc[0], sc[1]), fmaxf(sc[2], sc[3]))) * a.scale_log2;
    const bool lag = mx > m + kLag;
    if (__any(lag)) {
      const float mn = lag ? mx : m;
      const float alpha = mn == kNegInf ? 1.f : __builtin_amdgcn_exp2f(m - mn);
      l *= alpha;
#pragma unroll
      for (int t = 0; t < DTILES; ++t) o[t] *= alpha;
      m = mn;
    }
    const float base = m == kNegInf ? 0.f : m;  // nothing visible yet: every weight is exp2(-inf) = 0
    uint32_t pk[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      pk[i] = cvt2<DT>(__builtin_amdgcn_exp2f(fmaf(sc[2 * i], a.scale_log2, -base)),
                       __builtin_amdgcn_exp2f(fmaf(sc[2 * i + 1], a.scale_log2, -base)));
      l = add2<DT>(pk[i], l);
    }
    const int r = grp * 4 + (col >> 2), sub = (col & 1) * 8;
#pragma unroll
    for (int t = 0; t < DTILES; ++t) {
      const int c = (t * 2 + ((col & 3) >> 1)) ^ (((r & 7) << 1) & (CPR - 1));
      const uint2 v = __builtin_bit_cast(uint2, lds_read_tr(vb + uint32_t(r * DP * 2 + c * 16 + sub)));
      o[t] = mma16<DT>(v, make_uint2(pk[0], pk[1]), o[t]);
    }
    // this block's LDS reads are done before a later load may overwrite the buffer
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  };

#pragma unroll
  for (int j = 0; j < NB - 1; ++j)
    if (j < mine) start(j, masks[j]);
  for (int j0 = 0; j0 < mine; j0 += NB) {
#pragma unroll
    for (int u = 0; u < NB; ++u) {
      const int j = j0 + u;
      if (j < mine) {
        if (j + NB - 1 < mine) {
          start(j + NB - 1, masks[(u + NB - 1) % NB]);
          vm_wait<(NB - 1) * 2 * NI>();
        } else {
          vm_wait<0>();
        }
        asm volatile("" ::: "memory");
        compute(u, masks[u]);
      }
    }
  }
  l = add_groups(l);

  // join the waves: a common maximum, scaled outputs summed through LDS
  if (grp == 0) S.ml[wave][col] = make_float2(m, l);
  __syncthreads();
  float mm = kNegInf;
#pragma unroll
  for (int x = 0; x < kWaves; ++x) mm = fmaxf(mm, S.ml[x][col].x);
  const float base = mm == kNegInf ? 0.f : mm;
  float ll = 0.f;
#pragma unroll
  for (int x = 0; x < kWaves; ++x) ll += S.ml[x][col].y * __builtin_amdgcn_exp2f(S.ml[x][col].x - base);
  const float f = __builtin_amdgcn_exp2f(m - base);
  if (DIRECT && wave == 0 && grp == 0) S.inv[col] = inverse(ll);
  // [16 rows][DP + 4] fp32 per wave, over the wave's own (now idle) buffers and table
  constexpr int OP = DP + 4;
  static_assert(sizeof(RowsWave<DP>) >= sizeof(float) * 16 * OP, "join buffer");
  float* ob = reinterpret_cast<float*>(&L);
#pragma unroll
  for (int t = 0; t < DTILES; ++t)
    *reinterpret_cast<float4*>(ob + col * OP + t * 16 + grp * 4) = make_float4(o[t][0] * f, o[t][1] * f, o[t][2] * f, o[t][3] * f);
  __syncthreads();
  const int64_t rows_all = int64_t(a.T) * a.Hq;
  for (int e = int(threadIdx.x); e < 16 * DP / 4; e += 64 * kWaves) {
    const int r = e / (DP / 4), d = (e - r * (DP / 4)) * 4;
    if (r >= w.nrows || d >= a.D) continue;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int x = 0; x < kWaves; ++x) {
      const float4 u = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(&S.wave[x]) + r * OP + d);
      v.x += u.x; v.y += u.y; v.z += u.z; v.w += u.w;
    }
    const int rr = w.row0 + r;
    const int rp = a.by_grp.div(rr), rh = w.kvh * a.grp + rr - rp * a.grp;
    if constexpr (DIRECT) {  // the only range of its row
      const float inv = S.inv[r];
      store_out<DT>(a, a.permutation != nullptr ? a.permutation[rp] : rp, rh, d,
                    make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv));
      continue;
    }
    const int64_t prow = int64_t(rp) * a.Hq + rh;
    *reinterpret_cast<float4*>(a.part_o + (int64_t(w.slot) * rows_all + prow) * a.D + d) = v;
  }
  if (wave == 0 && grp == 0 && row_ok) {
    if constexpr (DIRECT) store_lse(a, tok, head, mm, ll);
    else a.part_ml[int64_t(w.slot) * rows_all + int64_t(pos) * a.Hq + head] = make_float2(mm, ll);
  }
}


template <int DP>
constexpr int tile_block() { return DP > 128 ? 32 : 64; }

// LDS of a shared tile: two buffers of a K and a V block, the byte offsets of the keys (two halves of
// 512) and their validity. The blocks come first and stay below 64 KiB, so that every read of them is one
// lane address and a constant offset.
template <int DP>
struct TileLds {
  static constexpr int kBlockBytes = tile_block<DP>() * DP * 2;
  unsigned char kv[2][2][kBlockBytes];  // [buffer][K, V]
  int64_t off[2][512];
  uint64_t mask[2][8];
};

// 16 bytes, or the transposing read, at lane address `p` plus a constant.
typedef __attribute__((address_space(3))) unsigned char lds_byte;
template <int OFF>
__device__ __forceinline__ uint4 tile_read16(lds_byte* p) {
  typedef unsigned int u32x4_t __attribute__((ext_vector_type(4)));
  typedef __attribute__((address_space(3))) u32x4_t lds_t;
  const u32x4_t v = *reinterpret_cast<lds_t*>(p + OFF);
  return make_uint4(v.x, v.y, v.z, v.w);
}
template <int OFF>
__device__ __forceinline__ uint2 tile_read_tr(lds_byte* p) {
  typedef __attribute__((address_space(3))) s16x4_t lds_t;
  return __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(reinterpret_cast<lds_t*>(p + OFF)));
}

template <int N, typename F>
__device__ __forceinline__ void static_for(F f) {
  [&]<int... I>(std::integer_sequence<int, I...>) { (f(std::integral_constant<int, I>{}), ...); }
  (std::make_integer_sequence<int, N>{});
}

// Shared prefix tile: 4 waves of 32 query rows each walk the same key blocks, staged once in LDS for
// all of them (double buffered, one barrier a block). Per block and wave (D 128, 64 keys) there are 32
// matrix steps of 32 cycles and about 170 vector instructions (32 exponentials among them). A block's
// offsets are read one block ahead, K fragments before the next loads are issued and V fragments before
// the softmax, so that LDS latency passes under other work: 508 TFLOP/s without any of that (256 tokens
// over a 16k prefix), 618 with the fragments, 663 with the offsets. Reading all 8 K steps ahead spills
// (318); forming the next scores beside the softmax in the same wave was slower too (480).
template <int DT, int DP>
__device__ __forceinline__ void tile_body(const PrefixAttnArgs& a, const Work& w, TileLds<DP>& S) {
  constexpr int BK = tile_block<DP>();
  constexpr int CPR = DP / 8, RPI = 64 / CPR;
  constexpr int NI = BK / RPI / 4;      // DMA instructions per wave, block and operand
  constexpr int KT = BK / 32, KS = DP / 16, DTILES = DP / 32, PK = BK / 16;
  constexpr int TB = 512 / BK;          // blocks per half of the offset table
  constexpr int BB = TileLds<DP>::kBlockBytes;
  // Chunk swizzles by LDS row; both are the same for every row a lane loads (rows wave * RPI + lane /
  // CPR + 4 RPI i).
  constexpr int KM = DP == 128 ? 15 : 7;
  static_assert((4 * RPI) % (KM + 1) == 0 && (4 * RPI) % 8 == 0, "swizzle constant over a lane's rows");

  const int lane = int(threadIdx.x) & 63, wave = wave_id();
  const int col = lane & 31, half = lane >> 5;

  const int r = wave * 32 + col;
  const bool row_ok = r < w.nrows;
  const int row = w.row0 + min(r, w.nrows - 1);
  const int pos = a.by_grp.div(row), head = w.kvh * a.grp + row - pos * a.grp;
  const int tok = a.permutation != nullptr ? a.permutation[pos] : pos;
  const bool tok_ok = row_ok && tok >= 0 && tok < a.T;
  uint4 qf[KS];
  {
    const uint16_t* qp = static_cast<const uint16_t*>(a.q) + int64_t(tok_ok ? tok : 0) * a.ldq +
                         int64_t(head) * a.D;
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      const int d = s * 16 + half * 8;
      qf[s] = make_uint4(0u, 0u, 0u, 0u);
      if (tok_ok && d < a.D) qf[s] = signed_chunk(gload16(qp + d), a.negate);
    }
  }
  f32x16_t o[DTILES];
#pragma unroll
  for (int t = 0; t < DTILES; ++t)
#pragma unroll
    for (int i = 0; i < 16; ++i) o[t][i] = 0.f;
  float m = kNegInf, l = 0.f;
  const bool busy = wave * 32 < w.nrows;  // waves without a row only help loading

  const int nblk = (w.k1 - w.k0 + BK - 1) / BK;
  // Page ids of the 512 keys from block `first` on: loaded here, two keys a thread, ...
  auto load_ids = [&](int first, int* id) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int key = w.k0 + first * BK + e * 256 + int(threadIdx.x);
      id[e] = key < w.k1 ? w.pages[a.by_page.div(key)] : -1;
    }
  };
  // ... and turned into byte offsets and masks in half `h` of the table here.
  auto fill_table = [&](int first, int h, const int* id) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int idx = e * 256 + int(threadIdx.x);
      const int key = w.k0 + first * BK + idx;
      const int place = key - a.by_page.div(key) * a.page_size;
      const bool ok = id[e] >= 0 && id[e] < a.num_pages;
      S.off[h][idx] = ok ? 2 * (int64_t(id[e]) * a.page_stride + int64_t(place) * a.token_stride +
                                int64_t(w.kvh) * a.head_stride)
                         : int64_t(-1);
      const unsigned long long bits = __ballot(ok);
      if (lane == 0) S.mask[h][e * 4 + wave] = bits;
    }
  };
  const int lrow = wave * RPI + lane / CPR, cs = lane % CPR;
  // Mask and offsets of the next block to load, read from LDS a block ahead of their use.
  int64_t off[NI];
  uint64_t raw_mask;
  auto look_up = [&](int j) {
    raw_mask = S.mask[(j / TB) & 1][j % TB * BK / 64];
    const int64_t* t = &S.off[(j / TB) & 1][(j % TB) * BK + lrow];
#pragma unroll
    for (int i = 0; i < NI; ++i) off[i] = t[i * 4 * RPI];
  };
  auto block_mask = [&](int j) {
    const uint32_t lo = uint32_t(uniform(int(uint32_t(raw_mask)))), hi = uint32_t(uniform(int(uint32_t(raw_mask >> 32))));
    if constexpr (BK == 64) return uint64_t(lo) | (uint64_t(hi) << 32);
    else return uint64_t((j & 1) ? hi : lo);
  };
  constexpr uint64_t kFull = BK == 64 ? ~uint64_t(0) : uint64_t(0xffffffffu);

  const int ck = cs ^ (lrow & KM), cv = cs ^ (((lrow & 7) << 1) & (CPR - 1));
  const bool k_in = ck * 8 < a.D, v_in = cv * 8 < a.D, whole = a.D == DP;
  const char* kbase = static_cast<const char*>(a.k_cache) + ck * 16;
  const char* vbase = static_cast<const char*>(a.v_cache) + cv * 16;
  const uint32_t lds0 = uint32_t(uniform(int(lds_addr(&S.kv[0][0][0])))) + wave * 1024;
  auto issue = [&](uint64_t mask, auto buf) {
    constexpr uint32_t kOff = buf.value * 2 * BB, vOff = kOff + BB;
    if (whole && mask == kFull) {
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        dma16(kbase + off[i], lds0 + kOff + i * 4096);
        dma16(vbase + off[i], lds0 + vOff + i * 4096);
      }
    } else {
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const void* kp = off[i] >= 0 && k_in ? static_cast<const void*>(kbase + off[i]) : &kZeroChunk;
        const void* vp = off[i] >= 0 && v_in ? static_cast<const void*>(vbase + off[i]) : &kZeroChunk;
        dma16(kp, lds0 + kOff + i * 4096);
        dma16(vp, lds0 + vOff + i * 4096);
      }
    }
  };

  // Lane addresses of the fragments: K row col, chunk 2 s + half; V row 4 half + q4 / 4 of 16 keys, the
  // 4 columns of q4 % 4 in the 16 of this lane group of 32-column tile t. The swizzle is an XOR, and so
  // is the step s or t: one address each, as the LDS is aligned beyond a row.
  const uint32_t lds = uint32_t(uniform(int(lds_addr(&S.kv[0][0][0]))));
  const uint32_t kaddr = lds + col * DP * 2 + (half ^ (col & KM)) * 16;
  uint32_t vaddr;
  {
    const int q4 = lane & 15, vr = half * 4 + (q4 >> 2);
    const int c = ((lane >> 4) & 1) * 2 + ((q4 & 3) >> 1);
    vaddr = lds + vr * DP * 2 + (c ^ (((vr & 7) << 1) & (CPR - 1))) * 16 + (q4 & 1) * 8;
  }

  constexpr int kAhead = 4;  // K steps read ahead
  uint4 kf[kAhead][KT];
  auto read_k = [&](auto buf, auto s) {
    static_for<KT>([&](auto t) {
      kf[s.value % kAhead][t.value] = tile_read16<buf.value * 2 * BB + t.value * 32 * DP * 2>(reinterpret_cast<lds_byte*>(kaddr ^ (s.value * 32)));
    });
  };
  auto compute = [&](uint64_t mask, auto buf) {
    constexpr int vOff = buf.value * 2 * BB + BB;
    f32x16_t sc[KT];
#pragma unroll
    for (int t = 0; t < KT; ++t)
#pragma unroll
      for (int i = 0; i < 16; ++i) sc[t][i] = 0.f;
    static_for<KS>([&](auto s) {
#pragma unroll
      for (int t = 0; t < KT; ++t) sc[t] = mma32<DT>(kf[s.value % kAhead][t], qf[s.value], sc[t]);
      if constexpr (s.value + kAhead < KS) read_k(buf, std::integral_constant<int, s.value + kAhead>{});
      __builtin_amdgcn_sched_barrier(0);
    });
    // V fragments of the first 32 keys, read under the softmax
    uint4 vf[2][DTILES];
    static_for<2>([&](auto kk) {
      static_for<DTILES>([&](auto t) {
        const uint2 u0 = tile_read_tr<vOff + kk.value * 16 * DP * 2>(reinterpret_cast<lds_byte*>(vaddr ^ (t.value * 64)));
        const uint2 u1 = tile_read_tr<vOff + (kk.value * 16 + 8) * DP * 2>(reinterpret_cast<lds_byte*>(vaddr ^ (t.value * 64)));
        vf[kk.value][t.value] = make_uint4(u0.x, u0.y, u1.x, u1.y);
      });
    });
    __builtin_amdgcn_sched_barrier(0);
    if (mask != kFull) {
#pragma unroll
      for (int t = 0; t < KT; ++t) {
        const uint32_t mine = uint32_t(mask >> (32 * t)) >> (4 * half);  // register i: key 8 (i / 4) + 4 half + i % 4
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (!((mine >> (8 * (i / 4) + i % 4)) & 1u)) sc[t][i] = kNegInf;
      }
    }
    float mx = sc[0][0];
#pragma unroll
    for (int t = 0; t < KT; ++t)
#pragma unroll
      for (int i = 0; i < 16; ++i) mx = fmaxf(mx, sc[t][i]);
    mx = max_halves(mx) * a.scale_log2;
    const bool lag = mx > m + kLag;
    if (__any(lag)) {
      const float mn = lag ? mx : m;
      const float alpha = mn == kNegInf ? 1.f : __builtin_amdgcn_exp2f(m - mn);
      l *= alpha;
#pragma unroll
      for (int t = 0; t < DTILES; ++t) o[t] *= alpha;
      m = mn;
    }
    const float base = m == kNegInf ? 0.f : m;
    uint4 pf[PK];
#pragma unroll
    for (int kk = 0; kk < PK; ++kk) {
      uint32_t pk[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float s0 = sc[kk / 2][(kk % 2) * 8 + 2 * i], s1 = sc[kk / 2][(kk % 2) * 8 + 2 * i + 1];
        pk[i] = cvt2<DT>(__builtin_amdgcn_exp2f(fmaf(s0, a.scale_log2, -base)),
                         __builtin_amdgcn_exp2f(fmaf(s1, a.scale_log2, -base)));
        l = add2<DT>(pk[i], l);
      }
      pf[kk] = make_uint4(pk[0], pk[1], pk[2], pk[3]);
    }
    static_for<PK>([&](auto kk) {
      static_for<DTILES>([&](auto t) {
        o[t.value] = mma32<DT>(vf[kk.value & 1][t.value], pf[kk.value], o[t.value]);
        if constexpr (kk.value + 2 < PK) {
          const uint2 u0 = tile_read_tr<vOff + (kk.value + 2) * 16 * DP * 2>(reinterpret_cast<lds_byte*>(vaddr ^ (t.value * 64)));
          const uint2 u1 = tile_read_tr<vOff + ((kk.value + 2) * 16 + 8) * DP * 2>(reinterpret_cast<lds_byte*>(vaddr ^ (t.value * 64)));
          vf[kk.value & 1][t.value] = make_uint4(u0.x, u0.y, u1.x, u1.y);
        }
      });
    });
  };

  int ids[2];
  load_ids(0, ids);
  fill_table(0, 0, ids);
  __syncthreads();
  look_up(0);
  uint64_t mask = block_mask(0), next = 0;
  issue(mask, std::integral_constant<int, 0>{});
  look_up(1);
  auto step = [&](int j, auto buf) {
    vm_wait<0>();
    __syncthreads();  // block j is in LDS, and nobody reads the other buffer any more
    if (busy) static_for<kAhead>([&](auto s) { read_k(buf, s); });
    __builtin_amdgcn_sched_barrier(0);
    const bool refill = j % TB == TB - 3 && j + 3 < nblk;
    if (refill) load_ids(j + 3, ids);
    if (j + 1 < nblk) {
      next = block_mask(j + 1);
      issue(next, std::integral_constant<int, 1 - buf.value>{});
      look_up(j + 2);  // not used beyond the last block
    }
    if (busy) compute(mask, buf);
    if (refill) fill_table(j + 3, ((j / TB) & 1) ^ 1, ids);
    mask = next;
  };
  for (int j = 0; j < nblk; j += 2) {
    step(j, std::integral_constant<int, 0>{});
    if (j + 1 < nblk) step(j + 1, std::integral_constant<int, 1>{});
  }
  l = add_halves(l);
  if (!row_ok) return;
  const int64_t rows_all = int64_t(a.T) * a.Hq, prow = int64_t(pos) * a.Hq + head;
  float* po = a.part_o + (int64_t(w.slot) * rows_all + prow) * a.D;
#pragma unroll
  for (int t = 0; t < DTILES; ++t)
#pragma unroll
    for (int i = 0; i < 16; i += 4) {
      const int d = t * 32 + 8 * (i / 4) + 4 * half;
      if (d < a.D) *reinterpret_cast<float4*>(po + d) = make_float4(o[t][i], o[t][i + 1], o[t][i + 2], o[t][i + 3]);
    }
  if (half == 0) a.part_ml[int64_t(w.slot) * rows_all + prow] = make_float2(m, l);
}

// One workgroup per (row tile, key head, key range); LDS is whichever layout its tile needs. DIRECT: no
// prefix and one range per row, which goes to the output at once (256 tokens with 1024 keys each: 191 us,
// 206 with a plane and the join).
template <int DT, int DP, bool DIRECT>
__global__ __launch_bounds__(256, DP > 128 ? 1 : 2) void prefix_attn_kernel(PrefixAttnArgs a) {
  constexpr size_t kLds = DIRECT || sizeof(RowsLds<DP>) > sizeof(TileLds<DP>) ? sizeof(RowsLds<DP>) : sizeof(TileLds<DP>);
  __shared__ __align__(1024) unsigned char s_mem[kLds];
  const Work w = find_work(a, int(blockIdx.x));
  if (w.k1 <= w.k0) {  // no keys in this range: its rows say so to the join, or are zeros
    const int64_t rows_all = int64_t(a.T) * a.Hq;
    for (int r = int(threadIdx.x); r < w.nrows; r += 64 * kWaves) {
      const int row = w.row0 + r, pos = a.by_grp.div(row), head = w.kvh * a.grp + row - pos * a.grp;
      if constexpr (DIRECT) {
        const int tok = a.permutation != nullptr ? a.permutation[pos] : pos;
        for (int d = 0; d < a.D; d += 4) store_out<DT>(a, tok, head, d, make_float4(0.f, 0.f, 0.f, 0.f));
        store_lse(a, tok, head, kNegInf, 0.f);
      } else {
        a.part_ml[int64_t(w.slot) * rows_all + int64_t(pos) * a.Hq + head] = make_float2(kNegInf, 0.f);
      }
    }
    return;
  }
  if constexpr (!DIRECT) {
    if (w.shared) {
      tile_body<DT, DP>(a, w, *reinterpret_cast<TileLds<DP>*>(s_mem));
      return;
    }
  }
  rows_body<DT, DP, DIRECT>(a, w, *reinterpret_cast<RowsLds<DP>*>(s_mem));
}

// Joins the key ranges of every (sorted position, query head): one wave per row. 64 ranges at a
// time, a lane holds the statistics of one; then 16-byte pieces of the partial rows, as many ranges at
// once as rows of D fit the wave, four loads in flight.
template <int DT>
__global__ __launch_bounds__(256) void prefix_attn_join_kernel(PrefixAttnArgs a) {
  const int64_t rows_all = int64_t(a.T) * a.Hq;
  const int row = int(blockIdx.x) * 4 + wave_id();  // T * Hq <= 2^26
  if (row >= rows_all) return;
  const int lane = int(threadIdx.x) & 63;
  const int i = a.by_hq.div(row), h = row - i * a.Hq;
  const int n = a.prefix_splits + a.own_splits;
  float2 ml = make_float2(kNegInf, 0.f);
  if (lane < n) ml = a.part_ml[lane * rows_all + row];
  const int first = a.seg_indptr[0], last = a.seg_indptr[a.G];
  const int tok = a.permutation != nullptr ? a.permutation[i] : i;
  if (i < first || i >= last || tok < 0 || tok >= a.T) return;

  const int pieces = a.D / 4, per = pieces > 32 ? 1 : 64 / pieces;  // rows of D a wave loads at once
  const int sub = lane / pieces, piece = lane - sub * pieces;
  const bool loads = sub < per;
  float mm = kNegInf, ll = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int s0 = 0; s0 < n; s0 += 64) {
    if (s0 > 0) {
      ml = make_float2(kNegInf, 0.f);
      if (s0 + lane < n) ml = a.part_ml[(s0 + lane) * rows_all + row];
    }
    const float mx = max_wave(ml.x);
    const float mn = fmaxf(mm, mx), base = mn == kNegInf ? 0.f : mn;
    const float old = __builtin_amdgcn_exp2f(mm - base);
    mm = mn;
    const float f = __builtin_amdgcn_exp2f(ml.x - base);
    ll = ll * old + add_wave(ml.y * f);
    acc.x *= old; acc.y *= old; acc.z *= old; acc.w *= old;
    // the ranges without keys (sum 0) hold no outputs; a NaN sum counts
    const unsigned long long used = __ballot(!(ml.y == 0.f));
    const int cnt = min(64, n - s0);
    for (int c = 0; c < cnt; c += 4 * per) {
      float4 v[4];
      float g[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int s = c + u * per + sub;
        const bool ok = loads && s < cnt && ((used >> (s & 63)) & 1);
        g[u] = __shfl(f, s & 63, 64);
        if (!ok) g[u] = 0.f;
        v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (ok) v[u] = *reinterpret_cast<const float4*>(a.part_o + ((s0 + s) * rows_all + row) * a.D + piece * 4);
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        acc.x += v[u].x * g[u]; acc.y += v[u].y * g[u]; acc.z += v[u].z * g[u]; acc.w += v[u].w * g[u];
      }
    }
  }
  // lanes piece, piece + pieces, .. hold shares of the same outputs: added in order into the first
  float4 tot = acc;
  for (int s = 1; s < per; ++s) {
    const int src = (piece + s * pieces) & 63;
    tot.x += __shfl(acc.x, src, 64); tot.y += __shfl(acc.y, src, 64);
    tot.z += __shfl(acc.z, src, 64); tot.w += __shfl(acc.w, src, 64);
  }
  const float inv = inverse(ll);
  if (lane < pieces) store_out<DT>(a, tok, h, lane * 4, make_float4(tot.x * inv, tot.y * inv, tot.z * inv, tot.w * inv));
  if (lane == 0) store_lse(a, tok, h, mm, ll);
}

int64_t cdiv64(int64_t a, int64_t b) { return (a + b - 1) / b; }

template <int DT, int DP>
hipError_t launch_dp(const PrefixAttnArgs& a, hipStream_t st) {
  const int64_t grid = int64_t(a.Hkv) * (int64_t(a.prefix_tiles) * a.prefix_splits +
                                         int64_t(a.T) * a.own_tiles * a.own_splits);
  if (a.direct) {
    hipLaunchKernelGGL((prefix_attn_kernel<DT, DP, true>), dim3(unsigned(grid)), dim3(64 * kWaves), 0, st, a);
    return hipGetLastError();
  }
  if (grid > 0)
    hipLaunchKernelGGL((prefix_attn_kernel<DT, DP, false>), dim3(unsigned(grid)), dim3(64 * kWaves), 0, st, a);
  hipLaunchKernelGGL((prefix_attn_join_kernel<DT>), dim3(unsigned(cdiv64(int64_t(a.T) * a.Hq, 4))),
                     dim3(256), 0, st, a);
  return hipGetLastError();
}

}  // namespace

PrefixAttnPlan prefix_attention_plan(int64_t T, int G, int Hq, int Hkv, int D, int page_size,
                                     int64_t prefix_width, int64_t own_width) {
  PrefixAttnPlan p{};
  p.dp = D <= 64 ? 64 : D <= 128 ? 128 : 256;
  const int grp = Hq / Hkv;
  const int64_t pmax = prefix_width * page_size, omax = own_width * page_size;
  p.shared = T * grp > 32 * int64_t(G);
  const int tile = p.shared ? kTileRows : kRows;
  p.prefix_tiles = int(cdiv64(T * grp, tile) + std::min<int64_t>(G, T));  // a segment of no rows has no tile
  p.own_tiles = int(cdiv64(grp, kRows));
  p.own_unit = 16 * kWaves;
  p.prefix_unit = p.shared ? (p.dp > 128 ? tile_block<256>() : tile_block<128>()) : p.own_unit;
  // Key ranges for about `target` workgroups, none shorter than `least` keys. Two workgroups fit a
  // compute unit, and a second round of them costs more than shorter ranges save: 512 in all (96 tokens
  // of one key head over 1024 keys of their own: 480 workgroups 7.9 us, 768 12.0 us). Shared tiles take
  // one per unit, so that the own ranges run beside them (64 tokens over a 16k prefix: 35 us, with
  // 512 tiles 45 us).
  auto splits = [](int64_t keys, int64_t wgs, int64_t target, int64_t least) {
    if (keys <= 0) return int64_t(0);
    const int64_t want = std::max<int64_t>(1, target / std::max<int64_t>(wgs, 1));
    return std::max<int64_t>(1, std::min(want, cdiv64(keys, least)));
  };
  const int64_t ptiles = std::max<int64_t>(1, cdiv64(T * grp, tile));
  p.prefix_splits = int(splits(pmax, ptiles * Hkv, p.shared ? 256 : 512, p.shared ? 256 : 64));
  const int64_t left = std::max<int64_t>(256, 512 - ptiles * Hkv * p.prefix_splits);
  p.own_splits = int(splits(omax, T * p.own_tiles * Hkv, left, 64));
  // one range a row and no prefix: the rows are written as they are
  p.direct = p.prefix_splits == 0 && p.own_splits == 1;
  const int64_t rows = p.direct ? 0 : T * Hq, slots = p.prefix_splits + p.own_splits;
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
