// Rotary positions for queries and keys, with keys and values appended to a paged cache.
//
// For token t and head h of q and of k:  u = x * w / sqrt(mean(x^2) + eps)  (x itself without a
// norm weight), then for each of the rot / 2 pairs p, with c, s = table[positions[t]],
//     (u_a, u_b) <- (u_a c_p - u_b s_p, u_b c_p + u_a s_p),
// a, b = p, p + rot / 2, or 2p, 2p + 1 when interleaved; the other elements pass. Everything is fp32
// from the load to the one rounding at the store. q goes to q_out, k to the cache row of slots[t];
// v is copied bit for bit.
//
// q_out may be q: whoever reads an element also writes it, and the norm's sum, which crosses lanes,
// is complete before the first store of the head.
#include "device_common.hpp"
#include "rope_append.hpp"

namespace lmx {

namespace {

// One head of one token: where it is read and written and what is done to it.
template <typename S>
struct Head {
  const S* src;
  S* dst;  // null: nothing is written
  const S* w;
  int pos;
  bool is_v;
};

template <typename S>
__device__ __forceinline__ Head<S> find_head(const RopeArgs& a, int t, int h) {
  Head<S> r{};
  r.pos = a.positions[t];
  if (h < a.Hq) {
    r.src = static_cast<const S*>(a.q) + int64_t(t) * a.ldq + int64_t(h) * a.D;
    r.dst = static_cast<S*>(a.q_out) + int64_t(t) * a.ldqo + int64_t(h) * a.D;
    r.w = static_cast<const S*>(a.q_norm);
  } else {
    r.is_v = h >= a.Hq + a.Hkv;
    const int hk = h - a.Hq - (r.is_v ? a.Hkv : 0);
    r.src = static_cast<const S*>(r.is_v ? a.v : a.k) + int64_t(t) * (r.is_v ? a.ldv : a.ldk) +
            int64_t(hk) * a.D;
    if (!r.is_v) r.w = static_cast<const S*>(a.k_norm);
    const int64_t slot = a.slots[t];
    if (slot >= 0 && slot < a.num_slots) {
      const int64_t pg = slot / a.page_size, place = slot - pg * a.page_size;
      r.dst = static_cast<S*>(r.is_v ? a.v_cache : a.k_cache) + pg * a.page_stride +
              place * a.token_stride + int64_t(hk) * a.head_stride;
    }
  }
  if (r.pos < 0 || r.pos >= a.table_rows) r.dst = nullptr;
  return r;
}

// 8 elements of a 16-byte aligned row as they are stored.
template <int DT>
struct Chunk {
  uint4 v[DT == DT_F32 ? 2 : 1];
  using S = typename Traits<DT>::store_t;
  __device__ __forceinline__ void load(const S* p) {
    v[0] = gload16(p);
    if constexpr (DT == DT_F32) v[1] = gload16(p + 4);
  }
  __device__ __forceinline__ void store(S* p) const {
    reinterpret_cast<uint4*>(p)[0] = v[0];
    if constexpr (DT == DT_F32) reinterpret_cast<uint4*>(p)[1] = v[1];
  }
  __device__ __forceinline__ void get(float* f) const {
    if constexpr (DT == DT_F32) {
      const uint32_t u[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w};
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = __uint_as_float(u[e]);
    } else {
      const uint32_t u[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        f[2 * e] = Traits<DT>::to_f32(uint16_t(u[e]));
        f[2 * e + 1] = Traits<DT>::to_f32(uint16_t(u[e] >> 16));
      }
    }
  }
  __device__ __forceinline__ void set(const float* f) {
    if constexpr (DT == DT_F32) {
      v[0] = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
      v[1] = make_uint4(__float_as_uint(f[4]), __float_as_uint(f[5]), __float_as_uint(f[6]), __float_as_uint(f[7]));
    } else {
      uint32_t u[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        u[e] = uint32_t(Traits<DT>::from_f32(f[2 * e])) | (uint32_t(Traits<DT>::from_f32(f[2 * e + 1])) << 16);
      v[0] = make_uint4(u[0], u[1], u[2], u[3]);
    }
  }
};

// 16-byte aligned rows, D % 8 == 0, rot % 16 == 0. A group of 2^lph lanes owns one head; lane j
// holds pairs 8j .. 8j + 7 as two 8-element chunks (pairs beyond rot / 2: 16 consecutive elements of
// the untouched tail), so only the norm's sum crosses lanes.
template <int DT, bool INTER>
__global__ __launch_bounds__(256) void rope_append_kernel(RopeArgs a, int lph) {
  using S = typename Traits<DT>::store_t;
  const int heads = a.Hq + 2 * a.Hkv;
  const int64_t unit = (int64_t(blockIdx.x) * 256 + threadIdx.x) >> lph;
  const int j = int(threadIdx.x) & ((1 << lph) - 1);
  const bool in = unit < int64_t(a.T) * heads;
  const int64_t u = in ? unit : 0;
  const int t = int(u / heads);
  const Head<S> hd = find_head<S>(a, t, int(u - int64_t(t) * heads));

  const int half = a.rot / 2, p0 = j * 8;
  const bool split = !INTER && p0 < half;
  const int e0 = split ? p0 : 2 * p0, e1 = split ? p0 + half : e0 + 8;
  const bool has0 = in && e0 < a.D, has1 = in && e1 < a.D;
  Chunk<DT> c0{}, c1{};
  if (has0) c0.load(hd.src + e0);
  if (has1) c1.load(hd.src + e1);
  if (!hd.is_v) {
    float x[2][8];
    c0.get(x[0]);
    c1.get(x[1]);
    const bool turn = hd.dst != nullptr && p0 < half;
    Chunk<DT_F32> cs{}, sn{};
    if (turn) {
      const uint32_t* row = reinterpret_cast<const uint32_t*>(a.table) + int64_t(hd.pos) * a.rot;
      cs.load(row + p0);
      sn.load(row + half + p0);
    }
    if (hd.w != nullptr) {
      Chunk<DT> w0{}, w1{};
      if (has0) w0.load(hd.w + e0);
      if (has1) w1.load(hd.w + e1);
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) ss += x[0][e] * x[0][e] + x[1][e] * x[1][e];
      for (int d = 1; d < (1 << lph); d <<= 1) ss += __shfl_xor(ss, d, 64);
      const float r = 1.f / sqrtf(ss / float(a.D) + a.eps);
      float f0[8], f1[8];
      w0.get(f0);
      w1.get(f1);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        x[0][e] *= r * f0[e];
        x[1][e] *= r * f1[e];
      }
    }
    if (turn) {
      float c[8], s[8];
      cs.get(c);
      sn.get(s);
#pragma unroll
      for (int p = 0; p < 8; ++p) {
        float& xa = INTER ? x[p / 4][2 * (p % 4)] : x[0][p];
        float& xb = INTER ? x[p / 4][2 * (p % 4) + 1] : x[1][p];
        const float ya = xa * c[p] - xb * s[p];
        xb = xb * c[p] + xa * s[p];
        xa = ya;
      }
    }
    c0.set(x[0]);
    c1.set(x[1]);
  }
  if (hd.dst == nullptr) return;
  if (has0) c0.store(hd.dst + e0);
  if (has1) c1.store(hd.dst + e1);
}

// Any size and alignment: one wave per head, one element or pair per lane and step.
template <int DT, bool INTER>
__global__ __launch_bounds__(256) void rope_append_any_kernel(RopeArgs a) {
  using Tr = Traits<DT>;
  using S = typename Tr::store_t;
  const int heads = a.Hq + 2 * a.Hkv, lane = int(threadIdx.x) & 63;
  const int64_t u = int64_t(blockIdx.x) * 4 + wave_id();
  if (u >= int64_t(a.T) * heads) return;
  const int t = int(u / heads);
  const Head<S> hd = find_head<S>(a, t, int(u - int64_t(t) * heads));
  if (hd.dst == nullptr) return;
  if (hd.is_v) {
    for (int d = lane; d < a.D; d += 64) hd.dst[d] = hd.src[d];
    return;
  }
  float r = 1.f;
  if (hd.w != nullptr) {
    float ss = 0.f;
    for (int d = lane; d < a.D; d += 64) {
      const float v = Tr::to_f32(hd.src[d]);
      ss += v * v;
    }
    for (int d = 1; d < 64; d <<= 1) ss += __shfl_xor(ss, d, 64);
    r = 1.f / sqrtf(ss / float(a.D) + a.eps);
  }
  auto in = [&](int d) {
    const float v = Tr::to_f32(hd.src[d]);
    return hd.w != nullptr ? v * (r * Tr::to_f32(hd.w[d])) : v;
  };
  const int half = a.rot / 2;
  const float* row = a.table + int64_t(hd.pos) * a.rot;
  for (int p = lane; p < half; p += 64) {
    const int ia = INTER ? 2 * p : p, ib = INTER ? 2 * p + 1 : p + half;
    const float xa = in(ia), xb = in(ib), c = row[p], s = row[half + p];
    hd.dst[ia] = Tr::from_f32(xa * c - xb * s);
    hd.dst[ib] = Tr::from_f32(xb * c + xa * s);
  }
  for (int d = a.rot + lane; d < a.D; d += 64) hd.dst[d] = Tr::from_f32(in(d));
}

template <int DT, bool INTER>
hipError_t launch_typed(const RopeArgs& a, bool vec, hipStream_t st) {
  const int64_t units = int64_t(a.T) * (a.Hq + 2 * a.Hkv);
  if (vec) {
    int lph = 0;
    while ((16 << lph) < a.D) ++lph;
    const int64_t grid = ((units << lph) + 255) / 256;
    hipLaunchKernelGGL((rope_append_kernel<DT, INTER>), dim3(unsigned(grid)), dim3(256), 0, st, a, lph);
  } else {
    hipLaunchKernelGGL((rope_append_any_kernel<DT, INTER>), dim3(unsigned((units + 3) / 4)), dim3(256),
                       0, st, a);
  }
  return hipGetLastError();
}

template <int DT>
hipError_t launch_dtype(const RopeArgs& a, bool interleaved, bool vec, hipStream_t st) {
  return interleaved ? launch_typed<DT, true>(a, vec, st) : launch_typed<DT, false>(a, vec, st);
}

}  // namespace

hipError_t launch_rope_append(const RopeArgs& a, int dtype, bool interleaved, bool vec,
                              hipStream_t st) {
  if (dtype == DT_F32) return launch_dtype<DT_F32>(a, interleaved, vec, st);
  if (dtype == DT_BF16) return launch_dtype<DT_BF16>(a, interleaved, vec, st);
  return launch_dtype<DT_F16>(a, interleaved, vec, st);
}

}  // namespace lmx
