// 16-byte vectors of the float types, whole or cut off at the ends of a row, and dropout on a vector.
#pragma once
#include "philox.cuh"
#include "rows.cuh"

namespace hlo {

template <int DT>
constexpr int kVec = DT == F32 ? 4 : 8;  // elements of a 16-byte vector

// Streamed once: first in line to leave L2. A plain load, because an output may be the input.
__device__ __forceinline__ uint4 load16(const void* p) { return __ldcs(reinterpret_cast<const uint4*>(p)); }

template <int DT>
__device__ __forceinline__ void unpack(const uint4& w, float (&v)[kVec<DT>]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
  if constexpr (DT == F32) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(u[i]);
  } else if constexpr (DT == BF16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(u[i] << 16);
      v[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
      v[2 * i] = f.x;
      v[2 * i + 1] = f.y;
    }
  }
}

template <int DT>
__device__ __forceinline__ uint4 pack(const float (&v)[kVec<DT>]) {
  uint32_t u[4];
  if constexpr (DT == F32) {
#pragma unroll
    for (int i = 0; i < 4; ++i) u[i] = __float_as_uint(v[i]);
  } else if constexpr (DT == BF16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      u[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
      u[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
  }
  return make_uint4(u[0], u[1], u[2], u[3]);
}

// The elements c0 .. c0 + W - 1 of a row of n that starts at element `off` of p; those outside 0 .. n-1
// read as 0. off + c0 is a multiple of W (counted from address 0), so a whole vector is one access.
template <int DT>
__device__ __forceinline__ uint4 load_cut(const void* p, int64_t off, int64_t c0, int64_t n) {
  constexpr int W = kVec<DT>, EB = 16 / W;
  const char* a = reinterpret_cast<const char*>(p) + (off + c0) * EB;
  if (c0 >= 0 && c0 + W <= n) return load16(a);
  uint32_t u[4] = {0, 0, 0, 0};
#pragma unroll
  for (int e = 0; e < W; ++e) {
    if (c0 + e < 0 || c0 + e >= n) continue;
    if (EB == 4) u[e & 3] = reinterpret_cast<const uint32_t*>(a)[e];
    else u[e >> 1] |= (uint32_t)reinterpret_cast<const uint16_t*>(a)[e] << (16 * (e & 1));
  }
  return make_uint4(u[0], u[1], u[2], u[3]);
}

template <int DT>
__device__ __forceinline__ void store_cut(void* p, int64_t off, int64_t c0, int64_t n, const float (&v)[kVec<DT>]) {
  constexpr int W = kVec<DT>, EB = 16 / W;
  char* a = reinterpret_cast<char*>(p) + (off + c0) * EB;
  if (c0 >= 0 && c0 + W <= n) {
    *reinterpret_cast<uint4*>(a) = pack<DT>(v);
    return;
  }
#pragma unroll
  for (int e = 0; e < W; ++e)
    if (c0 + e >= 0 && c0 + e < n) store_from_f32(a, DT, e, v[e]);
}

// drop(v) for the W elements from linear index i on. Their counters are i / 4, ...: W / 4 of them when i is a
// multiple of 4, one more otherwise, and the words wanted then start i mod 4 words in. i may be below 0 where
// a vector starts before the first row (those elements are not stored).
template <int W>
__device__ __forceinline__ void drop_vec(const DropPlan& d, const Philox& g, int64_t i, float (&v)[W]) {
  uint32_t w[W + 4];
  const int m = (int)(i & 3);
  const int64_t quad = i >> 2;
#pragma unroll
  for (int q = 0; q < W / 4; ++q) {
    const uint4 r = philox4(g, (uint64_t)(quad + q));
    w[4 * q] = r.x, w[4 * q + 1] = r.y, w[4 * q + 2] = r.z, w[4 * q + 3] = r.w;
  }
  if (m) {
    const uint4 r = philox4(g, (uint64_t)(quad + W / 4));
    w[W] = r.x, w[W + 1] = r.y, w[W + 2] = r.z, w[W + 3] = r.w;
    if (m & 1) {
#pragma unroll
      for (int e = 0; e < W + 2; ++e) w[e] = w[e + 1];
    }
    if (m & 2) {
#pragma unroll
      for (int e = 0; e < W; ++e) w[e] = w[e + 2];
    }
  }
#pragma unroll
  for (int e = 0; e < W; ++e) v[e] = kept(d, w[e]) ? __fmul_rn(v[e], d.scale) : 0.0f;
}

// Whether every view's rows can be read in vectors of W elements that fall on the same columns: addresses
// that are alike modulo W elements, for every row. *cut: some vector is cut off at an end of its row, or
// starts before it.
template <int NV>
inline bool vectors_fit(const Rows<NV>& m, const void* const (&ptr)[NV], const int (&eb)[NV], int64_t n, int w, bool* cut) {
  const int64_t r0 = (int64_t)((uintptr_t)ptr[0] / eb[0]) % w;
  *cut = r0 != 0 || n % w != 0;
  for (int v = 0; v < NV; ++v) {
    if (!ptr[v]) continue;
    if ((int64_t)((uintptr_t)ptr[v] / eb[v]) % w != r0) return false;
    for (int j = 0; j < m.n; ++j) {
      if ((m.stride[v][j] - m.stride[0][j]) % w != 0) return false;
      *cut = *cut || m.stride[v][j] % w != 0;
    }
  }
  return true;
}

}  // namespace hlo
