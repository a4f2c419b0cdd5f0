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

// The same as pairs, for packed f32x2 arithmetic.
template <int DT>
__device__ __forceinline__ void unpack2(const uint4& w, float2 (&v)[kVec<DT> / 2]) {
  float f[kVec<DT>];
  unpack<DT>(w, f);
#pragma unroll
  for (int i = 0; i < kVec<DT> / 2; ++i) v[i] = make_float2(f[2 * i], f[2 * i + 1]);
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
// read as 0. off + c0 is a multiple of W (counted from address 0), so a whole vector is one access; so is a
// cut one where all of it lies inside the operand, [p, end): its neighbours' elements are dropped.
template <int DT>
__device__ __forceinline__ uint4 load_cut(const void* p, int64_t off, int64_t c0, int64_t n, const char* end) {
  constexpr int W = kVec<DT>, EB = 16 / W;
  const char* a = reinterpret_cast<const char*>(p) + (off + c0) * EB;
  if (c0 >= 0 && c0 + W <= n) return load16(a);
  const int lo = c0 < 0 ? (int)-c0 : 0, hi = n - c0 < W ? (int)(n - c0) : W;
  uint32_t u[4] = {0, 0, 0, 0};
  if (a >= reinterpret_cast<const char*>(p) && a + 16 <= end) {
    const uint4 w = load16(a);
    const uint32_t all[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int e = 0; e < W; ++e)
      if (e >= lo && e < hi) u[EB == 4 ? e & 3 : e >> 1] |= EB == 4 ? all[e & 3] : all[e >> 1] & (0xFFFFu << (16 * (e & 1)));
  } else {
#pragma unroll
    for (int e = 0; e < W; ++e) {
      if (e < lo || e >= hi) continue;
      if (EB == 4) u[e & 3] = reinterpret_cast<const uint32_t*>(a)[e];
      else u[e >> 1] |= (uint32_t)reinterpret_cast<const uint16_t*>(a)[e] << (16 * (e & 1));
    }
  }
  return make_uint4(u[0], u[1], u[2], u[3]);
}

// Stores the elements that lie in the row: of a vector cut off at one end, in up to three accesses.
template <int DT>
__device__ __forceinline__ void store_cut(void* p, int64_t off, int64_t c0, int64_t n, const float (&v)[kVec<DT>]) {
  constexpr int W = kVec<DT>, EB = 16 / W;
  char* a = reinterpret_cast<char*>(p) + (off + c0) * EB;
  const uint4 w = pack<DT>(v);
  if (c0 >= 0 && c0 + W <= n) {
    *reinterpret_cast<uint4*>(a) = w;
    return;
  }
  const int lo = c0 < 0 ? (int)-c0 : 0, hi = n - c0 < W ? (int)(n - c0) : W;
  if (lo == 0) {  // the first hi elements
    const int words = hi * EB / 4;
    if (words & 2) *reinterpret_cast<uint2*>(a) = make_uint2(w.x, w.y);
    if (words & 1) *reinterpret_cast<uint32_t*>(a + 4 * (words & 2)) = (words & 2) ? w.z : w.x;
    if (EB == 2 && (hi & 1)) *reinterpret_cast<uint16_t*>(a + 4 * words) = (uint16_t)((words & 2) ? ((words & 1) ? w.w : w.z) : ((words & 1) ? w.y : w.x));
  } else if (hi == W) {  // the last W - lo
    const int words = (W - lo) * EB / 4;
    if (words & 2) *reinterpret_cast<uint2*>(a + 8) = make_uint2(w.z, w.w);
    if (words & 1) *reinterpret_cast<uint32_t*>(a + 12 - 4 * (words & 2)) = (words & 2) ? w.y : w.w;
    if (EB == 2 && (lo & 1)) *reinterpret_cast<uint16_t*>(a + 2 * lo) = (uint16_t)(((lo & 4) ? ((lo & 2) ? w.w : w.z) : ((lo & 2) ? w.y : w.x)) >> 16);
  } else {
#pragma unroll
    for (int e = 0; e < W; ++e)
      if (e >= lo && e < hi) store_from_f32(a, DT, e, v[e]);
  }
}

// The generator's words for the W elements from linear index i on. Their counters are i / 4, ...: W / 4 of them
// when i is a multiple of 4 (WHOLE: it always is), one more otherwise, and the words wanted then start i mod 4
// words in. i may be below 0 where a vector starts before the first row (those elements are not stored).
template <int MODE, bool WHOLE, int W>
__device__ __forceinline__ void drop_words(const DropPlan& d, const Philox<MODE>& g, int64_t i, uint32_t (&w)[W + 4]) {
  const int64_t quad = i >> 2;
#pragma unroll
  for (int q = 0; q < W / 4; ++q) {
    const uint4 r = g.words(d, (uint64_t)(quad + q));
    w[4 * q] = r.x, w[4 * q + 1] = r.y, w[4 * q + 2] = r.z, w[4 * q + 3] = r.w;
  }
  const int m = WHOLE ? 0 : (int)(i & 3);
  if (m) {
    const uint4 r = g.words(d, (uint64_t)(quad + W / 4));
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
}

// v = drop(v).
template <int MODE, bool WHOLE, int W>
__device__ __forceinline__ void drop_vec(const DropPlan& d, const Philox<MODE>& g, int64_t i, float (&v)[W]) {
  uint32_t w[W + 4];
  drop_words<MODE, WHOLE, W>(d, g, i, w);
#pragma unroll
  for (int e = 0; e < W; ++e) v[e] = dropped(d, w[e], v[e]);
}

// v = r + drop(v): r + 0 where v is dropped (+0 for an r of -0), the addition of v where it is kept. Two predicated results
// cost less than a select and an addition.
template <int MODE, bool WHOLE, int W>
__device__ __forceinline__ void drop_add_vec(const DropPlan& d, const Philox<MODE>& g, int64_t i, float (&v)[W], const float (&r)[W]) {
  uint32_t w[W + 4];
  drop_words<MODE, WHOLE, W>(d, g, i, w);
#pragma unroll
  for (int e = 0; e < W; e += 2) {
    const float2 t = __fmul2_rn(make_float2(v[e], v[e + 1]), make_float2(d.scale, d.scale));
    const float2 s = __fadd2_rn(make_float2(r[e], r[e + 1]), make_float2(0.0f, 0.0f));
    v[e] = s.x, v[e + 1] = s.y;
    if (kept(d, w[e])) v[e] = __fadd_rn(r[e], t.x);
    if (kept(d, w[e + 1])) v[e + 1] = __fadd_rn(r[e + 1], t.y);
  }
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
