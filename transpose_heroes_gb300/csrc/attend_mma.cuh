// What the attention's tensor-core kernels share: asynchronous 16-byte copies, 8-bit entries as f16, values that a mask
// hides, and a tile's results.
#pragma once
#include "attend_work.cuh"

namespace hlo {

__device__ __forceinline__ uint32_t attend_smem(const void* p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }

// 16 bytes, or zeros where !given (src is then any valid address).
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool given) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(given ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ float exp2_fast(float x) {  // relative error 2^-22; 0 below 2^-126
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Two e4m3 codes (the low 16 bits) as f16, which holds each of them exactly.
__device__ __forceinline__ uint32_t f16_of_codes(uint32_t two) {
  uint32_t r;
  asm("{ .reg .b16 c; cvt.u16.u32 c, %1; cvt.rn.f16x2.e4m3x2 %0, c; }" : "=r"(r) : "r"(two));
  return r;
}

// Two weights in the 16-bit type of the products, nearest even.
template <bool BF>
__device__ __forceinline__ uint32_t pack_pair(float lo, float hi) {
  if constexpr (BF) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}

// Replaces infinite and NaN elements of 16 bytes by 0; whether there were any. ONES: the exponent's bits of two 16-bit
// elements (or of four codes, whose only such value has all bits of exponent and fraction set).
template <bool F8, bool BF>
__device__ __forceinline__ bool clear_word(uint32_t& w) {
  constexpr uint32_t ones = F8 ? 0x7F7F7F7Fu : BF ? 0x7F807F80u : 0x7C007C00u;
  const uint32_t e = w & ones;
  uint32_t bad = 0;
  if constexpr (F8) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (((e >> (8 * i)) & 0x7F) == 0x7F) bad |= 0xFFu << (8 * i);
  } else {
    if ((e & 0xFFFFu) == (ones & 0xFFFFu)) bad |= 0xFFFFu;
    if ((e >> 16) == (ones >> 16)) bad |= 0xFFFF0000u;
  }
  w &= ~bad;
  return bad != 0;
}
// Whether 16 bytes hold such an element. Of two 16-bit elements an exponent of ones carries into the sign's place.
template <bool F8, bool BF>
__device__ __forceinline__ bool wants_clearing(const uint4& v) {
  if constexpr (F8) {
    constexpr uint32_t ones = 0x7F7F7F7Fu, step = 0x01010101u;  // 0x7F + 1: the code's sign
    return ((((v.x & ones) + step) | ((v.y & ones) + step) | ((v.z & ones) + step) | ((v.w & ones) + step)) & 0x80808080u) != 0;
  } else {
    constexpr uint32_t ones = BF ? 0x7F807F80u : 0x7C007C00u, step = BF ? 0x00800080u : 0x04000400u;
    return ((((v.x & ones) + step) | ((v.y & ones) + step) | ((v.z & ones) + step) | ((v.w & ones) + step)) & 0x80008000u) != 0;
  }
}
template <bool F8, bool BF>
__device__ __forceinline__ bool clear_vector(uint4* at) {
  uint4 v = *at;
  if (!wants_clearing<F8, BF>(v)) return false;
  clear_word<F8, BF>(v.x);
  clear_word<F8, BF>(v.y);
  clear_word<F8, BF>(v.z);
  clear_word<F8, BF>(v.w);
  *at = v;
  return true;
}

// An element of a value, as f32.
template <bool F8>
__device__ __forceinline__ float value_at(const AttendPlan& p, int64_t i) {
  if constexpr (F8) {
    const __half_raw h = __nv_cvt_fp8_to_halfraw(reinterpret_cast<const uint8_t*>(p.v)[i], __NV_E4M3);
    return __half2float(*reinterpret_cast<const __half*>(&h));
  } else {
    return load_plain(p.v, p.dt, i);
  }
}

// What a row's element c gains from the infinite and NaN values that the masked tiles cleared: those of the entries from
// `first` to `end` that its token sees. Their products would be infinite or NaN whatever the weights.
template <bool F8>
__device__ __noinline__ float cleared_values(const AttendPlan& p, const AttendItem& it, int t, int first, int end, int c) {
  float sum = 0.0f;
  const int32_t* const table = p.m.table + it.b * p.m.table_stride;
  for (int i = first; i < end; ++i) {
    if (!attend_sees(p, it, t, i)) continue;
    int page, place;
    cache_place(p.m, table, i, &page, &place);
    if (page < 0) continue;
    const float v = value_at<F8>(p, page * p.v_stride[0] + place * p.v_stride[1] + it.head * p.v_stride[2] + c);
    if (!(fabsf(v) < __int_as_float(0x7F800000))) sum += v;
  }
  return sum;
}

}  // namespace hlo
