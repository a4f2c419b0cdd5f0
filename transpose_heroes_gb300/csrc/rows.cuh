// Device helpers of the kernels between a decoder's matrix products: loads, the codes of 8-bit outputs,
// and the sums and maxima over the threads of a row.
#pragma once
#include <cuda_fp8.h>

#include "device_common.cuh"
#include "layer_plans.h"
#include "quant_common.cuh"

namespace hlo {

// Kernels of one stream that follow one another closely: a kernel launched by launch_after() may be set up, and its
// blocks placed, while the one before it ends. Every block of it calls follow() first: it lets the next kernel
// do the same, and waits until everything queued before this kernel has ended and its writes are seen. Back to
// back, 256 rows' norms (5120 bf16 to 8 bits) take 4 us a call in place of 6, and the gradient of 2049 x 1001 f32 1.5 us
// less.
// The gradient lets its join be set up only when its rows are done (allow_next() late): blocks of the join that wait
// from the start hold places that later blocks want (30000 x 129 bf16 29 us, so 23).
__device__ __forceinline__ void allow_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_last() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void follow() {
  allow_next();
  wait_for_last();
}
template <typename... P, typename... A>
cudaError_t launch_after(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t s, int cluster, A... args) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Plain loads, also of weights, tables and histories: the read-only path (__ldg) asks that nobody writes the data
// while the kernel runs, and here the kernel before may still be writing them when this one is set up. An output
// may also be the input.
template <typename T>
__device__ __forceinline__ T load_kept(const T* p) {
  return *p;
}
__device__ __forceinline__ float load_plain(const void* p, int dt, int64_t i) {
  switch (dt) {
    case F32: return reinterpret_cast<const float*>(p)[i];
    case BF16: return bf16_bits_to_f32(reinterpret_cast<const uint16_t*>(p)[i]);
    default: return f16_bits_to_f32(reinterpret_cast<const uint16_t*>(p)[i]);
  }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v = ieee_max(v, __shfl_xor_sync(0xffffffffu, v, off));
  return v;
}

// Sum and (NaN-propagating) maximum over a block of whole warps, to every thread. `red` holds 2 floats a
// warp; a second use of the same `red` needs a barrier between.
__device__ __forceinline__ void block_sum_max(float& s, float& m, float* red) {
  s = warp_sum(s);
  m = warp_max(m);
  const int warps = blockDim.x >> 5, lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  if (lane == 0) {
    red[2 * w] = s;
    red[2 * w + 1] = m;
  }
  __syncthreads();
  s = lane < warps ? red[2 * lane] : 0.0f;
  m = lane < warps ? red[2 * lane + 1] : 0.0f;  // maxima here are of magnitudes
  s = warp_sum(s);
  m = warp_max(m);
}

// y / scale in 8 bits, by the definition's own division.
__device__ __forceinline__ uint8_t f8_code(float y, float scale) {
  return (uint8_t)__nv_cvt_float_to_fp8(__fdiv_rn(y, scale), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ int8_t s8_code(float y, float scale) {
  const int q = __float2int_rn(__fdiv_rn(y, scale));  // NaN -> 0
  return (int8_t)max(-128, min(127, q));
}

// The scale of an 8-bit row whose largest |y| is m.
__device__ __forceinline__ float row_scale(float m, int out_dt) {
  const float s = __fdiv_rn(m, out_dt == S8 ? 127.0f : 448.0f);
  return s == 0.0f ? 1.0f : s;
}

// Four of them, y[i] in byte i.
static __device__ __noinline__ uint32_t codes_divided(float4 y, float scale, int f8) {
  const float v[4] = {y.x, y.y, y.z, y.w};
  uint32_t u = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) u |= (uint32_t)(f8 ? f8_code(v[i], scale) : (uint8_t)s8_code(v[i], scale)) << (8 * i);
  return u;
}

// The same without divisions. With inv = RN(1 / scale) finite and not 0, q = y inv is within 2^-23 relative of y / scale
// and the f32 quotient within 2^-24; so the quotient lies between q (1 - 2^-21) and q (1 + 2^-21), and where both ends
// round to one code, so does it. Where one of the four does not, or the scale is a NaN, infinite or below 2^-128, they
// are divided. 16384 x 8192 bf16 to f8 with residual: 147 us, 172 where every element is divided.
__device__ __forceinline__ uint32_t codes(float4 y, float scale, float inv, int f8) {
  const float2 q0 = __fmul2_rn(make_float2(y.x, y.y), make_float2(inv, inv));
  const float2 q1 = __fmul2_rn(make_float2(y.z, y.w), make_float2(inv, inv));
  const float2 lo = make_float2(1.0f - 0x1p-21f, 1.0f - 0x1p-21f), hi = make_float2(1.0f + 0x1p-21f, 1.0f + 0x1p-21f);
  uint32_t a, open;
  if (f8) {
    const auto both = [](float2 u, float2 v) {
      return (uint32_t)__nv_cvt_float2_to_fp8x2(u, __NV_SATFINITE, __NV_E4M3) |
             (uint32_t)__nv_cvt_float2_to_fp8x2(v, __NV_SATFINITE, __NV_E4M3) << 16;
    };
    a = both(__fmul2_rn(q0, lo), __fmul2_rn(q1, lo));
    open = a ^ both(__fmul2_rn(q0, hi), __fmul2_rn(q1, hi));
  } else {  // |q| < 127.5, and adding the magic number rounds to an integer, ties to even, into the low bits
    const float2 m = make_float2(kMagic, kMagic);
    const float2 a0 = __ffma2_rn(q0, lo, m), a1 = __ffma2_rn(q1, lo, m), b0 = __ffma2_rn(q0, hi, m), b1 = __ffma2_rn(q1, hi, m);
    const auto bytes = [](float2 u, float2 v) {
      return __byte_perm(__byte_perm(__float_as_uint(u.x), __float_as_uint(u.y), 0x0040),
                         __byte_perm(__float_as_uint(v.x), __float_as_uint(v.y), 0x0040), 0x5410);
    };
    a = bytes(a0, a1);
    open = a ^ bytes(b0, b1);
  }
  if (open || !(inv > 0.0f && inv <= 3.4028235e38f)) a = codes_divided(y, scale, f8);
  return a;
}

}  // namespace hlo
