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
// back, 256 rows' norms (5120 bf16 to 8 bits) take 4.0 us a call in place of 6.1, and the gradient of 2049 x 1001
// f32 12.9 in place of 14.4.
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

__device__ __forceinline__ uint8_t f8_bits(float v) {
  return (uint8_t)__nv_cvt_float_to_fp8(v, __NV_SATFINITE, __NV_E4M3);
}

// The scale of an 8-bit row whose largest magnitude is m.
__device__ __forceinline__ float row_scale(float m, int out_dt) {
  const float s = __fdiv_rn(m, out_dt == S8 ? 127.0f : 448.0f);
  return s == 0.0f ? 1.0f : s;
}

// y / scale in 8 bits: the quotient is y * inv with inv = RN(1 / scale), within 1.5 f32 ulps of it.
__device__ __forceinline__ int8_t s8_code(float y, float inv) {
  const int q = __float2int_rn(__fmul_rn(y, inv));  // NaN -> 0
  return (int8_t)max(-128, min(127, q));
}

}  // namespace hlo
