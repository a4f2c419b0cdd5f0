// Shared by the norm (k_norm.cu) and its gradient (k_norm_grad.cu): weights, the reduction over the threads
// of a row, and how many threads a row gets.
#pragma once
#include <algorithm>

#include "vectors.cuh"

namespace hlo {

constexpr int kAnyThreads = 256;

inline unsigned any_grid(int64_t rows) { return (unsigned)(rows < (1 << 20) ? rows : 1 << 20); }

__device__ __forceinline__ float weight_at(const void* w, int dt, float offset, int64_t i) {
  return w ? load_as_f32(w, dt, i) + offset : 1.0f + offset;
}

// Sum and maximum over the blockDim.x threads (whole warps) of this thread's row group, to all of them.
// Groups of one warp need shuffles alone; larger ones exchange through `red` (2 floats a warp of the block)
// behind the group's own named barrier, so groups of a block run apart.
__device__ __forceinline__ void group_barrier() {
  asm volatile("bar.sync %0, %1;" ::"r"(threadIdx.y + 1), "r"(blockDim.x) : "memory");
}
template <bool MAX>
__device__ __forceinline__ void group_sum_max(float& s, float& m, float* red) {
  s = warp_sum(s);
  if (MAX) m = warp_max(m);
  const int warps = blockDim.x >> 5;
  if (warps == 1) return;
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  float* const mine = red + 2 * warps * threadIdx.y;
  if (lane == 0) *reinterpret_cast<float2*>(mine + 2 * w) = make_float2(s, m);
  group_barrier();
  const float2 v = lane < warps ? *reinterpret_cast<const float2*>(mine + 2 * lane) : make_float2(0.0f, 0.0f);
  s = warp_sum(v.x);
  if (MAX) m = warp_max(v.y);
}

// W weights from column c0 on (columns outside the row: 1). `whole`: the vector may be one aligned access.
template <int DT>
__device__ __forceinline__ void load_weights(const void* w, int dt, float offset, int c0, int n, bool whole,
                                             float (&v)[kVec<DT>]) {
  constexpr int W = kVec<DT>;
  if (!w) {
#pragma unroll
    for (int e = 0; e < W; ++e) v[e] = 1.0f;
  } else if (whole && dt == DT) {
    unpack<DT>(__ldg(reinterpret_cast<const uint4*>(w) + c0 / W), v);
  } else if (whole) {
#pragma unroll
    for (int q = 0; q < W / 4; ++q) {
      const float4 f = __ldg(reinterpret_cast<const float4*>(reinterpret_cast<const float*>(w) + c0) + q);
      v[4 * q] = f.x, v[4 * q + 1] = f.y, v[4 * q + 2] = f.z, v[4 * q + 3] = f.w;
    }
  } else {
#pragma unroll
    for (int e = 0; e < W; ++e) v[e] = c0 + e >= 0 && c0 + e < n ? load_as_f32(w, dt, c0 + e) : 1.0f;
  }
  if (offset != 0.0f) {
#pragma unroll
    for (int e = 0; e < W; ++e) v[e] += offset;
  }
}

// Vectors a thread holds, threads a row and rows a block, for rows of `vectors` 16-byte vectors.
struct RowShape {
  int k, tx, ty;
};
inline RowShape row_shape(int64_t rows, int64_t vectors, int max_k) {
  const int sms = device_sm_count();
  int k = 1;
  // few rows: as many threads a row as there are vectors, for latency; many: more bytes in flight a thread
  const int64_t most = rows <= 2 * sms ? 1024 : 128;
  while (k < max_k && vectors > most * k) k *= 2;
  while (k < max_k && vectors > (k == 1 ? 1024 : 512 * (int64_t)k)) k *= 2;
  RowShape s;
  s.k = k;
  s.tx = (int)((vectors + k - 1) / k + 31) / 32 * 32;
  s.ty = s.tx >= 256 || rows <= sms ? 1 : (int)std::min<int64_t>(256 / s.tx, 15);
  return s;
}

}  // namespace hlo
