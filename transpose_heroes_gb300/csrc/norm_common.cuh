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

// Sum over the blockDim.x threads (whole warps) of this thread's row group, to all of them.
// Groups of one warp need shuffles alone; larger ones exchange through `red` (2 floats a warp of the block)
// behind the group's own named barrier, so groups of a block run apart. (With one float a warp the gradient of 32768 x 1001
// bf16 takes 81.4 us in place of 79.4.)
__device__ __forceinline__ void group_barrier() {
  asm volatile("bar.sync %0, %1;" ::"r"(threadIdx.y + 1), "r"(blockDim.x) : "memory");
}
__device__ __forceinline__ void group_sum(float& s, float* red) {
  s = warp_sum(s);
  const int warps = blockDim.x >> 5;
  if (warps == 1) return;
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  float* const mine = red + 2 * warps * threadIdx.y;
  if (lane == 0) *reinterpret_cast<float2*>(mine + 2 * w) = make_float2(s, 0.0f);
  group_barrier();
  const float2 v = lane < warps ? *reinterpret_cast<const float2*>(mine + 2 * lane) : make_float2(0.0f, 0.0f);
  s = warp_sum(v.x);
}
// The greatest of the group's magnitudes, as their bits: these order like the values, with NaN above all.
__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }
__device__ __forceinline__ float group_max(uint32_t top, uint32_t* red) {
  top = __reduce_max_sync(0xffffffffu, top);
  const int warps = blockDim.x >> 5;
  if (warps == 1) return __uint_as_float(top);
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  uint32_t* const mine = red + warps * threadIdx.y;
  if (lane == 0) mine[w] = top;
  group_barrier();
  return __uint_as_float(__reduce_max_sync(0xffffffffu, lane < warps ? mine[lane] : 0u));
}

// A row that need not start or end on a 16-byte boundary: its whole vectors are the columns [head, end), and
// up to 2 W - 2 elements lie outside them, one each for the row's first threads.
struct RowCut {
  int head, end;
  __device__ __forceinline__ int edge(int thread, int n) const {
    if (thread < head) return thread;
    const int c = end + thread - head;
    return c < n ? c : -1;
  }
};
template <int W>
__device__ __forceinline__ RowCut row_cut(const void* p, int eb, int64_t off, int n) {
  const int head = min(n, (int)(-((int64_t)((uintptr_t)p / eb) + off) & (W - 1)));
  return {head, head + (n - head) / W * W};
}

// W weights from column c0 on, all of them in the row. `whole`: c0 is a multiple of W and the weights are
// aligned to 16 bytes, so they are one vector (two in f32 for 16-bit rows).
template <int DT>
__device__ __forceinline__ void load_weights(const void* w, int dt, float offset, int c0, int n, bool whole,
                                             float (&v)[kVec<DT>]) {
  constexpr int W = kVec<DT>;
  if (!w) {
#pragma unroll
    for (int e = 0; e < W; ++e) v[e] = 1.0f;
  } else if (whole && dt == DT) {
    unpack<DT>(load_kept(reinterpret_cast<const uint4*>(w) + c0 / W), v);
  } else if (whole) {
#pragma unroll
    for (int q = 0; q < W / 4; ++q) {
      const float4 f = load_kept(reinterpret_cast<const float4*>(reinterpret_cast<const float*>(w) + c0) + q);
      v[4 * q] = f.x, v[4 * q + 1] = f.y, v[4 * q + 2] = f.z, v[4 * q + 3] = f.w;
    }
  } else if (dt == DT && (uintptr_t)w % 16 == 0) {
    // two aligned vectors, then the words and the half word that c0 asks for
    constexpr int EW = W / 4;  // elements a word
    const int j = c0 / W, s = c0 - j * W, last = (n - 1) / W;
    const uint4* const at = reinterpret_cast<const uint4*>(w);
    const bool tail = n % W != 0;  // the last vector would end behind the weights
    uint4 a = load_kept(at + j), b = a;
    if (s) {
      if (j + 1 == last && tail) b = load_cut<DT>(w, 0, (int64_t)(j + 1) * W, n, nullptr);
      else b = load_kept(at + j + 1);
    }
    uint32_t u[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    if ((s / EW) & 2) {
#pragma unroll
      for (int i = 0; i < 6; ++i) u[i] = u[i + 2];
    }
    if ((s / EW) & 1) {
#pragma unroll
      for (int i = 0; i < 5; ++i) u[i] = u[i + 1];
    }
    if (EW == 2 && (s & 1)) {
#pragma unroll
      for (int i = 0; i < 4; ++i) u[i] = __funnelshift_r(u[i], u[i + 1], 16);
    }
    unpack<DT>(make_uint4(u[0], u[1], u[2], u[3]), v);
  } else {
#pragma unroll
    for (int e = 0; e < W; ++e) v[e] = load_as_f32(w, dt, c0 + e);
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
// For many rows, another doubling of the vectors wants `lanes` more vectors a row.
inline RowShape row_shape(int64_t rows, int64_t vectors, int max_k, int lanes) {
  const int sms = device_sm_count();
  int k = 1;
  if (rows > 2 * sms)
    while (k < 4 && vectors >= 2 * (int64_t)lanes * k) k *= 2;
  // few rows: as many threads a row as it has vectors, for latency
  while (k < max_k && vectors > (k == 1 ? 1024 : 512 * (int64_t)k)) k *= 2;
  RowShape s;
  s.k = k;
  s.tx = (int)((vectors + k - 1) / k + 31) / 32 * 32;
  s.ty = s.tx >= 256 || rows <= sms ? 1 : 256 / s.tx;
  return s;
}

__device__ __forceinline__ void store_out(const NormPlan& p, int64_t i, float y, float scale) {
  if (p.quant == NQ_ROW) {
    if (p.out_dt == S8) reinterpret_cast<int8_t*>(p.out)[i] = s8_code(y, scale);
    else reinterpret_cast<uint8_t*>(p.out)[i] = f8_code(y, scale);
  } else if (p.quant == NQ_STATIC) {
    reinterpret_cast<int8_t*>(p.out)[i] = (int8_t)quant_code(y, p.q.scale, p.q.inv_scale, p.q.zp, p.q.smin, p.q.smax);
  } else {
    store_from_f32(p.out, p.out_dt, i, y);
  }
}

cudaError_t run_norm_f32(const NormPlan& p, const RowShape& r, bool cut, int whole, cudaStream_t s);
cudaError_t run_norm_bf16(const NormPlan& p, const RowShape& r, bool cut, int whole, cudaStream_t s);
cudaError_t run_norm_f16(const NormPlan& p, const RowShape& r, bool cut, int whole, cudaStream_t s);

}  // namespace hlo
