// Root-mean-square norm with the residual's addition (out = h r w, h = residual + drop(x)), and its
// gradient. See hlo_rms_norm in hlo_fusion.h for the formulas.
//
// The kernels here take any row length and any alignment: a block per row, threads take elements in turn,
// and the row is read twice (the second time from L2): once for the sum of squares and the largest
// |h w|, once for the outputs. A thread reads and writes the same elements in both passes, so outputs may
// replace inputs in place.
#include "philox.cuh"
#include "rows.cuh"

namespace hlo {

constexpr int kAnyThreads = 256;

static unsigned any_grid(int64_t rows) { return (unsigned)(rows < (1 << 20) ? rows : 1 << 20); }

__device__ __forceinline__ float weight_at(const void* w, int dt, float offset, int64_t i) {
  return w ? load_as_f32(w, dt, i) + offset : 1.0f + offset;
}

__device__ __forceinline__ void store_out(const NormPlan& p, int64_t i, float y, float inv) {
  if (p.quant == NQ_ROW) {
    if (p.out_dt == S8) reinterpret_cast<int8_t*>(p.out)[i] = s8_code(y, inv);
    else reinterpret_cast<uint8_t*>(p.out)[i] = f8_bits(__fmul_rn(y, inv));
  } else if (p.quant == NQ_STATIC) {
    reinterpret_cast<int8_t*>(p.out)[i] = (int8_t)quant_code(y, p.q.scale, p.q.inv_scale, p.q.zp, p.q.smin, p.q.smax);
  } else {
    store_from_f32(p.out, p.out_dt, i, y);
  }
}

__global__ void __launch_bounds__(kAnyThreads) norm_any_kernel(NormPlan p) {
  __shared__ float red[2 * kAnyThreads / 32];
  Philox g = {};
  if (p.drop.on) g = philox_of(p.drop);
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    int64_t off[4];
    row_offsets(p.map, row, off);
    auto h_at = [&](int64_t c) {
      float v = load_plain(p.x, p.dt, off[0] + c);
      if (p.drop.on) v = drop1(p.drop, g, (uint64_t)(row * p.n + c), v);
      return p.res ? __fadd_rn(load_plain(p.res, p.dt, off[1] + c), v) : v;
    };
    float ss = 0.0f, top = 0.0f;
    for (int64_t c = threadIdx.x; c < p.n; c += kAnyThreads) {
      const float h = h_at(c);
      ss = fmaf(h, h, ss);
      if (p.quant == NQ_ROW) top = ieee_max(top, fabsf(h * weight_at(p.w, p.w_dt, p.w_offset, c)));
    }
    block_sum_max(ss, top, red);
    const float r = rsqrtf(__fdiv_rn(ss, (float)p.n) + p.eps);
    if (threadIdx.x == 0 && p.rstd) p.rstd[row] = r;
    float inv = 0.0f;
    if (p.quant == NQ_ROW) {
      const float s = row_scale(r * top, p.out_dt);
      inv = __fdiv_rn(1.0f, s);
      if (threadIdx.x == 0) p.scales[row] = s;
    }
    for (int64_t c = threadIdx.x; c < p.n; c += kAnyThreads) {
      const float h = h_at(c);
      if (p.sum) store_from_f32(p.sum, p.dt, off[2] + c, h);
      store_out(p, off[3] + c, __fmul_rn(__fmul_rn(h, r), weight_at(p.w, p.w_dt, p.w_offset, c)), inv);
    }
    __syncthreads();  // red is used again by the next row
  }
}

cudaError_t launch_norm(const NormPlan& p, cudaStream_t s) {
  norm_any_kernel<<<any_grid(p.rows), kAnyThreads, 0, s>>>(p);
  return cudaGetLastError();
}

// ---- gradient --------------------------------------------------------------------------------------------
// dweight, before the rows' gradients replace anything: block (x, y) sums columns [256 x, 256 x + 256) over
// the rows y, y + groups, ... into the workspace; norm_grad_join_kernel adds the groups in order.
__global__ void __launch_bounds__(kAnyThreads) norm_grad_weight_any_kernel(NormGradPlan p) {
  const int64_t c = (int64_t)blockIdx.x * kAnyThreads + threadIdx.x;
  if (c >= p.n) return;
  float acc = 0.0f;
  for (int64_t row = blockIdx.y; row < p.rows; row += gridDim.y) {
    int64_t off[5];
    row_offsets(p.map, row, off);
    acc += load_plain(p.dy, p.dt, off[0] + c) * (load_plain(p.h, p.dt, off[1] + c) * p.rstd[row]);
  }
  p.ws[(int64_t)blockIdx.y * p.n + c] = acc;
}

__global__ void __launch_bounds__(kAnyThreads) norm_grad_join_kernel(const float* ws, float* dw, int64_t n, int64_t groups) {
  const int64_t c = (int64_t)blockIdx.x * kAnyThreads + threadIdx.x;
  if (c >= n) return;
  float acc = 0.0f;
  for (int64_t k = 0; k < groups; ++k) acc += ws[k * n + c];
  dw[c] = acc;
}

__global__ void __launch_bounds__(kAnyThreads) norm_grad_any_kernel(NormGradPlan p) {
  __shared__ float red[2 * kAnyThreads / 32];
  Philox g = {};
  if (p.drop.on) g = philox_of(p.drop);
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    int64_t off[5];
    row_offsets(p.map, row, off);
    const float r = p.rstd[row];
    float dot = 0.0f, none = 0.0f;
    for (int64_t c = threadIdx.x; c < p.n; c += kAnyThreads) {
      const float gy = load_plain(p.dy, p.dt, off[0] + c) * weight_at(p.w, p.w_dt, p.w_offset, c);
      dot = fmaf(gy, load_plain(p.h, p.dt, off[1] + c) * r, dot);
    }
    block_sum_max(dot, none, red);
    const float mean = __fdiv_rn(dot, (float)p.n);
    for (int64_t c = threadIdx.x; c < p.n; c += kAnyThreads) {
      const float gy = load_plain(p.dy, p.dt, off[0] + c) * weight_at(p.w, p.w_dt, p.w_offset, c);
      const float xh = load_plain(p.h, p.dt, off[1] + c) * r;
      float dh = r * (gy - xh * mean);
      if (p.dsum) dh += load_plain(p.dsum, p.dt, off[2] + c);
      store_from_f32(p.dh, p.dt, off[3] + c, dh);
      if (p.dx) store_from_f32(p.dx, p.dt, off[4] + c, drop1(p.drop, g, (uint64_t)(row * p.n + c), dh));
    }
    __syncthreads();  // red is used again by the next row
  }
}

int64_t norm_grad_partials(int64_t rows, int64_t n) {
  (void)n;
  return rows < 512 ? rows : 512;
}

cudaError_t launch_norm_grad(const NormGradPlan& p, cudaStream_t s) {
  if (p.dw) {
    const int64_t groups = norm_grad_partials(p.rows, p.n);
    const unsigned cols = (unsigned)((p.n + kAnyThreads - 1) / kAnyThreads);
    norm_grad_weight_any_kernel<<<dim3(cols, (unsigned)groups), kAnyThreads, 0, s>>>(p);
    norm_grad_join_kernel<<<cols, kAnyThreads, 0, s>>>(p.ws, p.dw, p.n, groups);
  }
  norm_grad_any_kernel<<<any_grid(p.rows), kAnyThreads, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace hlo
