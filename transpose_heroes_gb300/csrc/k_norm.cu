// Root-mean-square norm with the residual's addition: out = h r w, h = residual + drop(x). See hlo_rms_norm
// in hlo_fusion.h for the formulas.
//
//  norm_row_kernel -- rows of up to 32768 elements (16384 in f32) whose operands are aligned alike: the row
//                     stays in registers, one read and one write of everything.
//  norm_any_kernel -- any length and alignment: a block per row, threads take elements in turn, and the row
//                     is read twice (three times for 8 bits with scales; from L2 but for the first time). A thread reads and writes the same elements
//                     in every pass, so outputs may replace inputs in place.
#include "norm_common.cuh"

namespace hlo {

template <int DROP>
__global__ void __launch_bounds__(kAnyThreads) norm_any_kernel(const __grid_constant__ NormPlan p) {
  __shared__ float red[2 * kAnyThreads / 32];
  const Philox<DROP> g(p.drop);
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    int64_t off[4];
    row_offsets(p.map, row, off);
    auto h_at = [&](int64_t c) {
      float v = load_plain(p.x, p.dt, off[0] + c);
      if constexpr (DROP != DROP_NONE) v = drop1(p.drop, g, (uint64_t)(row * p.n + c), v);
      return p.res ? __fadd_rn(load_plain(p.res, p.dt, off[1] + c), v) : v;
    };
    const auto y_at = [&](int64_t c, float h, float r) { return __fmul_rn(__fmul_rn(h, r), weight_at(p.w, p.w_dt, p.w_offset, c)); };
    float ss = 0.0f, top = 0.0f;
    for (int64_t c = threadIdx.x; c < p.n; c += kAnyThreads) {
      const float h = h_at(c);
      ss = fmaf(h, h, ss);
    }
    block_sum_max(ss, top, red);
    const float r = rsqrtf(__fdiv_rn(ss, (float)p.n) + p.eps);
    if (threadIdx.x == 0 && p.rstd) p.rstd[row] = r;
    float scale = 0.0f;
    if (p.quant == NQ_ROW) {
      float none = 0.0f;
      for (int64_t c = threadIdx.x; c < p.n; c += kAnyThreads) top = ieee_max(top, fabsf(y_at(c, h_at(c), r)));
      __syncthreads();  // red is read
      block_sum_max(none, top, red);
      scale = row_scale(top, p.out_dt);
      if (threadIdx.x == 0) p.scales[row] = scale;
    }
    for (int64_t c = threadIdx.x; c < p.n; c += kAnyThreads) {
      const float h = h_at(c);
      if (p.sum) store_from_f32(p.sum, p.dt, off[2] + c, h);
      store_out(p, off[3] + c, y_at(c, h, r), scale);
    }
    __syncthreads();  // red is used again by the next row
  }
}

cudaError_t launch_norm(const NormPlan& p, cudaStream_t s) {
  const int w = p.dt == F32 ? 4 : 8, eb = dt_bytes(p.dt);
  const void* const ptr[4] = {p.x, p.res, p.sum, p.out};
  const int ebs[4] = {eb, eb, eb, view_dt_bytes(p.out_dt)};
  bool cut = false;
  const int64_t vectors = (p.n + w - 1) / w;
  if (vectors <= 512 * 8 && p.rows <= INT32_MAX && vectors_fit<4>(p.map, ptr, ebs, p.n, w, &cut)) {
    // up to four vectors a thread, as long as a warp's lanes are all used. 2^26 bf16 elements with residual: 82 us
    // with four (1024 to 16384 columns), 85 to 93 with two, 105 to 144 with one
    const RowShape r = row_shape(p.rows, vectors, 8, 24);
    const int whole = p.w && (uintptr_t)p.w % 16 == 0;
    if (p.dt == F32) return run_norm_f32(p, r, cut, whole, s);
    if (p.dt == BF16) return run_norm_bf16(p, r, cut, whole, s);
    return run_norm_f16(p, r, cut, whole, s);
  }
  if (p.drop.mode == DROP_NONE) norm_any_kernel<DROP_NONE><<<any_grid(p.rows), kAnyThreads, 0, s>>>(p);
  else if (p.drop.mode == DROP_HOST) norm_any_kernel<DROP_HOST><<<any_grid(p.rows), kAnyThreads, 0, s>>>(p);
  else norm_any_kernel<DROP_DEVICE><<<any_grid(p.rows), kAnyThreads, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace hlo
