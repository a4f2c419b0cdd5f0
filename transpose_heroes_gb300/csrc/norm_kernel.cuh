// The norm for rows held in registers (see k_norm.cu); compiled once per element type, in
// k_norm_f32.cu, k_norm_bf16.cu and k_norm_f16.cu.
#pragma once
#include "norm_common.cuh"

namespace hlo {

template <int DT>
__device__ __forceinline__ void store_row_vec(const NormPlan& p, int64_t at, const float (&y)[kVec<DT>], float inv) {
  constexpr int W = kVec<DT>;
  if (p.quant != NQ_NONE) {
    uint32_t u[2] = {0, 0};
#pragma unroll
    for (int e = 0; e < W; ++e) {
      uint8_t b;
      if (p.quant == NQ_STATIC) b = (uint8_t)quant_code(y[e], p.q.scale, p.q.inv_scale, p.q.zp, p.q.smin, p.q.smax);
      else if (p.out_dt == S8) b = (uint8_t)s8_code(y[e], inv);
      else b = f8_bits(__fmul_rn(y[e], inv));
      u[e >> 2] |= (uint32_t)b << (8 * (e & 3));
    }
    char* a = reinterpret_cast<char*>(p.out) + at;
    if (W == 8) *reinterpret_cast<uint2*>(a) = make_uint2(u[0], u[1]);
    else *reinterpret_cast<uint32_t*>(a) = u[0];
  } else if (p.out_dt == DT) {
    *reinterpret_cast<uint4*>(reinterpret_cast<char*>(p.out) + at * (16 / W)) = pack<DT>(y);
  } else {
#pragma unroll
    for (int q = 0; q < W / 4; ++q)
      *(reinterpret_cast<float4*>(reinterpret_cast<float*>(p.out) + at) + q) =
          make_float4(y[4 * q], y[4 * q + 1], y[4 * q + 2], y[4 * q + 3]);
  }
}

// One read and one write of everything: blockDim.x threads hold a row, K vectors of 16 bytes each, and the
// block blockDim.y rows. All of a thread's loads are issued before the first is used; sum is stored before
// the row's barrier, out after it.
// CUT: rows that start or end inside a vector (an odd length, a pitch): the vectors begin at the row's first
// 16-byte boundary, the same column in every operand, and the up to 2 W - 2 elements before and behind them
// go to a thread each.
// Bound: HBM. A row is read and written once, so the time is that of its bytes: 16384 x 8192 bf16 with
// residual (1074 MB) 157 us, 6.84 TB/s, the rate of a plain copy; cut rows, 32768 x 1001 bf16, 53 us (5.0 TB/s:
// the weights are shifted into place, and the ends are accesses of their own). With dropout the generator adds five
// wide multiplies an element: 8192 x 4096 (268 MB) 50 us, 5.4 TB/s, the issue slots and the multiplier each
// half busy. One token of 8192: 3.3 us a call, which is the launch.
template <int DT, int K, int DROP, bool CUT>
__global__ void __launch_bounds__(K == 1 ? 1024 : 512) norm_row_kernel(const __grid_constant__ NormPlan p, int weight_whole) {
  constexpr int W = kVec<DT>, EB = 16 / W;
  __shared__ float red[64];
  const int n = (int)p.n;
  follow();
  const int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  if (row >= p.rows) return;  // the whole group: its barrier is its own
  int64_t off[4];
  row_offsets(p.map, row, off);
  const RowCut cut = CUT ? row_cut<W>(p.x, EB, off[0], n) : RowCut{0, n};
  const int edge = CUT ? cut.edge(threadIdx.x, n) : -1;
  uint4 xr[K], rr[K];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int c0 = cut.head + (int)(threadIdx.x + k * blockDim.x) * W;
    xr[k] = rr[k] = make_uint4(0, 0, 0, 0);
    if (c0 >= cut.end) continue;
    xr[k] = load16(reinterpret_cast<const char*>(p.x) + (off[0] + c0) * EB);
    if (p.res) rr[k] = load16(reinterpret_cast<const char*>(p.res) + (off[1] + c0) * EB);
  }
  // one vector a thread is for few rows, where latency counts: the weights are requested with the row
  const bool whole_w = weight_whole && cut.head == 0, early_w = K == 1 && whole_w && p.w && p.w_dt == DT;
  uint4 wr = make_uint4(0, 0, 0, 0);
  if (early_w && cut.head + (int)threadIdx.x * W < cut.end) wr = load_kept(reinterpret_cast<const uint4*>(p.w) + threadIdx.x);
  const auto weights = [&](int c0, float (&w)[W]) {
    if (K == 1 && early_w) {
      unpack<DT>(wr, w);
      if (p.w_offset != 0.0f) {
#pragma unroll
        for (int e = 0; e < W; ++e) w[e] += p.w_offset;
      }
    } else {
      load_weights<DT>(p.w, p.w_dt, p.w_offset, c0, n, whole_w, w);
    }
  };
  float ve = 0.0f;
  if (CUT && edge >= 0) {
    ve = load_plain(p.x, DT, off[0] + edge);
    const float res = p.res ? load_plain(p.res, DT, off[1] + edge) : 0.0f;
    if constexpr (DROP != DROP_NONE) ve = drop1(p.drop, Philox<DROP>(p.drop), (uint64_t)(row * n + edge), ve);
    if (p.res) ve = __fadd_rn(res, ve);
    if (p.sum) store_from_f32(p.sum, DT, off[2] + edge, ve);
  }
  const Philox<DROP> g(p.drop);
  float v[K][W], ss = ve * ve, top = 0.0f;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int c0 = cut.head + (int)(threadIdx.x + k * blockDim.x) * W;
    unpack<DT>(xr[k], v[k]);
    float res[W];
    unpack<DT>(rr[k], res);  // +0 without a residual
    if constexpr (DROP != DROP_NONE) {
      drop_add_vec<DROP, !CUT, W>(p.drop, g, row * n + c0, v[k], res);
    } else if (p.res) {
#pragma unroll
      for (int e = 0; e < W; ++e) v[k][e] = __fadd_rn(res[e], v[k][e]);
    }
#pragma unroll
    for (int e = 0; e < W; ++e) ss = fmaf(v[k][e], v[k][e], ss);
    if (c0 >= cut.end) continue;
    if (p.sum) *reinterpret_cast<uint4*>(reinterpret_cast<char*>(p.sum) + (off[2] + c0) * EB) = pack<DT>(v[k]);
    if (p.quant == NQ_ROW) {
      float w[W];
      weights(c0, w);
#pragma unroll
      for (int e = 0; e < W; ++e) top = ieee_max(top, fabsf(v[k][e] * w[e]));
    }
  }
  const float we = CUT && edge >= 0 ? weight_at(p.w, p.w_dt, p.w_offset, edge) : 0.0f;
  if (CUT && edge >= 0) top = ieee_max(top, fabsf(ve * we));
  group_sum_max<true>(ss, top, red);
  const float r = rsqrtf(__fdiv_rn(ss, (float)p.n) + p.eps);
  if (threadIdx.x == 0 && p.rstd) p.rstd[row] = r;
  float inv = 0.0f;
  if (p.quant == NQ_ROW) {
    const float s = row_scale(r * top, p.out_dt);
    inv = __fdiv_rn(1.0f, s);
    if (threadIdx.x == 0) p.scales[row] = s;
  }
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int c0 = cut.head + (int)(threadIdx.x + k * blockDim.x) * W;
    if (c0 >= cut.end) continue;
    float w[W], y[W];
    weights(c0, w);
#pragma unroll
    for (int e = 0; e < W; ++e) y[e] = __fmul_rn(__fmul_rn(v[k][e], r), w[e]);
    store_row_vec<DT>(p, off[3] + c0, y, inv);
  }
  if (CUT && edge >= 0) store_out(p, off[3] + edge, __fmul_rn(__fmul_rn(ve, r), we), inv);
}

template <int DT, int K, int DROP>
cudaError_t run_norm_row(const NormPlan& p, const RowShape& r, bool cut, int whole, cudaStream_t s) {
  const dim3 block(r.tx, r.ty);
  const unsigned grid = (unsigned)((p.rows + r.ty - 1) / r.ty);
  return launch_after(cut ? norm_row_kernel<DT, K, DROP, true> : norm_row_kernel<DT, K, DROP, false>, grid, block, 0, s, 1, p, whole);
}

template <int DT>
cudaError_t run_norm(const NormPlan& p, const RowShape& r, bool cut, int whole, cudaStream_t s) {
#define HLO_CASE(KK)                                                                          \
  if (r.k == KK) {                                                                            \
    if (p.drop.mode == DROP_NONE) return run_norm_row<DT, KK, DROP_NONE>(p, r, cut, whole, s); \
    if (p.drop.mode == DROP_HOST) return run_norm_row<DT, KK, DROP_HOST>(p, r, cut, whole, s); \
    return run_norm_row<DT, KK, DROP_DEVICE>(p, r, cut, whole, s);                            \
  }
  HLO_CASE(1)
  HLO_CASE(2)
  HLO_CASE(4)
  HLO_CASE(8)
#undef HLO_CASE
  return cudaErrorInvalidValue;
}

}  // namespace hlo
