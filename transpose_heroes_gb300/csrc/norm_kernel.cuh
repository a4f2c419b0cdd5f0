// The norm for rows held in registers (see k_norm.cu); compiled once per element type, in
// k_norm_f32.cu, k_norm_bf16.cu and k_norm_f16.cu.
#pragma once
#include "norm_common.cuh"

namespace hlo {

// W codes with the row's scale; inv = RN(1 / scale).
template <int DT>
__device__ __forceinline__ void store_row_codes(const NormPlan& p, int64_t at, const float (&y)[kVec<DT>], float scale, float inv) {
  constexpr int W = kVec<DT>;
  char* a = reinterpret_cast<char*>(p.out) + at;
  const uint32_t u = codes(make_float4(y[0], y[1], y[2], y[3]), scale, inv, p.out_dt == F8);
  if constexpr (W == 8)
    *reinterpret_cast<uint2*>(a) = make_uint2(u, codes(make_float4(y[4], y[5], y[6], y[7]), scale, inv, p.out_dt == F8));
  else
    *reinterpret_cast<uint32_t*>(a) = u;
}

template <int DT>
__device__ __forceinline__ void store_row_vec(const NormPlan& p, int64_t at, const float (&y)[kVec<DT>]) {
  constexpr int W = kVec<DT>;
  if (p.quant == NQ_STATIC) {
    uint32_t u[2] = {0, 0};
#pragma unroll
    for (int e = 0; e < W; ++e)
      u[e >> 2] |= (uint32_t)(uint8_t)quant_code(y[e], p.q.scale, p.q.inv_scale, p.q.zp, p.q.smin, p.q.smax) << (8 * (e & 3));
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
// residual (1074 MB) 157 us, 6.84 TB/s, the rate of a plain copy, and 147 us to f8 with scales
// (940 MB, 6.4 TB/s); cut rows, 32768 x 1001 bf16, 52 us (5.1 TB/s: the weights are shifted into place, and the ends are
// accesses of their own). With dropout the generator adds five
// wide multiplies an element: 8192 x 4096 (268 MB) 48 us, 5.6 TB/s, the issue slots, the multiplier and the
// ALU each over half busy. One token of 8192: 3.1 to 3.7 us a call, which is the launch (2.3 in a captured graph).
template <int DT, int K, int DROP, bool CUT>
__global__ void __launch_bounds__(K == 1 ? 1024 : 512) norm_row_kernel(const __grid_constant__ NormPlan p, int weight_whole) {
  constexpr int W = kVec<DT>, EB = 16 / W;
  __shared__ float red[64];
  __shared__ uint32_t tops[32];
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
  float v[K][W], ss = ve * ve;
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
  }
  group_sum(ss, red);
  const float r = rsqrtf(__fdiv_rn(ss, (float)p.n) + p.eps);
  if (threadIdx.x == 0 && p.rstd) p.rstd[row] = r;
  if (CUT && edge >= 0) ve = __fmul_rn(__fmul_rn(ve, r), weight_at(p.w, p.w_dt, p.w_offset, edge));
  float scale = 0.0f;
  if (p.quant == NQ_ROW) {  // v becomes y; the scale is that of the largest |y|, a second reduction
    uint32_t top = magnitude(ve);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c0 = cut.head + (int)(threadIdx.x + k * blockDim.x) * W;
      if (c0 >= cut.end) continue;
      float w[W];
      weights(c0, w);
#pragma unroll
      for (int e = 0; e < W; ++e) {
        v[k][e] = __fmul_rn(__fmul_rn(v[k][e], r), w[e]);
        top = max(top, magnitude(v[k][e]));
      }
    }
    scale = row_scale(group_max(top, tops), p.out_dt);
    const float inv = __fdiv_rn(1.0f, scale);
    if (threadIdx.x == 0) p.scales[row] = scale;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c0 = cut.head + (int)(threadIdx.x + k * blockDim.x) * W;
      if (c0 < cut.end) store_row_codes<DT>(p, off[3] + c0, v[k], scale, inv);
    }
  } else {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c0 = cut.head + (int)(threadIdx.x + k * blockDim.x) * W;
      if (c0 >= cut.end) continue;
      float w[W], y[W];
      weights(c0, w);
#pragma unroll
      for (int e = 0; e < W; ++e) y[e] = __fmul_rn(__fmul_rn(v[k][e], r), w[e]);
      store_row_vec<DT>(p, off[3] + c0, y);
    }
  }
  if (CUT && edge >= 0) store_out(p, off[3] + edge, ve, scale);
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
