// Dropout with a mask that is never stored: out = residual + drop(x) (philox.cuh).
//
//  dropout_vec_kernel -- operands aligned alike: vectors of 16 bytes. Rows that follow one another were merged
//                        into one by the caller, so a dense array is one row and a row's ends cost nothing.
//  dropout_any_kernel -- any alignment: a thread per element.
#include <algorithm>

#include "vectors.cuh"

namespace hlo {

__global__ void __launch_bounds__(256) dropout_any_kernel(DropoutPlan p) {
  const Philox g = philox_of(p.drop);
  const int64_t total = p.rows * p.n;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    const int64_t row = i / p.n, c = i - row * p.n;
    int64_t off[3];
    row_offsets(p.map, row, off);
    float v = drop1(p.drop, g, (uint64_t)i, load_plain(p.x, p.dt, off[0] + c));
    if (p.res) v = __fadd_rn(load_plain(p.res, p.dt, off[1] + c), v);
    store_from_f32(p.out, p.dt, off[2] + c, v);
  }
}

// Block (x, y): blockDim.x U vectors of the rows y, y + gridDim.y, ...; all loads of a thread first.
template <int DT, int U>
__global__ void __launch_bounds__(256) dropout_vec_kernel(DropoutPlan p) {
  constexpr int W = kVec<DT>, EB = 16 / W;
  const Philox g = philox_of(p.drop);
  for (int64_t row = blockIdx.y; row < p.rows; row += gridDim.y) {
    int64_t off[3];
    row_offsets(p.map, row, off);
    const int shift = (int)(((int64_t)((uintptr_t)p.x / EB) + off[0]) & (W - 1));
    const int64_t first = ((int64_t)blockIdx.x * blockDim.x * U + threadIdx.x) * W - shift;
    uint4 xr[U], rr[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t c0 = first + (int64_t)u * blockDim.x * W;
      xr[u] = rr[u] = make_uint4(0, 0, 0, 0);
      if (c0 >= p.n) continue;
      xr[u] = load_cut<DT>(p.x, off[0], c0, p.n);
      if (p.res) rr[u] = load_cut<DT>(p.res, off[1], c0, p.n);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t c0 = first + (int64_t)u * blockDim.x * W;
      if (c0 >= p.n) continue;
      float v[W];
      unpack<DT>(xr[u], v);
      drop_vec<W>(p.drop, g, row * p.n + c0, v);
      if (p.res) {
        float r[W];
        unpack<DT>(rr[u], r);
#pragma unroll
        for (int e = 0; e < W; ++e) v[e] = __fadd_rn(r[e], v[e]);
      }
      store_cut<DT>(p.out, off[2], c0, p.n, v);
    }
  }
}

template <int DT>
cudaError_t run_dropout(const DropoutPlan& p, cudaStream_t s) {
  constexpr int W = kVec<DT>;
  const int64_t vectors = (p.n + W - 1) / W + 1;
  const int threads = (int)std::min<int64_t>(256, (vectors + 31) / 32 * 32);
  const unsigned rows = (unsigned)std::min<int64_t>(p.rows, 65535);
  // four vectors a thread once that still leaves every SM several blocks
  if (vectors * (int64_t)rows >= (int64_t)device_sm_count() * 8192) {
    const int64_t blocks = (vectors + threads * 4 - 1) / (threads * 4);
    dropout_vec_kernel<DT, 4><<<dim3((unsigned)blocks, rows), threads, 0, s>>>(p);
  } else {
    const int64_t blocks = (vectors + threads - 1) / threads;
    dropout_vec_kernel<DT, 1><<<dim3((unsigned)blocks, rows), threads, 0, s>>>(p);
  }
  return cudaGetLastError();
}

cudaError_t launch_dropout(const DropoutPlan& p, cudaStream_t s) {
  const int w = p.dt == F32 ? 4 : 8, eb = dt_bytes(p.dt);
  const void* const ptr[3] = {p.x, p.res, p.out};
  const int ebs[3] = {eb, eb, eb};
  bool cut = false;
  if (p.n / w < (int64_t)INT32_MAX * 128 && vectors_fit<3>(p.map, ptr, ebs, p.n, w, &cut)) {
    if (p.dt == F32) return run_dropout<F32>(p, s);
    if (p.dt == BF16) return run_dropout<BF16>(p, s);
    return run_dropout<F16>(p, s);
  }
  const int64_t blocks = (p.rows * p.n + 255) / 256, cap = (int64_t)device_sm_count() * 64;
  dropout_any_kernel<<<(unsigned)std::min(blocks, cap), 256, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace hlo
