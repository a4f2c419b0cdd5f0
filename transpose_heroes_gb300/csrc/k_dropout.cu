// Dropout with a mask that is never stored: out = residual + drop(x) (philox.cuh).
//
//  dropout_flat_kernel -- dense operands on 16-byte boundaries (rows that follow one another were merged into
//                         one by the caller).
//  dropout_row_kernel  -- rows that are aligned alike: vectors of 16 bytes, cut off at the rows' ends.
//  dropout_any_kernel  -- any alignment: a thread per element.
#include <algorithm>

#include "vectors.cuh"

namespace hlo {

template <int MODE>
__global__ void __launch_bounds__(256) dropout_any_kernel(const __grid_constant__ DropoutPlan p) {
  const Philox<MODE> g(p.drop);
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

// Dense operands, aligned to 16 bytes (one row): persistent blocks whose threads take vectors in turn, two
// vectors ahead of the one they work on. A loop that is not unrolled, so that the generator's ten rounds
// are in flight for one vector at a time and registers leave room for many warps.
// Bound: the wide multiplies (18 for the words of four elements; that pipe is 69% busy) beside HBM: 2^27 bf16
// elements with residual (805 MB) 132 us, 6.1 TB/s, 90% of the copy rate. Four vectors a thread at once (94
// registers, half the warps) took 170 us, two with spills 144.
template <int DT, int MODE, bool RES>
__global__ void __launch_bounds__(256, 4) dropout_flat_kernel(const __grid_constant__ DropoutPlan p) {
  constexpr int W = kVec<DT>;
  follow();
  const Philox<MODE> g(p.drop);
  const uint4* const x = reinterpret_cast<const uint4*>(p.x);
  const uint4* const res = reinterpret_cast<const uint4*>(p.res);
  uint4* const out = reinterpret_cast<uint4*>(p.out);
  const int64_t whole = p.n / W, step = (int64_t)gridDim.x * 256;
  int64_t j = (int64_t)blockIdx.x * 256 + threadIdx.x;
  uint4 x1 = {}, x2 = {}, r1 = {}, r2 = {};
  if (j < whole) {
    x1 = load16(x + j);
    if (RES) r1 = load16(res + j);
  }
  if (j + step < whole) {
    x2 = load16(x + j + step);
    if (RES) r2 = load16(res + j + step);
  }
#pragma unroll 1
  for (; j < whole; j += step) {
    float v[W], r[W];
    unpack<DT>(x1, v);
    if (RES) unpack<DT>(r1, r);
    x1 = x2, r1 = r2;
    const int64_t next = j + 2 * step;
    if (next < whole) {
      x2 = load16(x + next);
      if (RES) r2 = load16(res + next);
    }
    if constexpr (RES) drop_add_vec<MODE, true, W>(p.drop, g, j * W, v, r);
    else drop_vec<MODE, true, W>(p.drop, g, j * W, v);
    out[j] = pack<DT>(v);
  }
  // the elements after the last whole vector
  if (blockIdx.x == 0 && threadIdx.x < p.n - whole * W) {
    const int64_t i = whole * W + threadIdx.x;
    float v = drop1(p.drop, g, (uint64_t)i, load_plain(p.x, DT, i));
    if (RES) v = __fadd_rn(load_plain(p.res, DT, i), v);
    store_from_f32(p.out, DT, i, v);
  }
}

// Rows that are aligned alike, but not all of them, or not one dense run: block (x, y) does blockDim.x vectors
// of the rows y, y + gridDim.y, ...
template <int DT, int MODE, bool RES>
__global__ void __launch_bounds__(256) dropout_row_kernel(const __grid_constant__ DropoutPlan p) {
  constexpr int W = kVec<DT>, EB = 16 / W;
  follow();
  const Philox<MODE> g(p.drop);
  for (int64_t row = blockIdx.y; row < p.rows; row += gridDim.y) {
    int64_t off[3];
    row_offsets(p.map, row, off);
    const int shift = (int)(((int64_t)((uintptr_t)p.x / EB) + off[0]) & (W - 1));
    const int64_t c0 = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) * W - shift;
    if (c0 >= p.n) continue;
    float v[W], r[W];
    unpack<DT>(load_cut<DT>(p.x, off[0], c0, p.n, p.end[0]), v);
    if constexpr (RES) {
      unpack<DT>(load_cut<DT>(p.res, off[1], c0, p.n, p.end[1]), r);
      drop_add_vec<MODE, false, W>(p.drop, g, row * p.n + c0, v, r);
    } else {
      drop_vec<MODE, false, W>(p.drop, g, row * p.n + c0, v);
    }
    store_cut<DT>(p.out, off[2], c0, p.n, v);
  }
}

template <int DT, int MODE>
cudaError_t run_dropout(const DropoutPlan& p, bool flat, cudaStream_t s) {
  constexpr int W = kVec<DT>;
  if (flat) {
    const auto kernel = p.res ? dropout_flat_kernel<DT, MODE, true> : dropout_flat_kernel<DT, MODE, false>;
    const int64_t cap = (int64_t)device_sm_count() * kernel_blocks_per_sm((const void*)kernel, 256, 0);
    const int64_t blocks = std::max<int64_t>(1, std::min(cap, (p.n / W + 255) / 256));
    return launch_after(kernel, dim3((unsigned)blocks), dim3(256), 0, s, 1, p);
  }
  const int64_t vectors = (p.n + W - 1) / W + 1;
  const int threads = (int)std::min<int64_t>(256, (vectors + 31) / 32 * 32);
  const unsigned rows = (unsigned)std::min<int64_t>(p.rows, 65535);
  const dim3 grid((unsigned)((vectors + threads - 1) / threads), rows);
  return launch_after(p.res ? dropout_row_kernel<DT, MODE, true> : dropout_row_kernel<DT, MODE, false>, grid, dim3(threads), 0, s, 1, p);
}

template <int MODE>
cudaError_t run_dropout_mode(const DropoutPlan& p, cudaStream_t s) {
  const int w = p.dt == F32 ? 4 : 8, eb = dt_bytes(p.dt);
  const void* const ptr[3] = {p.x, p.res, p.out};
  const int ebs[3] = {eb, eb, eb};
  bool cut = false;
  if (p.n / w < (int64_t)INT32_MAX * 32 && vectors_fit<3>(p.map, ptr, ebs, p.n, w, &cut)) {
    const bool flat = p.rows == 1 && ((uintptr_t)p.x | (uintptr_t)p.res | (uintptr_t)p.out) % 16 == 0;
    if (p.dt == F32) return run_dropout<F32, MODE>(p, flat, s);
    if (p.dt == BF16) return run_dropout<BF16, MODE>(p, flat, s);
    return run_dropout<F16, MODE>(p, flat, s);
  }
  const int64_t blocks = (p.rows * p.n + 255) / 256, cap = (int64_t)device_sm_count() * 64;
  dropout_any_kernel<MODE><<<(unsigned)std::min(blocks, cap), 256, 0, s>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_dropout(const DropoutPlan& p, cudaStream_t s) {
  return p.drop.mode == DROP_DEVICE ? run_dropout_mode<DROP_DEVICE>(p, s) : run_dropout_mode<DROP_HOST>(p, s);
}

}  // namespace hlo
