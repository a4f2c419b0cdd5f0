// Dropout with a mask that is never stored: out = residual + drop(x) (philox.cuh).
#include "philox.cuh"
#include "rows.cuh"

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

cudaError_t launch_dropout(const DropoutPlan& p, cudaStream_t s) {
  const int64_t blocks = (p.rows * p.n + 255) / 256, cap = (int64_t)device_sm_count() * 64;
  dropout_any_kernel<<<(unsigned)(blocks < cap ? blocks : cap), 256, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace hlo
