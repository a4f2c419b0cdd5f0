// The norm's register kernels for f32.
#include "norm_kernel.cuh"

namespace hlo {

cudaError_t run_norm_f32(const NormPlan& p, const RowShape& r, bool cut, int whole, cudaStream_t s) {
  return run_norm<F32>(p, r, cut, whole, s);
}

}  // namespace hlo
