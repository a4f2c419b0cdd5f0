// The norm's register kernels for f16.
#include "norm_kernel.cuh"

namespace hlo {

cudaError_t run_norm_f16(const NormPlan& p, const RowShape& r, bool cut, int whole, cudaStream_t s) {
  return run_norm<F16>(p, r, cut, whole, s);
}

}  // namespace hlo
