// The norm's register kernels for bf16.
#include "norm_kernel.cuh"

namespace hlo {

cudaError_t run_norm_bf16(const NormPlan& p, const RowShape& r, bool cut, int whole, cudaStream_t s) {
  return run_norm<BF16>(p, r, cut, whole, s);
}

}  // namespace hlo
