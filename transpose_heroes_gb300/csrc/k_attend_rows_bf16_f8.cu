// Attention for few rows a key head, bf16 queries over an f8E4M3FN cache.
#include "attend_rows.cuh"

namespace hlo {

cudaError_t launch_attend_rows_bf16_f8(AttendPlan& p, void* ws, cudaStream_t s) { return run_attend_rows_type<BF16, true>(p, ws, s); }

}  // namespace hlo
