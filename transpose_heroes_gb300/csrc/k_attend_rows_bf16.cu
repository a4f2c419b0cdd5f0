// Attention for few rows a key head, bf16 queries over a cache of their type.
#include "attend_rows.cuh"

namespace hlo {

cudaError_t launch_attend_rows_bf16(AttendPlan& p, void* ws, cudaStream_t s) { return run_attend_rows_type<BF16, false>(p, ws, s); }

}  // namespace hlo
