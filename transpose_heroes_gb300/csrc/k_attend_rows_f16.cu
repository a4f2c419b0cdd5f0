// Attention for few rows a key head, f16 queries over a cache of their type.
#include "attend_rows.cuh"

namespace hlo {

cudaError_t launch_attend_rows_f16(AttendPlan& p, void* ws, cudaStream_t s) { return run_attend_rows_type<F16, false>(p, ws, s); }

}  // namespace hlo
