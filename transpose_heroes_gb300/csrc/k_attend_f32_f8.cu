// Attention with f32 queries over an f8E4M3FN cache.
#include "attend_f32.cuh"

namespace hlo {

cudaError_t launch_attend_f32_f8(AttendPlan& p, void* ws, cudaStream_t s) { return run_attend_f32_type<true>(p, ws, s); }

}  // namespace hlo
