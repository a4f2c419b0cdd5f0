// Attention with f32 queries over a cache of f32.
#include "attend_f32.cuh"

namespace hlo {

cudaError_t launch_attend_f32(AttendPlan& p, void* ws, cudaStream_t s) { return run_attend_f32_type<false>(p, ws, s); }

}  // namespace hlo
