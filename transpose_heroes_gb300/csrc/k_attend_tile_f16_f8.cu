// Attention for many rows a key head, f16 queries over an f8E4M3FN cache.
#include "attend_tile.cuh"

namespace hlo {

cudaError_t launch_attend_tile_f16_f8(AttendPlan& p, void* ws, cudaStream_t s) { return run_attend_tile_type<F16, true>(p, ws, s); }

}  // namespace hlo
