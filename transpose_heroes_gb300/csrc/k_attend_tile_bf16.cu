// Attention for many rows a key head, bf16 queries over a cache of their type.
#include "attend_tile.cuh"

namespace hlo {

cudaError_t launch_attend_tile_bf16(AttendPlan& p, void* ws, cudaStream_t s) { return run_attend_tile_type<BF16, false>(p, ws, s); }

}  // namespace hlo
