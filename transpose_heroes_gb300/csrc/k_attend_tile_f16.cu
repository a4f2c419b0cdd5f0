// Attention for many rows a key head, f16 queries over a cache of their type.
#include "attend_tile.cuh"

namespace hlo {

cudaError_t launch_attend_tile_f16(AttendPlan& p, void* ws, cudaStream_t s) {
  return p.dim <= 64 ? run_attend_tile<F16, false, 64>(p, ws, s) : run_attend_tile<F16, false, 128>(p, ws, s);
}

}  // namespace hlo
