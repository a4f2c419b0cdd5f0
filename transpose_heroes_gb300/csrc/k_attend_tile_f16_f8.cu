// Attention for many rows a key head, f16 queries over an f8E4M3FN cache.
#include "attend_tile.cuh"

namespace hlo {

cudaError_t launch_attend_tile_f16_f8(AttendPlan& p, void* ws, cudaStream_t s) {
  return p.dim <= 64 ? run_attend_tile<F16, true, 64>(p, ws, s) : run_attend_tile<F16, true, 128>(p, ws, s);
}

}  // namespace hlo
