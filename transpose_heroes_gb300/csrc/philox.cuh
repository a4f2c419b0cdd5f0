// Philox4x32 with 10 rounds, the counter-based generator of Salmon, Moraes, Dror and Shaw ("Parallel
// Random Numbers: As Easy as 1, 2, 3", SC 2011), and the keep rule of a random mask drawn from it.
#pragma once
#include <cstdint>

#include "layer_plans.h"

namespace hlo {

struct Philox {
  uint32_t k0, k1, o0, o1;
};

// Seed and offset of a plan: its own, or (state given) those of the device words.
__device__ __forceinline__ Philox philox_of(const DropPlan& d) {
  uint64_t seed = d.seed, offset = d.offset;
  if (d.state) {
    seed = __ldg(reinterpret_cast<const unsigned long long*>(d.state));
    offset += __ldg(reinterpret_cast<const unsigned long long*>(d.state) + 1);
  }
  return {(uint32_t)seed, (uint32_t)(seed >> 32), (uint32_t)offset, (uint32_t)(offset >> 32)};
}

// The four words for counter `quad`.
__device__ __forceinline__ uint4 philox4(const Philox& g, uint64_t quad) {
  uint32_t c0 = (uint32_t)quad, c1 = (uint32_t)(quad >> 32), c2 = g.o0, c3 = g.o1;
  uint32_t k0 = g.k0, k1 = g.k1;
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t p0 = (uint64_t)0xD2511F53u * c0, p1 = (uint64_t)0xCD9E8D57u * c2;
    c0 = (uint32_t)(p1 >> 32) ^ c1 ^ k0;
    c1 = (uint32_t)p1;
    c2 = (uint32_t)(p0 >> 32) ^ c3 ^ k1;
    c3 = (uint32_t)p0;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return make_uint4(c0, c1, c2, c3);
}

// The word of element `i`.
__device__ __forceinline__ uint32_t philox_word(const Philox& g, uint64_t i) {
  const uint4 w = philox4(g, i >> 2);
  const uint32_t lo = (i & 1) ? w.y : w.x, hi = (i & 1) ? w.w : w.z;
  return (i & 2) ? hi : lo;
}

__device__ __forceinline__ bool kept(const DropPlan& d, uint32_t word) { return word >= d.threshold && !d.all; }

// drop(v) for element `i`: a select, so that a dropped NaN or infinity becomes 0 as well.
__device__ __forceinline__ float drop1(const DropPlan& d, const Philox& g, uint64_t i, float v) {
  return kept(d, philox_word(g, i)) ? __fmul_rn(v, d.scale) : 0.0f;
}

}  // namespace hlo
