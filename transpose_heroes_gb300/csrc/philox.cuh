// Philox4x32 with 10 rounds, the counter-based generator of Salmon, Moraes, Dror and Shaw ("Parallel
// Random Numbers: As Easy as 1, 2, 3", SC 2011), and the keep rule of a random mask drawn from it.
#pragma once
#include <cstdint>

#include "layer_plans.h"

namespace hlo {

constexpr uint32_t kPhiloxM0 = 0xD2511F53u, kPhiloxM1 = 0xCD9E8D57u;  // multipliers
constexpr uint32_t kPhiloxW0 = 0x9E3779B9u, kPhiloxW1 = 0xBB67AE85u;  // key increments

// Host: the constants of a plan with this seed and offset. For a counter (q, 0, o0, o1) the first round's
// product M1 o0 is the same for every q; so is then the second round's M0 c0.
inline void philox_constants(DropPlan* d, uint64_t seed, uint64_t offset) {
  for (int r = 0; r < 10; ++r) {
    d->key[2 * r] = (uint32_t)seed + (uint32_t)r * kPhiloxW0;
    d->key[2 * r + 1] = (uint32_t)(seed >> 32) + (uint32_t)r * kPhiloxW1;
  }
  const uint64_t p1 = (uint64_t)kPhiloxM1 * (uint32_t)offset;         // round 1
  const uint64_t p0 = (uint64_t)kPhiloxM0 * ((uint32_t)(p1 >> 32) ^ d->key[0]);  // round 2
  d->x1 = (uint32_t)(offset >> 32) ^ d->key[1];
  d->y2 = (uint32_t)p1 ^ d->key[2];
  d->x2 = (uint32_t)(p0 >> 32) ^ d->key[3];
  d->y3 = (uint32_t)p0 ^ d->key[5];
}

// What a thread holds of the generator: nothing with DROP_HOST, seed and offset with DROP_DEVICE.
template <int MODE>
struct Philox {
  uint32_t k0 = 0, k1 = 0, o0 = 0, o1 = 0;
  __device__ __forceinline__ explicit Philox(const DropPlan& d) {
    if constexpr (MODE == DROP_DEVICE) {
      uint64_t seed = d.seed, offset = d.offset;
      if (d.state) {
        seed = reinterpret_cast<const unsigned long long*>(d.state)[0];
        offset += reinterpret_cast<const unsigned long long*>(d.state)[1];
      }
      k0 = (uint32_t)seed, k1 = (uint32_t)(seed >> 32), o0 = (uint32_t)offset, o1 = (uint32_t)(offset >> 32);
    }
  }
  // The four words for counter `quad` (DROP_HOST: below 2^32).
  __device__ __forceinline__ uint4 words(const DropPlan& d, uint64_t quad) const {
    uint32_t c0, c1, c2, c3;
    if constexpr (MODE == DROP_HOST) {
      uint64_t p0 = (uint64_t)kPhiloxM0 * (uint32_t)quad;                               // round 1
      uint64_t p1 = (uint64_t)kPhiloxM1 * ((uint32_t)(p0 >> 32) ^ d.x1);     // round 2
      c0 = (uint32_t)(p1 >> 32) ^ d.y2, c1 = (uint32_t)p1, c2 = (uint32_t)p0 ^ d.x2;
      p0 = (uint64_t)kPhiloxM0 * c0, p1 = (uint64_t)kPhiloxM1 * c2;          // round 3
      c0 = (uint32_t)(p1 >> 32) ^ c1 ^ d.key[4], c1 = (uint32_t)p1, c2 = (uint32_t)(p0 >> 32) ^ d.y3, c3 = (uint32_t)p0;
    } else {
      c0 = (uint32_t)quad, c1 = (uint32_t)(quad >> 32), c2 = o0, c3 = o1;
    }
#pragma unroll
    for (int r = MODE == DROP_HOST ? 3 : 0; r < 10; ++r) {
      const uint64_t p0 = (uint64_t)kPhiloxM0 * c0, p1 = (uint64_t)kPhiloxM1 * c2;
      c0 = (uint32_t)(p1 >> 32) ^ c1 ^ (MODE == DROP_HOST ? d.key[2 * r] : k0 + r * kPhiloxW0);
      c1 = (uint32_t)p1;
      c2 = (uint32_t)(p0 >> 32) ^ c3 ^ (MODE == DROP_HOST ? d.key[2 * r + 1] : k1 + r * kPhiloxW1);
      c3 = (uint32_t)p0;
    }
    return make_uint4(c0, c1, c2, c3);
  }
};

__device__ __forceinline__ bool kept(const DropPlan& d, uint32_t word) { return word >= d.threshold && !d.all; }

// drop(v): a select, so that a dropped NaN or infinity becomes 0 as well.
__device__ __forceinline__ float dropped(const DropPlan& d, uint32_t word, float v) {
  return kept(d, word) ? __fmul_rn(v, d.scale) : 0.0f;
}

// drop(v) for element `i` alone.
template <int MODE>
__device__ __forceinline__ float drop1(const DropPlan& d, const Philox<MODE>& g, uint64_t i, float v) {
  const uint4 w = g.words(d, i >> 2);
  const uint32_t lo = (i & 1) ? w.y : w.x, hi = (i & 1) ? w.w : w.z;
  return dropped(d, (i & 2) ? hi : lo, v);
}

}  // namespace hlo
