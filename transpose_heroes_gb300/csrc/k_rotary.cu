// Rotary positions (hlo_rotary): each pair of a head turns by 2 pi frac(position * turns / 2^64).
#include "rows.cuh"

namespace hlo {

// The product is formed mod 2^64, i.e. exactly mod one turn; its high 32 bits, as a signed number of
// 2^-31 half turns, lose less than 2^-32 turn.
__device__ __forceinline__ float2 cos_sin(const RotaryPlan& p, int32_t pos, uint64_t turns) {
  const uint64_t t = (uint64_t)(int64_t)pos * turns;
  const float half_turns = (float)(int32_t)(t >> 32) * 0x1p-31f;
  float s, c;
  sincospif(half_turns, &s, &c);
  return make_float2(c * p.scale, s * p.sin_scale);
}

// A thread per pair, then per element that is copied.
__global__ void __launch_bounds__(256) rotary_any_kernel(RotaryPlan p, RotaryArray a, int64_t total) {
  const int per = p.dim - p.pairs;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    const int k = (int)(i % per);
    int64_t rest = i / per;
    const int64_t head = rest % a.heads;
    rest /= a.heads;
    const int64_t t = rest % p.seq, b = rest / p.seq;
    const int64_t in = b * a.in_stride[0] + t * a.in_stride[1] + head * a.in_stride[2];
    const int64_t out = b * a.out_stride[0] + t * a.out_stride[1] + head * a.out_stride[2];
    if (k >= p.pairs) {
      const int e = k + p.pairs;
      store_from_f32(a.out, p.dt, out + e, load_plain(a.in, p.dt, in + e));
      continue;
    }
    const int eu = p.interleaved ? 2 * k : k, ev = p.interleaved ? 2 * k + 1 : k + p.pairs;
    const float2 cs = cos_sin(p, p.pos[b * p.pos_stride[0] + t * p.pos_stride[1]], p.turns[k]);
    const float u = load_plain(a.in, p.dt, in + eu), v = load_plain(a.in, p.dt, in + ev);
    store_from_f32(a.out, p.dt, out + eu, u * cs.x - v * cs.y);
    store_from_f32(a.out, p.dt, out + ev, v * cs.x + u * cs.y);
  }
}

cudaError_t launch_rotary(const RotaryPlan& p, cudaStream_t s) {
  for (int k = 0; k < p.arrays; ++k) {
    const int64_t total = p.batch * p.seq * p.a[k].heads * (p.dim - p.pairs);
    const int64_t blocks = (total + 255) / 256, cap = (int64_t)device_sm_count() * 64;
    rotary_any_kernel<<<(unsigned)(blocks < cap ? blocks : cap), 256, 0, s>>>(p, p.a[k], total);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace hlo
