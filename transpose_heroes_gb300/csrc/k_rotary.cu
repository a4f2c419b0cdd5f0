// Rotary positions (hlo_rotary): each pair of a head turns by 2 pi frac(position * turns / 2^64).
#include <algorithm>

#include "vectors.cuh"

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

// V elements of a 16-bit or 32-bit type as one access of V elements.
template <int DT, int V>
struct Piece {
  static constexpr int EB = DT == F32 ? 4 : 2;
  static constexpr int N = V * EB >= 4 ? V * EB / 4 : 1;
  uint32_t u[N];
  __device__ __forceinline__ void load(const void* p, int64_t i) {
    const char* a = reinterpret_cast<const char*>(p) + i * EB;
    if constexpr (V * EB == 16) {
      const uint4 w = load16(a);
      u[0] = w.x, u[1] = w.y, u[2] = w.z, u[3] = w.w;
    } else if constexpr (V * EB == 8) {
      const uint2 w = __ldcs(reinterpret_cast<const uint2*>(a));
      u[0] = w.x, u[1] = w.y;
    } else if constexpr (V * EB == 4) {
      u[0] = __ldcs(reinterpret_cast<const uint32_t*>(a));
    } else {
      u[0] = __ldcs(reinterpret_cast<const uint16_t*>(a));
    }
  }
  __device__ __forceinline__ void store(void* p, int64_t i) const {
    char* a = reinterpret_cast<char*>(p) + i * EB;
    if constexpr (V * EB == 16) *reinterpret_cast<uint4*>(a) = make_uint4(u[0], u[1], u[2], u[3]);
    else if constexpr (V * EB == 8) *reinterpret_cast<uint2*>(a) = make_uint2(u[0], u[1]);
    else if constexpr (V * EB == 4) *reinterpret_cast<uint32_t*>(a) = u[0];
    else *reinterpret_cast<uint16_t*>(a) = (uint16_t)u[0];
  }
  __device__ __forceinline__ void get(float (&v)[V]) const {
#pragma unroll
    for (int e = 0; e < V; ++e) {
      if constexpr (DT == F32) v[e] = __uint_as_float(u[e]);
      else if constexpr (DT == BF16) v[e] = __uint_as_float((e & 1) ? (u[e / 2] & 0xFFFF0000u) : (u[e / 2] << 16));
      else v[e] = f16_bits_to_f32((uint16_t)(u[e / 2] >> (16 * (e & 1))));
    }
  }
  __device__ __forceinline__ void set(const float (&v)[V]) {
    if constexpr (DT == F32) {
#pragma unroll
      for (int e = 0; e < V; ++e) u[e] = __float_as_uint(v[e]);
    } else if constexpr (V == 1) {
      u[0] = DT == BF16 ? f32_to_bf16_bits(v[0]) : f32_to_f16_bits(v[0]);
    } else {
#pragma unroll
      for (int e = 0; e < V; e += 2) {
        if constexpr (DT == BF16) {
          const __nv_bfloat162 h = __floats2bfloat162_rn(v[e], v[e + 1]);
          u[e / 2] = *reinterpret_cast<const uint32_t*>(&h);
        } else {
          const __half2 h = __floats2half2_rn(v[e], v[e + 1]);
          u[e / 2] = *reinterpret_cast<const uint32_t*>(&h);
        }
      }
    }
  }
};

struct RotaryTile {
  int tokens;        // tokens a block
  int heads;         // heads (of both arrays together) a block
  int per_head;      // items a head: turned ones, then copied ones
  int turned;        // pairs / V
  int copied;        // copied elements / V
};

// A block turns `heads` heads (of x's and then y's) of `tokens` tokens. It first computes the cosine and sine of
// each (token, pair) once, into shared memory; an item is then two accesses of V elements: the two halves
// of V pairs (half layout) or V adjacent pairs (interleaved), or 2 V copied elements. Each thread issues the loads
// of its first U items before the cosines are there.
template <int DT, int V, int U, bool INTER>
__global__ void __launch_bounds__(256) rotary_kernel(RotaryPlan p, RotaryTile t, int64_t total_tokens, int total_heads) {
  extern __shared__ float2 cs[];
  const int64_t token0 = (int64_t)blockIdx.x * t.tokens;
  const int tokens = (int)(total_tokens - token0 < t.tokens ? total_tokens - token0 : t.tokens);
  const int head0 = blockIdx.y * t.heads;
  const int heads = total_heads - head0 < t.heads ? total_heads - head0 : t.heads;
  const int items = tokens * heads * t.per_head;
  for (int base = 0; base < items; base += 256 * U) {
    Piece<DT, V> a[U], b[U];
    int64_t out_at[U];
    int where[U];  // cosines' place, or -1: copied
    int ea[U], eb[U], which[U];
#pragma unroll
    for (int q = 0; q < U; ++q) {
      const int i = base + q * 256 + threadIdx.x;
      which[q] = -1;
      if (i >= items) continue;
      const int hi = i / t.per_head, k = i - hi * t.per_head;
      const int tok = hi / heads;
      int head = head0 + hi - tok * heads;
      which[q] = p.arrays > 1 && head >= p.a[0].heads ? 1 : 0;
      const RotaryArray& r = which[q] ? p.a[1] : p.a[0];
      if (which[q]) head -= (int)p.a[0].heads;
      const uint32_t g = (uint32_t)(token0 + tok), bi = p.batch > 1 ? g / (uint32_t)p.seq : 0, si = g - bi * (uint32_t)p.seq;
      const int64_t in = bi * r.in_stride[0] + si * r.in_stride[1] + head * r.in_stride[2];
      out_at[q] = bi * r.out_stride[0] + si * r.out_stride[1] + head * r.out_stride[2];
      if (k < t.turned) {
        where[q] = tok * p.pairs + k * V;
        ea[q] = INTER ? 2 * k * V : k * V;
        eb[q] = INTER ? ea[q] + V : ea[q] + p.pairs;
      } else {
        where[q] = -1;
        ea[q] = 2 * p.pairs + 2 * (k - t.turned) * V;
        eb[q] = 2 * (k - t.turned) + 1 < t.copied ? ea[q] + V : -1;
      }
      a[q].load(r.in, in + ea[q]);
      if (eb[q] >= 0) b[q].load(r.in, in + eb[q]);
    }
    if (base == 0) {
      for (int i = threadIdx.x; i < tokens * p.pairs; i += 256) {
        const int tok = i / p.pairs, k = i - tok * p.pairs;
        const uint32_t g = (uint32_t)(token0 + tok), bi = p.batch > 1 ? g / (uint32_t)p.seq : 0, si = g - bi * (uint32_t)p.seq;
        cs[i] = cos_sin(p, p.pos[bi * p.pos_stride[0] + si * p.pos_stride[1]], __ldg(reinterpret_cast<const unsigned long long*>(p.turns) + k));
      }
      __syncthreads();
    }
#pragma unroll
    for (int q = 0; q < U; ++q) {
      if (which[q] < 0) continue;
      void* const out = which[q] ? p.a[1].out : p.a[0].out;
      if (where[q] >= 0) {
        float u[V], v[V];
        a[q].get(u);
        b[q].get(v);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const float2 w = cs[where[q] + e];
          if constexpr (!INTER || V == 1) {
            const float x = u[e], y = v[e];
            u[e] = x * w.x - y * w.y;
            v[e] = y * w.x + x * w.y;
          } else {
            float& x = 2 * e < V ? u[2 * e] : v[2 * e - V];
            float& y = 2 * e < V ? u[2 * e + 1] : v[2 * e + 1 - V];
            const float x0 = x, y0 = y;
            x = x0 * w.x - y0 * w.y;
            y = y0 * w.x + x0 * w.y;
          }
        }
        a[q].set(u);
        b[q].set(v);
      }
      a[q].store(out, out_at[q] + ea[q]);
      if (eb[q] >= 0) b[q].store(out, out_at[q] + eb[q]);
    }
  }
}

template <int DT, int V, int U>
cudaError_t run_rotary(const RotaryPlan& p, cudaStream_t s) {
  const int64_t tokens = p.batch * p.seq;
  const int64_t heads = p.a[0].heads + (p.arrays > 1 ? p.a[1].heads : 0);
  RotaryTile t;
  t.turned = p.pairs / V;
  t.copied = (p.dim - 2 * p.pairs) / V;
  bool in_place = true;
  for (int k = 0; k < p.arrays; ++k) in_place = in_place && p.a[k].in == p.a[k].out;
  if (in_place) t.copied = 0;
  t.per_head = t.turned + (t.copied + 1) / 2;
  if (t.per_head == 0) return cudaSuccess;  // nothing turns, and nothing has to be copied
  // whole heads, then whole tokens, up to 256 U items; never more cosines than 40 KB hold
  const int64_t most = 256 * U;
  t.heads = (int)std::max<int64_t>(1, std::min(heads, most / t.per_head));
  const int64_t cap = p.pairs ? std::max<int64_t>(1, 5120 / p.pairs) : most;
  t.tokens = t.heads < heads ? 1 : (int)std::max<int64_t>(1, std::min({tokens, most / (heads * t.per_head), cap}));
  const int64_t gx = (tokens + t.tokens - 1) / t.tokens, gy = (heads + t.heads - 1) / t.heads;
  if (gx > INT32_MAX || gy > 65535) return cudaErrorInvalidValue;
  const size_t smem = (size_t)t.tokens * p.pairs * sizeof(float2);
  const auto kernel = p.interleaved ? rotary_kernel<DT, V, U, true> : rotary_kernel<DT, V, U, false>;
  if (smem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
  }
  kernel<<<dim3((unsigned)gx, (unsigned)gy), 256, smem, s>>>(p, t, tokens, (int)heads);
  return cudaGetLastError();
}

// Any alignment and size: a thread per pair, then per element that is copied.
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
    const float2 w = cos_sin(p, p.pos[b * p.pos_stride[0] + t * p.pos_stride[1]], p.turns[k]);
    const float u = load_plain(a.in, p.dt, in + eu), v = load_plain(a.in, p.dt, in + ev);
    store_from_f32(a.out, p.dt, out + eu, u * w.x - v * w.y);
    store_from_f32(a.out, p.dt, out + ev, v * w.x + u * w.y);
  }
}

// Elements of the widest access that every pair, head and row allows.
int access_width(const RotaryPlan& p) {
  const int eb = dt_bytes(p.dt);
  int v = 16 / eb;
  for (; v > 1; v /= 2) {
    bool fits = p.pairs % v == 0 && (p.dim - 2 * p.pairs) % v == 0;
    for (int k = 0; k < p.arrays; ++k) {
      const RotaryArray& a = p.a[k];
      fits = fits && ((uintptr_t)a.in | (uintptr_t)a.out) % (v * eb) == 0;
      const int64_t size[3] = {p.batch, p.seq, a.heads};
      for (int d = 0; d < 3; ++d)
        if (size[d] > 1) fits = fits && (a.in_stride[d] | a.out_stride[d]) % v == 0;
    }
    if (fits) break;
  }
  return v;
}

template <int DT>
cudaError_t run_rotary_type(const RotaryPlan& p, cudaStream_t s) {
  const int64_t heads = p.a[0].heads + (p.arrays > 1 ? p.a[1].heads : 0);
  const int v = access_width(p);
  // several items a thread once one each fills the device
  const bool many = p.batch * p.seq * heads * (p.dim / 2) / v >= (int64_t)device_sm_count() * 4 * 1024;
#define HLO_CASE(VV) \
  if (v == VV) return many ? run_rotary<DT, VV, 4>(p, s) : run_rotary<DT, VV, 1>(p, s)
  if constexpr (DT != F32) HLO_CASE(8);
  HLO_CASE(4);
  HLO_CASE(2);
  HLO_CASE(1);
#undef HLO_CASE
  return cudaErrorInvalidValue;
}

cudaError_t launch_rotary(const RotaryPlan& p, cudaStream_t s) {
  const int64_t heads = std::max(p.a[0].heads, p.arrays > 1 ? p.a[1].heads : 0);
  if (p.batch <= INT32_MAX / p.seq && p.pairs <= 8192 && heads <= 65535 / 4) {
    if (p.dt == F32) return run_rotary_type<F32>(p, s);
    if (p.dt == BF16) return run_rotary_type<BF16>(p, s);
    return run_rotary_type<F16>(p, s);
  }
  for (int k = 0; k < p.arrays; ++k) {
    const int64_t total = p.batch * p.seq * p.a[k].heads * (p.dim - p.pairs);
    const int64_t blocks = (total + 255) / 256, cap = (int64_t)device_sm_count() * 64;
    rotary_any_kernel<<<(unsigned)std::min(blocks, cap), 256, 0, s>>>(p, p.a[k], total);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace hlo
