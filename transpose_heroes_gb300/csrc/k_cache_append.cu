// Appending to a paged cache (hlo_cache_append): the new tokens' keys turn by their positions and go to their pages, the
// values go there as they are, and the queries turn on the way.
#include <algorithm>

#include "cache_plans.h"
#include "vectors.cuh"

namespace hlo {

// As in the rotation alone: position * turns mod 2^64, the high half as a signed number of 2^-31 half turns.
__device__ __forceinline__ float2 append_cos_sin(int32_t pos, uint64_t turns, float scale) {
  const uint64_t t = (uint64_t)(int64_t)pos * turns;
  float s, c;
  sincospif((float)(int32_t)(t >> 32) * 0x1p-31f, &s, &c);
  return make_float2(c * scale, s * scale);
}

// V elements as they are loaded: a 16-byte vector, or one.
template <int DT, int V>
struct AppendPiece {
  uint4 w;
  __device__ __forceinline__ void load(const char* a) { w = load16(a); }
  __device__ __forceinline__ void get(float (&v)[V]) const { unpack<DT>(w, v); }
};
template <int DT>
struct AppendPiece<DT, 1> {
  float w;
  __device__ __forceinline__ void load(const char* a) { w = load_plain(a, DT, 0); }
  __device__ __forceinline__ void get(float (&v)[1]) const { v[0] = w; }
};
template <int DT, int V, bool F8>
__device__ __forceinline__ void append_store(char* a, const float (&v)[V], float scale, float inv) {
  if constexpr (F8 && V == 8) {
    *reinterpret_cast<uint2*>(a) = make_uint2(codes(make_float4(v[0], v[1], v[2], v[3]), scale, inv, 1),
                                              codes(make_float4(v[4], v[5], v[6], v[7]), scale, inv, 1));
  } else if constexpr (F8 && V == 4) {
    *reinterpret_cast<uint32_t*>(a) = codes(make_float4(v[0], v[1], v[2], v[3]), scale, inv, 1);
  } else if constexpr (F8) {
    *reinterpret_cast<uint8_t*>(a) = f8_code(v[0], scale);
  } else if constexpr (V > 1) {
    *reinterpret_cast<uint4*>(a) = pack<DT>(v);
  } else {
    store_from_f32(a, DT, 0, v[0]);
  }
}

// How a block's 256 threads share its work: a thread has one item (two accesses of V elements) of a head, at one
// token, in every slots-th head of the block's share. Heads are numbered q's, k's, v's.
struct AppendTile {
  int items, turned, copied;  // of a head; accesses: 2 turned + copied
  int slots, tokens, heads;
};

struct AppendToken {
  int64_t at[2];  // byte offset of the token's place in k and v; at[0] < 0: dropped
  int b, t;       // b < 0: behind the sequence's tokens
};

// A block finds its tokens' places and cosines once, while its first loads are on their way. Bound: launch and a chain of
// dependent loads (count and length, page, entry) for a few tokens (32 tokens of 32 + 2 x 8 heads of 128: 3.0 us in a captured
// graph); for many the blocks' phases, which follow one another (2 x 8192 tokens, 403 MB: 72 us, 82% of the copy
// rate). Six heads a thread and two blocks an SM are the best of what was tried: four heads and three blocks, with a quarter of
// the threads idle at 48 heads and some registers spilled, 94 us; three heads 78 us; three heads and four blocks 104 us.
template <int DT, int V, int U, bool INTER, bool F8>
__global__ void __launch_bounds__(256, U > 1 ? 2 : 3) append_kernel(const __grid_constant__ AppendPlan p, const AppendTile t, int total_tokens,
                                                        int total_heads) {
  extern __shared__ __align__(16) char mem[];
  AppendToken* const info = reinterpret_cast<AppendToken*>(mem);
  float2* const cs = reinterpret_cast<float2*>(info + t.tokens);
  constexpr int EB = DT == F32 ? 4 : 2, CB = F8 ? 1 : EB;
  const bool inter = V > 1 ? INTER : p.interleaved;
  follow();
  const int token0 = blockIdx.x * t.tokens;
  const int tokens = min(t.tokens, total_tokens - token0);
  const int head_end = min(total_heads, (int)(blockIdx.y + 1) * t.heads);
  const int group = threadIdx.x / t.items, k = threadIdx.x - group * t.items;
  const int tok = group / t.slots;
  const int head0 = blockIdx.y * t.heads + group - tok * t.slots;
  const bool busy = tok < tokens;
  const bool turn = k < t.turned;
  // of a head that turns, and of one that does not
  const int ea = turn ? (inter ? 2 * k * V : k * V) : 2 * p.pairs + 2 * (k - t.turned) * V;
  const int eb = turn ? (inter ? ea + V : ea + p.pairs) : (2 * (k - t.turned) + 1 < t.copied ? ea + V : -1);
  const int va = 2 * k * V, vb = va + V < p.dim ? va + V : -1;
  const int hk = p.heads, hv = p.heads + p.kv;  // where k's and v's heads begin
  const char* in[3] = {nullptr, nullptr, nullptr};
  if (busy) {
    const uint32_t g = (uint32_t)(token0 + tok), bi = g / (uint32_t)p.m.seq, si = g - bi * (uint32_t)p.m.seq;
#pragma unroll
    for (int a = 0; a < 3; ++a)
      if (p.in[a]) in[a] = reinterpret_cast<const char*>(p.in[a]) + ((int64_t)bi * p.in_stride[a][0] + (int64_t)si * p.in_stride[a][1]) * EB;
  }
  const auto from = [&](int head) {
    return head < hk ? in[0] + head * p.in_stride[0][2] * EB
                     : head < hv ? in[1] + (head - hk) * p.in_stride[1][2] * EB : in[2] + (head - hv) * p.in_stride[2][2] * EB;
  };
  float2 w[V];
  for (int base = head0;; base += U * t.slots) {
    AppendPiece<DT, V> ra[U], rb[U];
#pragma unroll
    for (int q = 0; q < U; ++q) {
      const int head = base + q * t.slots;
      if (!busy || head >= head_end) continue;
      const char* const at = from(head);
      const int first = head < hv ? ea : va, second = head < hv ? eb : vb;
      ra[q].load(at + first * EB);
      if (second >= 0) rb[q].load(at + second * EB);
    }
    if (base == head0) {
      for (int i = threadIdx.x; i < tokens; i += 256) {
        const uint32_t g = (uint32_t)(token0 + i), bi = g / (uint32_t)p.m.seq, si = g - bi * (uint32_t)p.m.seq;
        const int length = cache_length(p.m, bi);
        AppendToken n = {{-1, -1}, (int)si < cache_count(p.m, bi) ? (int)bi : -1, (int)si};
        if (n.b >= 0 && (int64_t)length + si < p.m.capacity) {
          int page, place;
          cache_place(p.m, p.m.table + bi * p.m.table_stride, length + (int)si, &page, &place);
          if (page >= 0) {
            n.at[0] = (page * p.cache_stride[0][0] + place * p.cache_stride[0][1]) * CB;
            n.at[1] = (page * p.cache_stride[1][0] + place * p.cache_stride[1][1]) * CB;
          }
        }
        info[i] = n;
      }
      for (int i = threadIdx.x; i < tokens * p.pairs; i += 256) {
        const int tk = i / p.pairs, pair = i - tk * p.pairs;
        const uint32_t g = (uint32_t)(token0 + tk), bi = g / (uint32_t)p.m.seq, si = g - bi * (uint32_t)p.m.seq;
        const int32_t pos = p.pos ? p.pos[bi * p.pos_stride[0] + si * p.pos_stride[1]] : cache_length(p.m, bi) + (int)si;
        cs[i] = append_cos_sin(pos, load_kept(reinterpret_cast<const unsigned long long*>(p.turns) + pair), p.scale);
      }
      __syncthreads();
      if (!busy || info[tok].b < 0) return;
      if (turn) {
#pragma unroll
        for (int e = 0; e < V; ++e) w[e] = cs[tok * p.pairs + k * V + e];
      }
    }
#pragma unroll
    for (int q = 0; q < U; ++q) {
      const int head = base + q * t.slots;
      if (head >= head_end) continue;
      const int first = head < hv ? ea : va, second = head < hv ? eb : vb;
      float a[V], b[V];
      ra[q].get(a);
      rb[q].get(b);
      if (turn && head < hv) {
#pragma unroll
        for (int e = 0; e < V; ++e) {
          if constexpr (!INTER || V == 1) {
            const float x = a[e], y = b[e];
            a[e] = x * w[e].x - y * w[e].y;
            b[e] = y * w[e].x + x * w[e].y;
          } else {
            float& x = 2 * e < V ? a[2 * e] : b[2 * e - V];
            float& y = 2 * e < V ? a[2 * e + 1] : b[2 * e + 1 - V];
            const float x0 = x, y0 = y;
            x = x0 * w[e].x - y0 * w[e].y;
            y = y0 * w[e].x + x0 * w[e].y;
          }
        }
      }
      if (head < hk) {
        char* const to = reinterpret_cast<char*>(p.q_out) +
                         (info[tok].b * p.q_stride[0] + info[tok].t * p.q_stride[1] + head * p.q_stride[2]) * EB;
        append_store<DT, V, false>(to + first * EB, a, 1.0f, 1.0f);
        if (second >= 0) append_store<DT, V, false>(to + second * EB, b, 1.0f, 1.0f);
      } else if (info[tok].at[0] >= 0) {
        const int side = head < hv ? 0 : 1;
        char* const to = reinterpret_cast<char*>(p.cache[side]) + info[tok].at[side] +
                         (side ? head - hv : head - hk) * p.cache_stride[side][2] * CB;
        append_store<DT, V, F8>(to + first * CB, a, p.code_scale[side], p.code_inv[side]);
        if (second >= 0) append_store<DT, V, F8>(to + second * CB, b, p.code_scale[side], p.code_inv[side]);
      }
    }
    if (base + U * t.slots >= head_end) break;
  }
}

template <int DT, int V, int U, bool INTER, bool F8>
cudaError_t run_append(const AppendPlan& p, cudaStream_t s) {
  AppendTile t = {};
  t.turned = p.pairs / V;
  t.copied = (p.dim - 2 * p.pairs) / V;
  t.items = t.turned + (t.copied + 1) / 2;
  const int tokens = p.m.batch * p.m.seq, heads = p.heads + 2 * p.kv;
  const int groups = 256 / t.items;
  // U heads a thread: then as many tokens a block as there are threads for, but not more than 40 KB of cosines
  t.slots = std::min(groups, (heads + U - 1) / U);
  const int cap = p.pairs ? std::max(1, 5120 / p.pairs) : groups;
  t.heads = std::min(heads, t.slots * U);
  if (U > 1) {  // a power of two leaves no thread without a token where items are one too; a block has all heads then
    while (t.slots & (t.slots - 1)) t.slots &= t.slots - 1;
    t.heads = heads;
  }
  t.tokens = std::max(1, std::min({groups / t.slots, tokens, cap}));
  const int gx = (tokens + t.tokens - 1) / t.tokens, gy = (heads + t.heads - 1) / t.heads;
  const size_t smem = t.tokens * (sizeof(AppendToken) + (size_t)p.pairs * sizeof(float2));
  return launch_after(append_kernel<DT, V, U, INTER, F8>, dim3(gx, gy), dim3(256), smem, s, 1, p, t, tokens, heads);
}

template <int DT, bool F8>
cudaError_t run_append_type(const AppendPlan& p, cudaStream_t s) {
  constexpr int V = kVec<DT>, EB = 16 / V, CB = F8 ? 1 : EB;
  // whole vectors, where every pair, head, place and row allows them
  bool fits = p.pairs % V == 0 && p.dim % V == 0;
  for (int a = 0; a < 3; ++a) {
    if (!p.in[a]) continue;
    fits = fits && (uintptr_t)p.in[a] % 16 == 0;
    for (int d = 0; d < 3; ++d) fits = fits && p.in_stride[a][d] % V == 0;
  }
  for (int d = 0; d < 3 && p.in[0]; ++d) fits = fits && p.q_stride[d] % V == 0;
  fits = fits && (uintptr_t)p.q_out % 16 == 0;
  for (int a = 0; a < 2; ++a) {
    fits = fits && (uintptr_t)p.cache[a] % (V * CB) == 0;
    for (int d = 0; d < 3; ++d) fits = fits && p.cache_stride[a][d] % V == 0;
  }
  if (!fits) return run_append<DT, 1, 1, false, F8>(p, s);
  // several heads a thread once one each fills the device twice over
  const bool many = (int64_t)p.m.batch * p.m.seq * (p.heads + 2 * p.kv) * (p.dim / V / 2) >= (int64_t)device_sm_count() * 8 * 1024;
  if (p.interleaved) return many ? run_append<DT, V, 6, true, F8>(p, s) : run_append<DT, V, 1, true, F8>(p, s);
  return many ? run_append<DT, V, 6, false, F8>(p, s) : run_append<DT, V, 1, false, F8>(p, s);
}

cudaError_t launch_append(const AppendPlan& p, cudaStream_t s) {
  if (p.dt == F32) return p.f8 ? run_append_type<F32, true>(p, s) : run_append_type<F32, false>(p, s);
  if (p.dt == BF16) return p.f8 ? run_append_type<BF16, true>(p, s) : run_append_type<BF16, false>(p, s);
  return p.f8 ? run_append_type<F16, true>(p, s) : run_append_type<F16, false>(p, s);
}

}  // namespace hlo
