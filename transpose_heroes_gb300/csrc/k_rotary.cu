// Rotary positions (hlo_rotary): each pair of a head turns by 2 pi frac(position * turns / 2^64).
#include <algorithm>

#include "async_copy.cuh"
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
  __device__ __forceinline__ void load(const char* a) {
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
  __device__ __forceinline__ void store(char* a) const {
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

// How a block's 256 threads share its work: a thread has one item (two accesses of V elements) of a head, at
// one token, in every slots-th head of the block's share.
struct RotaryTile {
  int items;    // of a head: the turned ones, then the copied ones
  int turned;   // pairs / V
  int copied;   // copied elements / V
  int slots;    // threads (of one item and token) that share the heads
  int tokens;   // tokens a block
  int heads;    // heads a block (of x's and then y's)
};

// A block first computes the cosine and sine of each (token, pair) once, into shared memory. An item is the
// two halves of V pairs (half layout), V adjacent pairs (interleaved), or 2 V copied elements; a thread's
// item and token stay, so the places of its elements and its cosines are found once for U heads. The
// loads of the first U heads are issued before the cosines are computed. Bound: latency for a few tokens (32 tokens
// of 32 + 8 heads: 4 us a call, the launch); HBM and the phases of a block for many (see below).
template <int DT, int V, int U, bool INTER>
__global__ void __launch_bounds__(256, 3) rotary_kernel(const __grid_constant__ RotaryPlan p, const RotaryTile t, int total_tokens,
                                                     int total_heads) {
  extern __shared__ float2 cs[];
  follow();
  const int token0 = blockIdx.x * t.tokens;
  const int tokens = min(t.tokens, total_tokens - token0);
  const int head_end = min(total_heads, (int)(blockIdx.y + 1) * t.heads);
  const int group = threadIdx.x / t.items, k = threadIdx.x - group * t.items;
  const int tok = group / t.slots;
  const int head0 = blockIdx.y * t.heads + group - tok * t.slots;
  const bool busy = tok < tokens;
  const bool turn = k < t.turned;
  const int ea = turn ? (INTER ? 2 * k * V : k * V) : 2 * p.pairs + 2 * (k - t.turned) * V;
  const int eb = turn ? (INTER ? ea + V : ea + p.pairs) : (2 * (k - t.turned) + 1 < t.copied ? ea + V : -1);
  const int split = (int)p.a[0].heads;  // heads from here on are y's
  const char* in[2] = {nullptr, nullptr};
  char* out[2] = {nullptr, nullptr};
  constexpr int EB = DT == F32 ? 4 : 2;
  if (busy) {
    const uint32_t g = (uint32_t)(token0 + tok), bi = p.batch > 1 ? g / (uint32_t)p.seq : 0, si = g - bi * (uint32_t)p.seq;
#pragma unroll
    for (int a = 0; a < 2; ++a) {
      in[a] = reinterpret_cast<const char*>(p.a[a].in) + (bi * p.a[a].in_stride[0] + si * p.a[a].in_stride[1] + ea) * EB;
      out[a] = reinterpret_cast<char*>(p.a[a].out) + (bi * p.a[a].out_stride[0] + si * p.a[a].out_stride[1] + ea) * EB;
    }
  }
  const int64_t second = (int64_t)(eb - ea) * EB;
  float2 w[V];
  for (int base = head0;; base += U * t.slots) {
    Piece<DT, V> a[U], b[U];
#pragma unroll
    for (int q = 0; q < U; ++q) {
      const int head = base + q * t.slots;
      if (!busy || head >= head_end) continue;
      const char* const at = head < split ? in[0] + head * p.a[0].in_stride[2] * EB : in[1] + (head - split) * p.a[1].in_stride[2] * EB;
      a[q].load(at);
      if (eb >= 0) b[q].load(at + second);
    }
    if (base == head0) {
      for (int i = threadIdx.x; i < tokens * p.pairs; i += 256) {
        const int tk = i / p.pairs, pair = i - tk * p.pairs;
        const uint32_t g = (uint32_t)(token0 + tk), bi = p.batch > 1 ? g / (uint32_t)p.seq : 0, si = g - bi * (uint32_t)p.seq;
        cs[i] = cos_sin(p, p.pos[bi * p.pos_stride[0] + si * p.pos_stride[1]], load_kept(reinterpret_cast<const unsigned long long*>(p.turns) + pair));
      }
      __syncthreads();
      if (!busy) return;
      if (turn) {
#pragma unroll
        for (int e = 0; e < V; ++e) w[e] = cs[tok * p.pairs + k * V + e];
      }
    }
#pragma unroll
    for (int q = 0; q < U; ++q) {
      const int head = base + q * t.slots;
      if (head >= head_end) continue;
      if (turn) {
        float u[V], v[V];
        a[q].get(u);
        b[q].get(v);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          if constexpr (!INTER || V == 1) {
            const float x = u[e], y = v[e];
            u[e] = x * w[e].x - y * w[e].y;
            v[e] = y * w[e].x + x * w[e].y;
          } else {
            float& x = 2 * e < V ? u[2 * e] : v[2 * e - V];
            float& y = 2 * e < V ? u[2 * e + 1] : v[2 * e + 1 - V];
            const float x0 = x, y0 = y;
            x = x0 * w[e].x - y0 * w[e].y;
            y = y0 * w[e].x + x0 * w[e].y;
          }
        }
        a[q].set(u);
        b[q].set(v);
      }
      char* const at = head < split ? out[0] + head * p.a[0].out_stride[2] * EB : out[1] + (head - split) * p.a[1].out_stride[2] * EB;
      a[q].store(at);
      if (eb >= 0) b[q].store(at + second);
    }
    if (base + U * t.slots >= head_end) break;
  }
}

// Heads a thread turns at a time: 4 accesses of 2 x 16 bytes in flight once the device is full.
template <int DT, int V, int U>
cudaError_t run_rotary(const RotaryPlan& p, const RotaryTile& tile, cudaStream_t s) {
  RotaryTile t = tile;
  const int tokens = (int)(p.batch * p.seq);
  const int heads = (int)(p.a[0].heads + (p.arrays > 1 ? p.a[1].heads : 0));
  const int groups = 256 / t.items;
  // U heads a thread: then as many tokens a block as there are threads for, but not more than 40 KB of cosines
  t.slots = std::min(groups, (heads + U - 1) / U);
  const int cap = p.pairs ? std::max(1, 5120 / p.pairs) : groups;
  t.tokens = std::max(1, std::min({groups / t.slots, tokens, cap}));
  t.heads = std::min(heads, t.slots * U);
  const int gx = (tokens + t.tokens - 1) / t.tokens, gy = (heads + t.heads - 1) / t.heads;
  const size_t smem = (size_t)t.tokens * p.pairs * sizeof(float2);
  return launch_after(p.interleaved ? rotary_kernel<DT, V, U, true> : rotary_kernel<DT, V, U, false>, dim3(gx, gy), dim3(256), smem, s, 1, p, t,
                      tokens, heads);
}

// ---- many tokens whose heads lie together --------------------------------------------------------------------
// Persistent blocks; thread 0 keeps a ring of `stages` groups of t.tokens tokens (their heads of x, then of y)
// coming with one bulk copy a token and array, so the loads never wait for the cosines. A group's cosines go
// to one of two tables in shared memory before its one barrier, behind which every thread has left the group
// before, whose stage is refilled then. Threads share the heads as in rotary_kernel.
// Bound: HBM. 2 x 16384 tokens of 32 + 8 heads of 128 bf16 (671 MB): 106 us, 6.3 TB/s, 93% of the copy rate;
// rotary_kernel takes 117 us, as its blocks' loads, cosines and stores follow one another.
constexpr int kMaxStages = 4;

template <int DT, bool INTER>
__global__ void __launch_bounds__(256, 2) rotary_stream_kernel(const __grid_constant__ RotaryPlan p, const RotaryTile t, int total_tokens,
                                                               int total_heads, int stages) {
  constexpr int V = kVec<DT>, EB = 16 / V;
  extern __shared__ __align__(128) char ring[];
  __shared__ __align__(8) uint64_t full[kMaxStages];
  follow();
  const int split = (int)p.a[0].heads, tid = threadIdx.x;
  const int x_bytes = split * p.dim * EB, token_bytes = total_heads * p.dim * EB, stage_bytes = t.tokens * token_bytes;
  float2* const tables = reinterpret_cast<float2*>(ring + (size_t)stages * stage_bytes);
  const int groups = (total_tokens + t.tokens - 1) / t.tokens;
  const int mine = (groups - (int)blockIdx.x + (int)gridDim.x - 1) / (int)gridDim.x;  // groups of this block
  const auto place = [&](int token, int a, bool out) {  // bytes from the array's start
    const uint32_t bi = p.batch > 1 ? (uint32_t)token / (uint32_t)p.seq : 0, si = (uint32_t)token - bi * (uint32_t)p.seq;
    const int64_t* const s = out ? p.a[a].out_stride : p.a[a].in_stride;
    return (bi * s[0] + si * s[1]) * EB;
  };
  const auto request = [&](int i) {
    const int s = i % stages, first = ((int)blockIdx.x + i * (int)gridDim.x) * t.tokens, n = min(t.tokens, total_tokens - first);
    const uint32_t bar = smem_addr(&full[s]);
    mbar_arrive_expect_tx(bar, n * token_bytes);
    for (int k = 0; k < n; ++k) {
      char* const to = ring + (size_t)s * stage_bytes + k * token_bytes;
      bulk_load(to, reinterpret_cast<const char*>(p.a[0].in) + place(first + k, 0, false), x_bytes, bar);
      if (p.arrays > 1) bulk_load(to + x_bytes, reinterpret_cast<const char*>(p.a[1].in) + place(first + k, 1, false), token_bytes - x_bytes, bar);
    }
  };
  if (tid == 0) {
    for (int s = 0; s < stages; ++s) mbar_init(smem_addr(&full[s]), 1);
    fence_mbar_init();
  }
  __syncthreads();
  if (tid == 0)
    for (int i = 0; i < min(stages, mine); ++i) request(i);
  const int part = tid / t.items, k = tid - part * t.items;
  const int tok = part / t.slots, slot = part - tok * t.slots;
  const bool turn = k < t.turned;
  const int ea = (turn ? (INTER ? 2 * k * V : k * V) : 2 * p.pairs + 2 * (k - t.turned) * V) * EB;
  const int eb = turn ? (INTER ? ea + 16 : ea + p.pairs * EB) : (2 * (k - t.turned) + 1 < t.copied ? ea + 16 : -1);
  for (int i = 0; i < mine; ++i) {
    const int s = i % stages, first = ((int)blockIdx.x + i * (int)gridDim.x) * t.tokens, n = min(t.tokens, total_tokens - first);
    float2* const cs = tables + (i & 1) * t.tokens * p.pairs;
    for (int j = tid; j < n * p.pairs; j += 256) {
      const int tk = j / p.pairs, pair = j - tk * p.pairs;
      const uint32_t g = (uint32_t)(first + tk), bi = p.batch > 1 ? g / (uint32_t)p.seq : 0, si = g - bi * (uint32_t)p.seq;
      cs[j] = cos_sin(p, p.pos[bi * p.pos_stride[0] + si * p.pos_stride[1]], load_kept(reinterpret_cast<const unsigned long long*>(p.turns) + pair));
    }
    const bool arrived = mbar_wait(smem_addr(&full[s]), (i / stages) & 1);
    if (!__syncthreads_and(arrived)) {  // a copy did not come: give up, when the others have come or their waits run out
      if (tid == 0) {
        record_fault(kFaultCopyTimeout);
        for (int j = i; j < min(i + stages - (i > 0 ? 1 : 0), mine); ++j) mbar_wait(smem_addr(&full[j % stages]), (j / stages) & 1);
      }
      __syncthreads();
      return;
    }
    if (tid == 0 && i > 0 && i - 1 + stages < mine) request(i - 1 + stages);
    if (tok >= n) continue;
    float2 w[V];
    if (turn) {
#pragma unroll
      for (int e = 0; e < V; ++e) w[e] = cs[tok * p.pairs + k * V + e];
    }
    const char* const from = ring + (size_t)s * stage_bytes + tok * token_bytes;
    char* const x_out = reinterpret_cast<char*>(p.a[0].out) + place(first + tok, 0, true);
    char* const y_out = reinterpret_cast<char*>(p.a[1].out) + place(first + tok, 1, true);
#pragma unroll 2
    for (int head = slot; head < total_heads; head += t.slots) {
      const char* const at = from + head * p.dim * EB;
      char* const to = head < split ? x_out + head * p.a[0].out_stride[2] * EB : y_out + (head - split) * p.a[1].out_stride[2] * EB;
      uint4 a = *reinterpret_cast<const uint4*>(at + ea), b = eb >= 0 ? *reinterpret_cast<const uint4*>(at + eb) : a;
      if (turn) {
        float u[V], v[V];
        unpack<DT>(a, u);
        unpack<DT>(b, v);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          float& x = !INTER ? u[e] : 2 * e < V ? u[2 * e] : v[2 * e - V];
          float& y = !INTER ? v[e] : 2 * e < V ? u[2 * e + 1] : v[2 * e + 1 - V];
          const float x0 = x, y0 = y;
          x = x0 * w[e].x - y0 * w[e].y;
          y = y0 * w[e].x + x0 * w[e].y;
        }
        a = pack<DT>(u);
        b = pack<DT>(v);
      }
      *reinterpret_cast<uint4*>(to + ea) = a;
      if (eb >= 0) *reinterpret_cast<uint4*>(to + eb) = b;
    }
  }
}

// The ring's shape, if these arrays can use it: heads that lie together, and enough tokens for several groups a
// block. false otherwise.
template <int DT>
bool run_rotary_stream(const RotaryPlan& p, const RotaryTile& tile, cudaStream_t s, cudaError_t* result) {
  constexpr int EB = 16 / kVec<DT>;
  int64_t heads = 0;
  for (int k = 0; k < p.arrays; ++k) {
    if (p.a[k].heads > 1 && p.a[k].in_stride[2] != p.dim) return false;
    heads += p.a[k].heads;
  }
  RotaryTile t = tile;
  const int parts = 256 / t.items;
  const int64_t tokens = p.batch * p.seq, token_bytes = heads * p.dim * EB;
  t.slots = 1;
  while (t.slots * 2 <= parts && heads > 8 * t.slots) t.slots *= 2;  // up to eight heads a thread
  t.tokens = (int)std::min<int64_t>(parts / t.slots, std::max<int64_t>(1, 40 * 1024 / token_bytes));
  if (t.tokens * token_bytes > 100 * 1024 || t.tokens * (int64_t)p.pairs > 4096) return false;
  const size_t stage = t.tokens * token_bytes, tables = (size_t)2 * t.tokens * p.pairs * sizeof(float2);
  // two blocks an SM
  const int stages = (int)std::min<size_t>(kMaxStages, (108 * 1024 - tables) / stage);
  const int64_t groups = (tokens + t.tokens - 1) / t.tokens, blocks = (int64_t)device_sm_count() * 2;
  if (stages < 2 || groups < 4 * blocks) return false;
  const size_t smem = stages * stage + tables;
  const auto kernel = p.interleaved ? rotary_stream_kernel<DT, true> : rotary_stream_kernel<DT, false>;
  *result = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 108 * 1024);
  if (*result != cudaSuccess) return true;
  *result = launch_after(kernel, dim3((unsigned)blocks), dim3(256), smem, s, 1, p, t, (int)tokens, (int)heads, stages);
  return true;
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
cudaError_t run_rotary_type(const RotaryPlan& p, int v, const RotaryTile& t, cudaStream_t s) {
  const int64_t heads = p.a[0].heads + (p.arrays > 1 ? p.a[1].heads : 0);
  cudaError_t result = cudaSuccess;
  if (v == kVec<DT> && run_rotary_stream<DT>(p, t, s, &result)) return result;
  // several heads a thread once one each fills the device twice over
  const bool many = p.batch * p.seq * heads * t.items >= (int64_t)device_sm_count() * 8 * 1024;
#define HLO_CASE(VV) \
  if (v == VV) return many ? run_rotary<DT, VV, 4>(p, t, s) : run_rotary<DT, VV, 1>(p, t, s)
  if constexpr (DT != F32) HLO_CASE(8);
  HLO_CASE(4);
  HLO_CASE(2);
  HLO_CASE(1);
#undef HLO_CASE
  return cudaErrorInvalidValue;
}

cudaError_t launch_rotary(const RotaryPlan& p, cudaStream_t s) {
  const int v = access_width(p);
  RotaryTile t = {};
  t.turned = p.pairs / v;
  t.copied = (p.dim - 2 * p.pairs) / v;
  bool in_place = true;
  for (int k = 0; k < p.arrays; ++k) in_place = in_place && p.a[k].in == p.a[k].out;
  if (in_place) t.copied = 0;
  t.items = t.turned + (t.copied + 1) / 2;
  if (t.items == 0) return cudaSuccess;  // nothing turns, and nothing has to be copied
  const int64_t heads = std::max(p.a[0].heads, p.arrays > 1 ? p.a[1].heads : 0);
  // tokens are counted in 32 bits, rounded up to whole blocks of at most 256
  if (t.items <= 256 && p.pairs <= 4096 && p.batch <= (INT32_MAX - 256) / p.seq && heads <= 32767) {
    if (p.dt == F32) return run_rotary_type<F32>(p, v, t, s);
    if (p.dt == BF16) return run_rotary_type<BF16>(p, v, t, s);
    return run_rotary_type<F16>(p, v, t, s);
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
