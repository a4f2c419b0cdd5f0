// Processing of logits (hlo_logits_process): bias, penalties for tokens of the history, mask, greedy token.
//
//  logits_kernel     -- rows in vectors of 16 bytes, each row shared by a cluster of up to 8 blocks.
//  logits_any_kernel -- any alignment: a block per row, a thread per token.
#include <cooperative_groups.h>

#include <algorithm>

#include "vectors.cuh"

namespace cg = cooperative_groups;

namespace hlo {

constexpr int kThreads = 512;
constexpr int kSlab = 8192;  // tokens whose occurrences logits_any_kernel counts at once, in shared memory

// A key whose order is "greater value first, lower token on ties"; 0 for NaN and -inf, which are never
// chosen. Adding +0 makes -0 equal to +0.
__device__ __forceinline__ unsigned long long choice_key(float l, int token) {
  l = __fadd_rn(l, 0.0f);
  if (!(l > __int_as_float(0xFF800000))) return 0;
  const uint32_t b = __float_as_uint(l);
  const uint32_t ordered = (b & 0x80000000u) ? ~b : b | 0x80000000u;
  return ((unsigned long long)ordered << 32) | (uint32_t)~token;
}

// The processed value; `seen`: whether the token occurs, c: how often after the prompt.
__device__ __forceinline__ float penalised(float l, float c, float rep, float freq, float pres) {
  l = l > 0.0f ? __fdiv_rn(l, rep) : __fmul_rn(l, rep);
  l = __fsub_rn(l, __fmul_rn(freq, c));
  return c > 0.0f ? __fsub_rn(l, pres) : l;
}

__global__ void __launch_bounds__(kThreads) logits_any_kernel(LogitsPlan p) {
  __shared__ uint32_t seen[kSlab];  // top bit: occurs at all; the rest: occurrences after the prompt
  __shared__ unsigned long long best_of[kThreads / 32];
  const int64_t b = blockIdx.x;
  int32_t len = 0, prompt = 0;
  if (p.history) {
    len = (int32_t)p.max_length;
    if (p.lengths) len = max(0, min(len, p.lengths[b]));
    if (p.prompts) prompt = p.prompts[b];
  }
  const float rep = p.repetition ? p.repetition[b] : 1.0f;
  const float freq = p.frequency ? p.frequency[b] : 0.0f, pres = p.presence ? p.presence[b] : 0.0f;
  unsigned long long best = 0;
  for (int64_t v0 = 0; v0 < p.vocab; v0 += kSlab) {
    if (len > 0) {
      __syncthreads();
      for (int i = threadIdx.x; i < kSlab; i += kThreads) seen[i] = 0;
      __syncthreads();
      const int32_t* h = p.history + b * p.history_stride;
      for (int32_t i = threadIdx.x; i < len; i += kThreads) {
        const int64_t t = (int64_t)h[i] - v0;
        if (t < 0 || t >= kSlab) continue;
        if (i >= prompt) atomicAdd(&seen[t], 1u);
        atomicOr(&seen[t], 0x80000000u);
      }
      __syncthreads();
    }
    const int64_t end = v0 + kSlab < p.vocab ? v0 + kSlab : p.vocab;
    for (int64_t v = v0 + threadIdx.x; v < end; v += kThreads) {
      float l = load_plain(p.x, p.dt, b * p.x_stride + v);
      if (p.bias) l = __fadd_rn(l, p.bias[b * p.bias_stride + v]);
      const uint32_t s = len > 0 ? seen[v - v0] : 0;
      if (s) {
        l = penalised(l, (float)(s & 0x7FFFFFFFu), rep, freq, pres);
      }
      if (p.mask && !((p.mask[b * p.mask_stride + (v >> 5)] >> (v & 31)) & 1u)) l = __int_as_float(0xFF800000);
      if (p.out) store_from_f32(p.out, p.out_dt, b * p.out_stride + v, l);
      const unsigned long long k = choice_key(l, (int)v);
      best = k > best ? k : best;
    }
  }
  if (!p.token) return;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    const unsigned long long o = __shfl_xor_sync(0xffffffffu, best, off);
    best = o > best ? o : best;
  }
  if ((threadIdx.x & 31) == 0) best_of[threadIdx.x >> 5] = best;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < kThreads / 32; ++w) best = best_of[w] > best ? best_of[w] : best;
    p.token[b] = best ? (int32_t)~(uint32_t)best : -1;
  }
}

// The greatest value of the warp's lanes; NaN only if all are.
__device__ __forceinline__ float warp_max_of(float v) {
  float r;
  asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}

// Dynamic shared memory for slabs of `slab` tokens: their counts (`places` words of `width` bytes: one for each token
// of the slab, or the places of a table); a bit for each that occurs; and the list of those, with their values.
struct LogitsShared {
  size_t bits, value, list, bytes;
  __host__ __device__ LogitsShared(int slab, int places, int width, int count_bytes, int64_t max_length) {
    const size_t listed = (size_t)(slab < max_length ? slab : max_length);
    bits = (size_t)places * width;
    value = bits + slab / 8;
    list = value + listed * 4;
    bytes = list + listed * count_bytes;
  }
};

// The dynamic shared memory that a block can have beside the kernel's own few hundred bytes (227 KB in all).
constexpr size_t kMostShared = 226 * 1024;

// A place of the table: 1 + the token's number in the slab, above a count. So slabs have at most 2^17 tokens, and
// histories fewer than 2^14 entries.
constexpr int kCountBits = 14;
constexpr int kTableSlab = 1 << 17;

// A cluster of blocks shares a row; its blocks take slabs of `batches` times blockDim.x U vectors in turn.
// The penalties touch a few of a slab's tokens (those of the history), but nearly every warp would meet one
// and all its lanes would run their division. So a slab has three parts:
//  1. mark the tokens that occur in the history and count their occurrences after the prompt, in shared memory
//     (COUNT is uint16_t for histories below 2^16, else uint32_t; adding and or-ing whole numbers gives one
//     result in any order). Whoever finds a token first puts it on a list. TABLE: counts are kept for the
//     tokens that occur alone, in a table with open addressing, so that a slab can be a whole row; else
//     for every token of the slab.
//  2. a thread for each listed token works out its value, from the logit itself.
//  3. stream the slab, with the listed tokens masked out; then store their values over it.
// ALONE: an SM has one block, which has its registers for itself and nobody to hide its waits: parts 1 and 2 take
// four tokens a thread at a time.
// Bound: for a batch, the scattered accesses of the listed tokens (a wavefront each) and the waits of parts 1
// and 2, not HBM: 256 rows of 131072 bf16 with histories of up to 4096 entries, bias and mask (141 MB) 60 us, or 56
// where most of it is in the second-level cache; without a history 34 us, without bias as well 25.5, 5.4 TB/s, without the
// mask 24.
// One row of 32000 with 700 entries 5.3 us.
// The slab's first logits are requested before all this. The blocks' best tokens are written to the first
// block's shared memory, and only that block waits for them.
template <int DT, int U, typename COUNT, bool TABLE, bool ALONE>
__global__ void __launch_bounds__(kThreads, ALONE ? 1 : 2)
    logits_kernel(const __grid_constant__ LogitsPlan p, int cluster, int batches, int table) {
  constexpr int W = kVec<DT>, EB = 16 / W;
  constexpr int CB = sizeof(COUNT), CPW = 4 / CB;  // counts a 32-bit word
  constexpr int Q = ALONE ? 4 : 1;
  extern __shared__ __align__(16) char shared[];
  __shared__ unsigned long long best_of[kThreads / 32], cluster_best[8];
  __shared__ int listed;
  follow();
  const bool meet = cluster > 1 && p.token;
  // the first of the cluster's two barriers: every block has started before one writes to another
  if (meet) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  const int64_t b = blockIdx.x / cluster;
  const int rank = (int)(blockIdx.x - b * cluster), tid = threadIdx.x, threads = blockDim.x;
  const int vocab = (int)p.vocab, words = (vocab + 31) / 32;
  const int batch = threads * U * W, slab = batches * batch;
  const LogitsShared parts(slab, TABLE ? table : slab, TABLE ? 4 : CB, CB, p.max_length);
  uint32_t* const seen = reinterpret_cast<uint32_t*>(shared);
  uint32_t* const bits = reinterpret_cast<uint32_t*>(shared + parts.bits);
  float* const value = reinterpret_cast<float*>(shared + parts.value);
  COUNT* const list = reinterpret_cast<COUNT*>(shared + parts.list);
  const char* const x_row = reinterpret_cast<const char*>(p.x) + b * p.x_stride * EB;
  const int64_t out_off = b * p.out_stride;
  const int shift = (int)(((uintptr_t)x_row / EB) & (W - 1));
  const uint32_t* const mask = p.mask ? p.mask + b * p.mask_stride : nullptr;
  const float* const bias = p.bias ? p.bias + b * p.bias_stride : nullptr;
  const bool whole_rows = shift == 0 && (uintptr_t)bias % 16 == 0;
  int len = 0, prompt = 0;
  if (p.history) {
    len = (int)p.max_length;
    if (p.lengths) len = max(0, min(len, p.lengths[b]));
    if (p.prompts) prompt = p.prompts[b];
    for (int i = tid; i < (int)(parts.value / 16); i += threads) reinterpret_cast<uint4*>(shared)[i] = make_uint4(0, 0, 0, 0);
    if (tid == 0) listed = 0;
  }
  float best_v = __int_as_float(0xFF800000);
  int best_i = -1;
  float warp_best = best_v;
  unsigned long long best = 0;
  for (int64_t start = (int64_t)rank * slab - shift; start < vocab; start += (int64_t)cluster * slab) {
    const int s0 = (int)start;
    uint4 x[U];
    uint32_t allowed[U];
    const auto request = [&](int at) {
      const int c0 = at + tid * W;
      if (whole_rows && at + batch <= vocab) {
#pragma unroll
        for (int u = 0; u < U; ++u) x[u] = load16(x_row + (int64_t)(c0 + u * threads * W) * EB);
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int c = c0 + u * threads * W;  // a multiple of W: its bits lie in one byte
          allowed[u] = mask ? (uint32_t)load_kept(reinterpret_cast<const uint8_t*>(mask) + (c >> 3)) >> (c & 7) : 0xFFFFFFFFu;
        }
        return;
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int c = c0 + u * threads * W;
        x[u] = make_uint4(0, 0, 0, 0);
        allowed[u] = 0xFFFFFFFFu;
        if (c >= vocab) continue;
        x[u] = load_cut<DT>(p.x, b * p.x_stride, c, vocab, p.x_end);
        if (mask) {
          const int w0 = c >> 5;  // -1 for the columns before the row
          const uint32_t lo = w0 >= 0 ? load_kept(mask + w0) : 0;
          const uint32_t hi = (c & 31) + W > 32 && w0 + 1 < words ? load_kept(mask + w0 + 1) : 0;
          allowed[u] = __funnelshift_r(lo, hi, c & 31);
        }
      }
    };
    request(s0);
    int n = 0;
    if (len > 0) {
      __syncthreads();  // counts and bits are 0, the list is empty
      const int32_t* const h = p.history + b * p.history_stride;
      const uint32_t limit = (uint32_t)min(slab, vocab - s0);
      const int lane = tid & 31;
      const auto count = [&](int token, int i) {  // one entry a lane; -1 where the history has ended
        const uint32_t at = (uint32_t)token - (uint32_t)s0;
        bool first = false;
        uint32_t place = at;
        if (at < limit && token >= 0) {  // not another slab's token, nor one outside the vocabulary
          const uint32_t m = 1u << (at & 31);
          const uint32_t made = i >= prompt;
          if (TABLE) {
            atomicOr(&bits[at >> 5], m);
            // the table has more places than the history has entries, so one is free
            place = __umulhi(at * 2654435761u, (uint32_t)table);
            uint32_t found;
            while ((found = atomicCAS(&seen[place], 0u, (at + 1) << kCountBits | made)) != 0 && found >> kCountBits != at + 1)
              place = place + 1 == (uint32_t)table ? 0 : place + 1;
            first = found == 0;
            if (!first && made) atomicAdd(&seen[place], 1u);
          } else {
            first = !(atomicOr(&bits[at >> 5], m) & m);
            if (made) atomicAdd(&seen[at / CPW], 1u << (8 * CB * (int)(at % CPW)));
          }
        }
        const uint32_t firsts = __ballot_sync(0xffffffffu, first);
        if (firsts) {  // one place on the list for all of the warp's
          int index = 0;
          if (lane == 0) index = atomicAdd(&listed, __popc(firsts));
          index = __shfl_sync(0xffffffffu, index, 0) + __popc(firsts & ((1u << lane) - 1));
          if (first) list[index] = (COUNT)place;
        }
      };
      for (int base = tid - lane; base < len; base += Q * threads) {
        int tokens[Q];
#pragma unroll
        for (int q = 0; q < Q; ++q) tokens[q] = base + q * threads + lane < len ? load_kept(h + base + q * threads + lane) : -1;
#pragma unroll
        for (int q = 0; q < Q; ++q) count(tokens[q], base + q * threads + lane);
      }
      __syncthreads();
      n = listed;
      if (n > 0) {
        const float rep = p.repetition ? p.repetition[b] : 1.0f;
        const float freq = p.frequency ? p.frequency[b] : 0.0f, pres = p.presence ? p.presence[b] : 0.0f;
        float top_v = __int_as_float(0xFF800000);
        int top_i = -1;
        for (int base = tid; base < n; base += Q * threads) {
          int place[Q], c[Q];
          float l[Q], add[Q];
          uint32_t open[Q];
#pragma unroll
          for (int q = 0; q < Q; ++q) {
            const int i = base + q * threads;
            if (i >= n) continue;
            place[q] = (int)list[i];
            c[q] = s0 + (TABLE ? (int)(seen[place[q]] >> kCountBits) - 1 : place[q]);
            l[q] = load_plain(x_row, DT, c[q]);
            add[q] = bias ? load_kept(bias + c[q]) : 0.0f;
            open[q] = mask ? load_kept(mask + (c[q] >> 5)) >> (c[q] & 31) : 1u;
          }
#pragma unroll
          for (int q = 0; q < Q; ++q) {
            const int i = base + q * threads;
            if (i >= n) continue;
            const uint32_t times = TABLE ? seen[place[q]] & ((1u << kCountBits) - 1) : reinterpret_cast<const COUNT*>(seen)[place[q]];
            if (bias) l[q] = __fadd_rn(l[q], add[q]);
            float v = penalised(l[q], (float)times, rep, freq, pres);
            if (!(open[q] & 1u)) v = __int_as_float(0xFF800000);
            value[i] = v;
            if (v > top_v || (v == top_v && c[q] < top_i)) {
              top_v = v;
              top_i = c[q];
            }
          }
        }
        const unsigned long long found = top_i >= 0 ? choice_key(top_v, top_i) : 0;
        best = found > best ? found : best;
        __syncthreads();
      }
    }
    for (int k = 0; k < batches; ++k) {
      const int base = s0 + k * batch;
      if (base >= vocab) break;
      if (k > 0) request(base);
      const auto masked = [&](float (&v)[W], uint32_t open, int place) {
        if (n > 0) open &= ~((uint32_t)reinterpret_cast<const uint8_t*>(bits)[place >> 3] >> (place & 7));
#pragma unroll
        for (int e = 0; e < W; ++e)
          if (!((open >> e) & 1u)) v[e] = __int_as_float(0xFF800000);
      };
      if (whole_rows && base + batch <= vocab) {
        float4 w[W / 4];  // the bias of a vector, requested one vector ahead
        const float* const bias_at = bias + base + tid * W;
        if (bias) {
#pragma unroll
          for (int q = 0; q < W / 4; ++q) w[q] = load_kept(reinterpret_cast<const float4*>(bias_at) + q);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int place = k * batch + (tid + u * threads) * W, c0 = s0 + place;
          float v[W];
          unpack<DT>(x[u], v);
          if (bias) {
#pragma unroll
            for (int q = 0; q < W / 4; ++q) {
              const float2 a = __fadd2_rn(make_float2(v[4 * q], v[4 * q + 1]), make_float2(w[q].x, w[q].y));
              const float2 c = __fadd2_rn(make_float2(v[4 * q + 2], v[4 * q + 3]), make_float2(w[q].z, w[q].w));
              v[4 * q] = a.x, v[4 * q + 1] = a.y, v[4 * q + 2] = c.x, v[4 * q + 3] = c.y;
            }
            if (u + 1 < U) {
#pragma unroll
              for (int q = 0; q < W / 4; ++q) w[q] = load_kept(reinterpret_cast<const float4*>(bias_at + (u + 1) * threads * W) + q);
            }
          }
          if (mask || n > 0) masked(v, allowed[u], place);
          if (p.out) {
            if (p.out_dt == DT) {
              *reinterpret_cast<uint4*>(reinterpret_cast<char*>(p.out) + (out_off + c0) * EB) = pack<DT>(v);
            } else {
#pragma unroll
              for (int q = 0; q < W / 4; ++q)
                *(reinterpret_cast<float4*>(reinterpret_cast<float*>(p.out) + out_off + c0) + q) =
                    make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
            }
          }
          if (p.token) {  // only the warps that beat their best so far (one in t at their t-th vector) look for the place
            float top = v[0];
#pragma unroll
            for (int e = 1; e < W; ++e) top = fmaxf(top, v[e]);  // NaN is passed over
            const float warp_top = warp_max_of(top);
            if (warp_top > warp_best) {
              warp_best = warp_top;
              if (top == warp_top) {
                best_v = top;
#pragma unroll
                for (int e = W - 1; e >= 0; --e)
                  if (v[e] == top) best_i = c0 + e;
              }
            }
          }
        }
        continue;
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int place = k * batch + (tid + u * threads) * W, c0 = s0 + place;
        if (c0 >= vocab) continue;
        float v[W];
        unpack<DT>(x[u], v);
        if (bias) {
#pragma unroll
          for (int e = 0; e < W; ++e)
            if (c0 + e >= 0 && c0 + e < vocab) v[e] = __fadd_rn(v[e], load_kept(bias + c0 + e));
        }
        masked(v, allowed[u], place);
        const bool full = c0 >= 0 && c0 + W <= vocab;
#pragma unroll
        for (int e = 0; e < W; ++e) {
          if (!full && (c0 + e < 0 || c0 + e >= vocab)) continue;
          if (v[e] > best_v) {  // false for NaN; the lowest token on ties
            best_v = v[e];
            best_i = c0 + e;
          }
        }
        if (!p.out) continue;
        if (p.out_dt == DT) {
          store_cut<DT>(p.out, out_off, c0, vocab, v);
        } else {
#pragma unroll
          for (int e = 0; e < W; ++e)
            if (full || (c0 + e >= 0 && c0 + e < vocab)) reinterpret_cast<float*>(p.out)[out_off + c0 + e] = v[e];
        }
      }
    }
    if (n > 0) {
      __syncthreads();  // the slab is stored
      for (int i = tid; i < n; i += threads) {
        const int place = (int)list[i], at = TABLE ? (int)(seen[place] >> kCountBits) - 1 : place;
        if (p.out) store_from_f32(p.out, p.out_dt, out_off + s0 + at, value[i]);
        bits[at >> 5] = 0;
        if (TABLE) seen[place] = 0;
        else reinterpret_cast<COUNT*>(seen)[place] = 0;
      }
      if (tid == 0) listed = 0;
    }
  }
  if (!p.token) return;
  const unsigned long long streamed = best_i >= 0 ? choice_key(best_v, best_i) : 0;
  best = streamed > best ? streamed : best;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    const unsigned long long o = __shfl_xor_sync(0xffffffffu, best, off);
    best = o > best ? o : best;
  }
  if ((tid & 31) == 0) best_of[tid >> 5] = best;
  __syncthreads();
  if (tid == 0)
    for (int w = 1; w < (threads >> 5); ++w) best = best_of[w] > best ? best_of[w] : best;
  if (meet) {
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    if (tid == 0) *cg::this_cluster().map_shared_rank(&cluster_best[rank], 0) = best;
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    if (rank != 0) return;  // nobody reads this block's shared memory
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    if (tid == 0)
      for (int k = 1; k < cluster; ++k) best = cluster_best[k] > best ? cluster_best[k] : best;
  }
  if (tid == 0) p.token[b] = best ? (int32_t)~(uint32_t)best : -1;
}

template <int DT, int U, typename COUNT, bool TABLE, bool ALONE>
cudaError_t run_logits(const LogitsPlan& p, int threads, int cluster, int batches, int table, cudaStream_t s) {
  const auto kernel = logits_kernel<DT, U, COUNT, TABLE, ALONE>;
  const int slab = threads * U * kVec<DT> * batches;
  const size_t smem = p.history ? LogitsShared(slab, TABLE ? table : slab, TABLE ? 4 : (int)sizeof(COUNT), sizeof(COUNT), p.max_length).bytes : 0;
  if (smem > 40 * 1024) {  // always to the most, never this call's: threads share the attribute, and a smaller call would lower it
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMostShared);
    if (e != cudaSuccess) return e;
  }
  return launch_after(kernel, dim3((unsigned)(p.batch * cluster)), dim3(threads), smem, s, cluster, p, cluster, batches, table);
}

template <int DT, bool ALONE>
cudaError_t run_logits_blocks(const LogitsPlan& p, int threads, int cluster, cudaStream_t s) {
  constexpr int W = kVec<DT>;
  const int64_t vectors = p.vocab / W + 2;
  // four vectors a thread where a block has that many
  const int u = vectors >= (int64_t)3 * threads * cluster ? 4 : 1;
  const int64_t batch = (int64_t)threads * u * W, needed = (vectors * W + batch * cluster - 1) / (batch * cluster);
  // A table, half full at most, where it leaves an SM its blocks; slabs of 131072 tokens then, as the work on a slab's
  // history does not shrink with it. 256 rows of 131072 with 4096 entries each take 50 us, with 6500 85 us (with bias and mask 62
  // and 134: the shared memory is then missing from the first-level cache); with counts for all of a slab's tokens (slabs
  // of 64 KB of counts) 61 and 97 (75 and 133)
  const int table = (int)std::min<int64_t>((2 * p.max_length + 7) / 4 * 4, 1 << 20);
  const int table_batches = (int)std::max<int64_t>(1, std::min(kTableSlab / batch, needed));
  const size_t room = (ALONE ? 220 : 110) * 1024;
  if (p.max_length < (1 << kCountBits) && LogitsShared((int)(table_batches * batch), table, 4, 2, p.max_length).bytes <= room) {
    if (u == 4) return run_logits<DT, 4, uint16_t, true, ALONE>(p, threads, cluster, table_batches, table, s);
    return run_logits<DT, 1, uint16_t, true, ALONE>(p, threads, cluster, table_batches, table, s);
  }
  const bool narrow = p.max_length < (1 << 16);
  // as many tokens a slab as 64 KB of counts take, and as their list leaves room for: one batch always has (16384 tokens
  // at most, which are 194 KB with counts of 32 bits)
  int batches = (int)std::max<int64_t>(1, std::min(64 * 1024 / (batch * (narrow ? 2 : 4)), needed));
  const auto bytes = [&](int n) { return LogitsShared((int)(n * batch), (int)(n * batch), narrow ? 2 : 4, narrow ? 2 : 4, p.max_length).bytes; };
  while (batches > 1 && bytes(batches) > kMostShared) --batches;
  if (u == 4)
    return narrow ? run_logits<DT, 4, uint16_t, false, ALONE>(p, threads, cluster, batches, 0, s)
                  : run_logits<DT, 4, uint32_t, false, ALONE>(p, threads, cluster, batches, 0, s);
  return narrow ? run_logits<DT, 1, uint16_t, false, ALONE>(p, threads, cluster, batches, 0, s)
                : run_logits<DT, 1, uint32_t, false, ALONE>(p, threads, cluster, batches, 0, s);
}

template <int DT>
cudaError_t run_logits_type(const LogitsPlan& p, cudaStream_t s) {
  const int64_t vectors = p.vocab / kVec<DT> + 2;
  const int threads = (int)std::min<int64_t>(kThreads, (vectors + 31) / 32 * 32);
  // as many blocks a row as give every SM one and a half, but no more than the row has vectors for
  int cluster = 1;
  while (cluster < 8 && p.batch * cluster * 2 < 3 * device_sm_count() && cluster * threads < vectors) cluster *= 2;
  if (p.batch * cluster <= device_sm_count()) return run_logits_blocks<DT, true>(p, threads, cluster, s);
  return run_logits_blocks<DT, false>(p, threads, cluster, s);
}

cudaError_t launch_logits(const LogitsPlan& p, cudaStream_t s) {
  Rows<2> m = {};
  m.n = p.batch > 1 ? 1 : 0;
  m.stride[0][0] = p.x_stride;
  m.stride[1][0] = p.out_stride;
  const void* const ptr[2] = {p.x, p.out};
  const int eb[2] = {dt_bytes(p.dt), dt_bytes(p.out_dt)};
  bool cut = false;
  if (p.vocab > 0 && p.vocab <= (1 << 30) && vectors_fit<2>(m, ptr, eb, p.vocab, p.dt == F32 ? 4 : 8, &cut)) {
    if (p.dt == F32) return run_logits_type<F32>(p, s);
    if (p.dt == BF16) return run_logits_type<BF16>(p, s);
    return run_logits_type<F16>(p, s);
  }
  logits_any_kernel<<<(unsigned)p.batch, kThreads, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace hlo
