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

// Blocks of a cluster take slabs of one row in turn: blockDim.x U vectors each. A slab's logits are requested
// first; while they come, the block counts the occurrences of the slab's tokens in shared memory: COUNT
// is uint16_t (histories below 2^15) or uint32_t, its top bit says "occurs in the prompt" and the rest
// counts what came after. Adding and or-ing whole numbers gives one result in any order. The blocks' best
// tokens meet in the first block through distributed shared memory.
template <int DT, int U, typename COUNT>
__global__ void __launch_bounds__(kThreads) logits_kernel(LogitsPlan p, int cluster) {
  constexpr int W = kVec<DT>, EB = 16 / W;
  constexpr int CB = sizeof(COUNT), CPW = 4 / CB;  // counts a 32-bit word
  constexpr uint32_t TOP = CB == 2 ? 0x8000u : 0x80000000u;
  extern __shared__ uint4 seen4[];
  uint32_t* const seen = reinterpret_cast<uint32_t*>(seen4);
  __shared__ unsigned long long best_of[kThreads / 32];
  __shared__ unsigned long long block_best;
  const int64_t b = blockIdx.x / cluster;
  const int rank = (int)(blockIdx.x - b * cluster);
  const int vocab = (int)p.vocab;
  const int64_t x_off = b * p.x_stride, out_off = b * p.out_stride;
  const int shift = (int)(((int64_t)((uintptr_t)p.x / EB) + x_off) & (W - 1));
  int32_t len = 0, prompt = 0;
  if (p.history) {
    len = (int32_t)p.max_length;
    if (p.lengths) len = max(0, min(len, p.lengths[b]));
    if (p.prompts) prompt = p.prompts[b];
  }
  const float rep = p.repetition ? p.repetition[b] : 1.0f;
  const float freq = p.frequency ? p.frequency[b] : 0.0f, pres = p.presence ? p.presence[b] : 0.0f;
  const int words = (vocab + 31) / 32;
  const uint32_t* const mask = p.mask ? p.mask + b * p.mask_stride : nullptr;
  const float* const bias = p.bias ? p.bias + b * p.bias_stride : nullptr;
  const bool bias_whole = bias && shift == 0 && (uintptr_t)bias % 16 == 0;
  const int slab = (int)blockDim.x * U * W;
  float best_v = __int_as_float(0xFF800000);
  int best_i = -1;
  for (int64_t start = (int64_t)rank * slab - shift; start < vocab; start += (int64_t)cluster * slab) {
    const int s0 = (int)start;
    uint4 xr[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t c0 = start + (int64_t)(threadIdx.x + u * blockDim.x) * W;
      xr[u] = c0 < vocab ? load_cut<DT>(p.x, x_off, c0, vocab) : make_uint4(0, 0, 0, 0);
    }
    if (len > 0) {
      for (int i = threadIdx.x; i < slab * CB / 16; i += blockDim.x) seen4[i] = make_uint4(0, 0, 0, 0);
      __syncthreads();
      const int32_t* const h = p.history + b * p.history_stride;
#pragma unroll 4
      for (int32_t i = threadIdx.x; i < len; i += blockDim.x) {
        const int64_t t = (int64_t)__ldg(h + i) - s0;
        if (t < 0 || t >= slab) continue;
        const int at = (int)t, bit = 8 * CB * (at % CPW);
        if (i < prompt) atomicOr(&seen[at / CPW], TOP << bit);
        else atomicAdd(&seen[at / CPW], 1u << bit);
      }
      __syncthreads();
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int place = (int)(threadIdx.x + u * blockDim.x) * W;
      if ((int64_t)s0 + place >= vocab) continue;
      const int c0 = s0 + place;
      float v[W];
      unpack<DT>(xr[u], v);
      if (bias) {
        float w[W];
        if (bias_whole && c0 + W <= vocab) {
#pragma unroll
          for (int q = 0; q < W / 4; ++q) {
            const float4 f = __ldg(reinterpret_cast<const float4*>(bias + c0) + q);
            w[4 * q] = f.x, w[4 * q + 1] = f.y, w[4 * q + 2] = f.z, w[4 * q + 3] = f.w;
          }
        } else {
#pragma unroll
          for (int e = 0; e < W; ++e) w[e] = c0 + e >= 0 && c0 + e < vocab ? __ldg(bias + c0 + e) : 0.0f;
        }
#pragma unroll
        for (int e = 0; e < W; ++e) v[e] = __fadd_rn(v[e], w[e]);
      }
      if (len > 0) {
        uint32_t n[W / CPW], any = 0;
#pragma unroll
        for (int q = 0; q < W / CPW; ++q) any |= n[q] = seen[place / CPW + q];
        if (any) {
#pragma unroll
          for (int e = 0; e < W; ++e) {
            const uint32_t c = CB == 2 ? (n[e / CPW] >> (16 * (e % CPW))) & 0xFFFFu : n[e / CPW];
            if (c) v[e] = penalised(v[e], (float)(c & (TOP - 1)), rep, freq, pres);
          }
        }
      }
      if (mask) {
        const int w0 = c0 >> 5;  // -1 for the columns before the row, which are not stored
        const uint32_t lo = w0 >= 0 ? __ldg(mask + w0) : 0;
        const uint32_t hi = (c0 & 31) + W > 32 && w0 + 1 < words ? __ldg(mask + w0 + 1) : 0;
        const uint32_t bits = __funnelshift_r(lo, hi, c0 & 31);
#pragma unroll
        for (int e = 0; e < W; ++e)
          if (!((bits >> e) & 1u)) v[e] = __int_as_float(0xFF800000);
      }
      const bool full = c0 >= 0 && c0 + W <= vocab;
#pragma unroll
      for (int e = 0; e < W; ++e) {
        if (v[e] > best_v && (full || (c0 + e >= 0 && c0 + e < vocab))) {  // false for NaN; the lowest token on ties
          best_v = v[e];
          best_i = c0 + e;
        }
      }
      if (!p.out) continue;
      if (p.out_dt == DT) {
        store_cut<DT>(p.out, out_off, c0, vocab, v);
      } else if (full) {
#pragma unroll
        for (int q = 0; q < W / 4; ++q)
          *(reinterpret_cast<float4*>(reinterpret_cast<float*>(p.out) + out_off + c0) + q) =
              make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
      } else {
#pragma unroll
        for (int e = 0; e < W; ++e)
          if (c0 + e >= 0 && c0 + e < vocab) reinterpret_cast<float*>(p.out)[out_off + c0 + e] = v[e];
      }
    }
    if (len > 0) __syncthreads();  // the counts are zeroed for the next slab
  }
  if (!p.token) return;
  unsigned long long best = best_i >= 0 ? choice_key(best_v, best_i) : 0;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    const unsigned long long o = __shfl_xor_sync(0xffffffffu, best, off);
    best = o > best ? o : best;
  }
  if ((threadIdx.x & 31) == 0) best_of[threadIdx.x >> 5] = best;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < (int)(blockDim.x >> 5); ++w) best = best_of[w] > best ? best_of[w] : best;
    block_best = best;
  }
  if (cluster > 1) {
    cg::cluster_group c = cg::this_cluster();
    c.sync();
    if (rank == 0 && threadIdx.x < 32) {
      best = threadIdx.x < cluster ? *c.map_shared_rank(&block_best, threadIdx.x) : 0;
#pragma unroll
      for (int off = 4; off > 0; off >>= 1) {
        const unsigned long long o = __shfl_xor_sync(0xffffffffu, best, off);
        best = o > best ? o : best;
      }
    }
    c.sync();  // no block leaves before its best was read
  }
  if (rank == 0 && threadIdx.x == 0) p.token[b] = best ? (int32_t)~(uint32_t)best : -1;
}

template <int DT, int U, typename COUNT>
cudaError_t run_logits(const LogitsPlan& p, int threads, int cluster, cudaStream_t s) {
  const auto kernel = logits_kernel<DT, U, COUNT>;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3((unsigned)(p.batch * cluster));
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = p.history ? (size_t)threads * U * kVec<DT> * sizeof(COUNT) : 0;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 1 : 0;
  if (cfg.dynamicSmemBytes > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)cfg.dynamicSmemBytes);
    if (e != cudaSuccess) return e;
  }
  return cudaLaunchKernelEx(&cfg, kernel, p, cluster);
}

template <int DT>
cudaError_t run_logits_type(const LogitsPlan& p, cudaStream_t s) {
  const int64_t vectors = p.vocab / kVec<DT> + 2;
  const int threads = (int)std::min<int64_t>(kThreads, (vectors + 31) / 32 * 32);
  // four vectors a thread once that leaves every SM two blocks; then as many blocks a row as it has slabs
  const bool many = p.batch * vectors >= (int64_t)device_sm_count() * 2 * 4 * kThreads;
  const int64_t slabs = (vectors + threads * (many ? 4 : 1) - 1) / (threads * (many ? 4 : 1));
  int cluster = 1;
  while (cluster < 8 && cluster < slabs) cluster *= 2;
  const bool narrow = p.max_length < (1 << 15);
  if (many) return narrow ? run_logits<DT, 4, uint16_t>(p, threads, cluster, s) : run_logits<DT, 4, uint32_t>(p, threads, cluster, s);
  return narrow ? run_logits<DT, 1, uint16_t>(p, threads, cluster, s) : run_logits<DT, 1, uint32_t>(p, threads, cluster, s);
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
