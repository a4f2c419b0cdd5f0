// Processing of logits (hlo_logits_process): bias, penalties for tokens of the history, mask, greedy token.
#include "rows.cuh"

namespace hlo {

constexpr int kThreads = 512;
constexpr int kSlab = 8192;  // tokens whose occurrences are counted at once, in shared memory

// A key whose order is "greater value first, lower token on ties"; 0 for NaN and -inf, which are never
// chosen. Adding +0 makes -0 equal to +0.
__device__ __forceinline__ unsigned long long choice_key(float l, int token) {
  l = __fadd_rn(l, 0.0f);
  if (!(l > __int_as_float(0xFF800000))) return 0;
  const uint32_t b = __float_as_uint(l);
  const uint32_t ordered = (b & 0x80000000u) ? ~b : b | 0x80000000u;
  return ((unsigned long long)ordered << 32) | (uint32_t)~token;
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
        const float c = (float)(s & 0x7FFFFFFFu);
        l = l > 0.0f ? __fdiv_rn(l, rep) : __fmul_rn(l, rep);
        l = __fsub_rn(l, __fmul_rn(freq, c));
        if (c > 0.0f) l = __fsub_rn(l, pres);
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

cudaError_t launch_logits(const LogitsPlan& p, cudaStream_t s) {
  logits_any_kernel<<<(unsigned)p.batch, kThreads, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace hlo
