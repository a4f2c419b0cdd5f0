// Gradient of the root-mean-square norm. See hlo_rms_norm_backward in hlo_fusion.h for the formulas.
#include <map>
#include <mutex>
#include <tuple>

#include "norm_common.cuh"

namespace hlo {

// ---- gradient --------------------------------------------------------------------------------------------
// dweight, before the rows' gradients replace anything: block (x, y) sums columns [256 x, 256 x + 256) over
// the rows y, y + groups, ... into the workspace; norm_grad_join_kernel adds the groups in order.
__global__ void __launch_bounds__(kAnyThreads) norm_grad_weight_any_kernel(NormGradPlan p) {
  const int64_t c = (int64_t)blockIdx.x * kAnyThreads + threadIdx.x;
  if (c >= p.n) return;
  float acc = 0.0f;
  for (int64_t row = blockIdx.y; row < p.rows; row += gridDim.y) {
    int64_t off[5];
    row_offsets(p.map, row, off);
    acc += load_plain(p.dy, p.dt, off[0] + c) * (load_plain(p.h, p.dt, off[1] + c) * p.rstd[row]);
  }
  p.ws[(int64_t)blockIdx.y * p.n + c] = acc;
}

__global__ void __launch_bounds__(kAnyThreads) norm_grad_any_kernel(NormGradPlan p) {
  __shared__ float red[2 * kAnyThreads / 32];
  Philox g = {};
  if (p.drop.on) g = philox_of(p.drop);
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    int64_t off[5];
    row_offsets(p.map, row, off);
    const float r = p.rstd[row];
    float dot = 0.0f, none = 0.0f;
    for (int64_t c = threadIdx.x; c < p.n; c += kAnyThreads) {
      const float gy = load_plain(p.dy, p.dt, off[0] + c) * weight_at(p.w, p.w_dt, p.w_offset, c);
      dot = fmaf(gy, load_plain(p.h, p.dt, off[1] + c) * r, dot);
    }
    block_sum_max(dot, none, red);
    const float mean = __fdiv_rn(dot, (float)p.n);
    for (int64_t c = threadIdx.x; c < p.n; c += kAnyThreads) {
      const float gy = load_plain(p.dy, p.dt, off[0] + c) * weight_at(p.w, p.w_dt, p.w_offset, c);
      const float xh = load_plain(p.h, p.dt, off[1] + c) * r;
      float dh = r * (gy - xh * mean);
      if (p.dsum) dh += load_plain(p.dsum, p.dt, off[2] + c);
      store_from_f32(p.dh, p.dt, off[3] + c, dh);
      if (p.dx) store_from_f32(p.dx, p.dt, off[4] + c, drop1(p.drop, g, (uint64_t)(row * p.n + c), dh));
    }
    __syncthreads();  // red is used again by the next row
  }
}

// ---- gradient, rows held in registers ------------------------------------------------------------------------
// Row groups walk the rows with a stride of all groups, keep dy, h and dsum of a row in registers (packed)
// across its one reduction, and add each row's share of dweight to sums of their own: in registers, where
// every row has the same columns in a thread (!CUT), else in shared memory, where column c of a group sits
// at c + c / W, so that threads W columns apart meet no bank twice. A thread adds to a column only behind
// its group's barrier of that row, so two rows never add to one at once. The groups' sums go to the
// workspace, and norm_grad_join_kernel adds them in order.
template <int DT, int K, bool DROP, bool CUT>
__global__ void __launch_bounds__(K == 1 ? 1024 : 512) norm_grad_row_kernel(NormGradPlan p, int weight_whole, int64_t groups) {
  constexpr int W = kVec<DT>, EB = 16 / W;
  __shared__ float red[2][64];
  extern __shared__ float dw_shared[];
  const int n = (int)p.n;
  const int64_t group = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  if (group >= groups) return;  // the whole group: its barrier is its own
  Philox g = {};
  if (DROP) g = philox_of(p.drop);
  float acc[K][W];
  float* const cols = CUT ? dw_shared + (int)threadIdx.y * (n + n / W + 1) : nullptr;
  if (CUT) {
    if (p.dw)
      for (int c = threadIdx.x; c < n + n / W + 1; c += blockDim.x) cols[c] = 0.0f;
  } else {
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int e = 0; e < W; ++e) acc[k][e] = 0.0f;
  }
  int phase = 0;
  for (int64_t row = group; row < p.rows; row += groups, phase ^= 1) {
    int64_t off[5];
    row_offsets(p.map, row, off);
    const int shift = CUT ? (int)(((int64_t)((uintptr_t)p.dy / EB) + off[0]) & (W - 1)) : 0;
    const bool whole_w = weight_whole && shift == 0;
    const float r = p.rstd[row];
    uint4 yr[K], hr[K], sr[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c0 = (int)(threadIdx.x + k * blockDim.x) * W - shift;
      yr[k] = hr[k] = sr[k] = make_uint4(0, 0, 0, 0);
      if (c0 >= n) continue;
      if (CUT) {
        yr[k] = load_cut<DT>(p.dy, off[0], c0, p.n);
        hr[k] = load_cut<DT>(p.h, off[1], c0, p.n);
        if (p.dsum) sr[k] = load_cut<DT>(p.dsum, off[2], c0, p.n);
      } else {
        yr[k] = load16(reinterpret_cast<const char*>(p.dy) + (off[0] + c0) * EB);
        hr[k] = load16(reinterpret_cast<const char*>(p.h) + (off[1] + c0) * EB);
        if (p.dsum) sr[k] = load16(reinterpret_cast<const char*>(p.dsum) + (off[2] + c0) * EB);
      }
    }
    float dot = 0.0f, none = 0.0f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c0 = (int)(threadIdx.x + k * blockDim.x) * W - shift;
      if (c0 >= n) continue;
      float y[W], h[W], w[W];
      unpack<DT>(yr[k], y);
      unpack<DT>(hr[k], h);
      load_weights<DT>(p.w, p.w_dt, p.w_offset, c0, n, whole_w && (!CUT || c0 + W <= n), w);
#pragma unroll
      for (int e = 0; e < W; ++e) dot = fmaf(y[e] * w[e], h[e] * r, dot);
    }
    group_sum_max<false>(dot, none, red[phase]);
    if (CUT && blockDim.x == 32) __syncwarp();
    const float mean = __fdiv_rn(dot, (float)p.n);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c0 = (int)(threadIdx.x + k * blockDim.x) * W - shift;
      if (c0 >= n) continue;
      float y[W], h[W], w[W], d[W];
      unpack<DT>(yr[k], y);
      unpack<DT>(hr[k], h);
      unpack<DT>(sr[k], d);
      load_weights<DT>(p.w, p.w_dt, p.w_offset, c0, n, whole_w && (!CUT || c0 + W <= n), w);
#pragma unroll
      for (int e = 0; e < W; ++e) {
        const float xh = h[e] * r;
        if (CUT) {
          const int c = c0 + e;
          if (p.dw && c >= 0 && c < n) cols[c + c / W] = fmaf(y[e], xh, cols[c + c / W]);
        } else {
          acc[k][e] = fmaf(y[e], xh, acc[k][e]);
        }
        d[e] = fmaf(r, fmaf(-xh, mean, y[e] * w[e]), d[e]);
      }
      if (CUT) store_cut<DT>(p.dh, off[3], c0, n, d);
      else *reinterpret_cast<uint4*>(reinterpret_cast<char*>(p.dh) + (off[3] + c0) * EB) = pack<DT>(d);
      if (DROP) {
        drop_vec<W>(p.drop, g, row * n + c0, d);
        if (CUT) store_cut<DT>(p.dx, off[4], c0, n, d);
        else *reinterpret_cast<uint4*>(reinterpret_cast<char*>(p.dx) + (off[4] + c0) * EB) = pack<DT>(d);
      }
    }
  }
  if (!p.dw) return;
  float* const out = p.ws + group * p.n;
  if (CUT) {
    if (blockDim.x == 32) __syncwarp();
    else group_barrier();
    for (int c = threadIdx.x; c < n; c += blockDim.x) out[c] = cols[c + c / W];
  } else {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c0 = (int)(threadIdx.x + k * blockDim.x) * W;
      if (c0 >= n) continue;
#pragma unroll
      for (int q = 0; q < W / 4; ++q)
        *(reinterpret_cast<float4*>(out + c0) + q) = make_float4(acc[k][4 * q], acc[k][4 * q + 1], acc[k][4 * q + 2], acc[k][4 * q + 3]);
    }
  }
}

// dw[c] = sum of the groups' shares, in a fixed order: 32 columns a block, 32 threads a column.
__global__ void __launch_bounds__(1024) norm_grad_join_kernel(const float* ws, float* dw, int64_t n, int64_t groups) {
  __shared__ float part[32][33];
  const int64_t c = (int64_t)blockIdx.x * 32 + threadIdx.x;
  float acc = 0.0f;
  if (c < n)
    for (int64_t k = threadIdx.y; k < groups; k += 32) acc += ws[k * n + c];
  part[threadIdx.y][threadIdx.x] = acc;
  __syncthreads();
  acc = warp_sum(part[threadIdx.x][threadIdx.y]);
  if (threadIdx.x == 0 && (int64_t)blockIdx.x * 32 + threadIdx.y < n) dw[(int64_t)blockIdx.x * 32 + threadIdx.y] = acc;
}

// At most 16 groups an SM (short rows), and not more than 8 MB of shares in all, but two groups an SM at
// least.
int64_t norm_grad_partials(int64_t rows, int64_t n) {
  const int64_t sms = device_sm_count();
  const int64_t most = std::max<int64_t>(2 * sms, std::min<int64_t>(16 * sms, (1 << 21) / n));
  return std::min(rows, most);
}

// Blocks of a kernel that an SM holds at this size, asked for once per (kernel, size, device); raises the
// kernel's dynamic shared-memory limit where that is needed.
cudaError_t resident_blocks(const void* kernel, int threads, size_t smem, int* blocks) {
  static std::mutex mu;
  static std::map<std::tuple<const void*, int, size_t, int>, int> cache;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::lock_guard<std::mutex> lock(mu);
  const auto key = std::make_tuple(kernel, threads, smem, dev);
  const auto it = cache.find(key);
  if (it != cache.end()) {
    *blocks = it->second;
    return cudaSuccess;
  }
  if (smem > 48 * 1024) {  // to the most that this library asks for, whatever the order of the calls
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 100 * 1024);
    if (e != cudaSuccess) return e;
  }
  int n = 0;
  e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, threads, smem);
  if (e != cudaSuccess) return e;
  if (cache.size() > 65536) cache.clear();
  *blocks = cache[key] = n > 0 ? n : 1;
  return cudaSuccess;
}

template <int DT, int K, bool DROP, bool CUT>
cudaError_t run_norm_grad_row(const NormGradPlan& p, const RowShape& r, int whole, int64_t* groups, cudaStream_t s) {
  const auto kernel = norm_grad_row_kernel<DT, K, DROP, CUT>;
  const size_t smem = CUT && p.dw ? (size_t)r.ty * (p.n + p.n / kVec<DT> + 1) * 4 : 0;
  int per_sm = 1;
  const cudaError_t e = resident_blocks((const void*)kernel, r.tx * r.ty, smem, &per_sm);
  if (e != cudaSuccess) return e;
  *groups = std::min({p.rows, norm_grad_partials(p.rows, p.n), (int64_t)device_sm_count() * per_sm * r.ty});
  kernel<<<(unsigned)((*groups + r.ty - 1) / r.ty), dim3(r.tx, r.ty), smem, s>>>(p, whole, *groups);
  return cudaGetLastError();
}

template <int DT>
cudaError_t run_norm_grad(const NormGradPlan& p, const RowShape& r, bool cut, int whole, int64_t* groups, cudaStream_t s) {
  const bool drop = p.drop.on;
#define HLO_CASE(KK)                                                                                             \
  if (r.k == KK)                                                                                                 \
    return cut ? (drop ? run_norm_grad_row<DT, KK, true, true>(p, r, whole, groups, s)                           \
                       : run_norm_grad_row<DT, KK, false, true>(p, r, whole, groups, s))                         \
               : (drop ? run_norm_grad_row<DT, KK, true, false>(p, r, whole, groups, s)                          \
                       : run_norm_grad_row<DT, KK, false, false>(p, r, whole, groups, s))
  HLO_CASE(1);
  HLO_CASE(2);
  HLO_CASE(4);
#undef HLO_CASE
  return cudaErrorInvalidValue;
}

cudaError_t launch_norm_grad(const NormGradPlan& p, cudaStream_t s) {
  const int w = p.dt == F32 ? 4 : 8, eb = dt_bytes(p.dt);
  const void* const ptr[5] = {p.dy, p.h, p.dsum, p.dh, p.dx};
  const int ebs[5] = {eb, eb, eb, eb, eb};
  bool cut = false;
  const int64_t vectors = (p.n + w - 1) / w + 1;
  int64_t groups = norm_grad_partials(p.rows, p.n);
  if (vectors <= 512 * 4 && vectors_fit<5>(p.map, ptr, ebs, p.n, w, &cut)) {
    const RowShape r = row_shape(p.rows, vectors - (cut ? 0 : 1), 4);
    const int whole = p.w && (uintptr_t)p.w % 16 == 0;
    const cudaError_t e = p.dt == F32    ? run_norm_grad<F32>(p, r, cut, whole, &groups, s)
                          : p.dt == BF16 ? run_norm_grad<BF16>(p, r, cut, whole, &groups, s)
                                         : run_norm_grad<F16>(p, r, cut, whole, &groups, s);
    if (e != cudaSuccess) return e;
  } else {
    if (p.dw) {
      const unsigned cols = (unsigned)((p.n + kAnyThreads - 1) / kAnyThreads);
      norm_grad_weight_any_kernel<<<dim3(cols, (unsigned)groups), kAnyThreads, 0, s>>>(p);
    }
    norm_grad_any_kernel<<<any_grid(p.rows), kAnyThreads, 0, s>>>(p);
  }
  if (p.dw) norm_grad_join_kernel<<<(unsigned)((p.n + 31) / 32), dim3(32, 32), 0, s>>>(p.ws, p.dw, p.n, groups);
  return cudaGetLastError();
}

}  // namespace hlo
