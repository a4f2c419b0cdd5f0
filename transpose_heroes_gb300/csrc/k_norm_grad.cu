// Gradient of the root-mean-square norm. See hlo_rms_norm_backward in hlo_fusion.h for the formulas.
#include <map>
#include <mutex>
#include <tuple>

#include "async_copy.cuh"
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

template <int DROP>
__global__ void __launch_bounds__(kAnyThreads) norm_grad_any_kernel(const __grid_constant__ NormGradPlan p) {
  __shared__ float red[2 * kAnyThreads / 32];
  const Philox<DROP> g(p.drop);
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
      if constexpr (DROP != DROP_NONE)
        store_from_f32(p.dx, p.dt, off[4] + c, drop1(p.drop, g, (uint64_t)(row * p.n + c), dh));
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
//
// CUT rows are taken apart as in norm_row_kernel; their weights lie in shared memory too, in the same places. (A column a thread, for
// sums and weights in registers at any alignment, took 120 us in place of 80: one element an access.)
// Bound: the loads wait for the row's reduction, so an SM has few bytes in flight; this form serves cut rows and
// few rows. 2049 x 1001 f32 (33 MB, in the second-level cache) 12 us with dweight, 16384 x 1001 f32 (262 MB) 52 us,
// 5.1 TB/s; 32768 x 1001 bf16 80 us, the column sums in shared memory costing as much as the row itself.
template <int DT, int K, int DROP, bool CUT>
__global__ void __launch_bounds__(K == 1 ? 1024 : 512) norm_grad_row_kernel(const __grid_constant__ NormGradPlan p, int weight_whole, int64_t groups) {
  constexpr int W = kVec<DT>, EB = 16 / W;
  __shared__ float red[2][64];
  extern __shared__ float cut_shared[];
  const int n = (int)p.n, places = n + n / W + 1;
  wait_for_last();
  const int64_t group = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  const bool idle = group >= groups;
  const Philox<DROP> g(p.drop);
  float acc[K][W];
  float* const ws = cut_shared;
  float* const cols = cut_shared + (1 + (int)threadIdx.y) * places;
  if (CUT) {
    const int t0 = threadIdx.y * blockDim.x + threadIdx.x, step = blockDim.x * blockDim.y;
    if (p.w && p.w_dt == DT) {  // without the choices of weight_at the loads go out eight at a time: 333 x 8191 bf16 10 us in place of 16
#pragma unroll 8
      for (int c = t0; c < n; c += step) ws[c + c / W] = load_plain(p.w, DT, c) + p.w_offset;
    } else {
      for (int c = t0; c < n; c += step) ws[c + c / W] = weight_at(p.w, p.w_dt, p.w_offset, c);
    }
    if (p.dw)
      for (int c = threadIdx.x; c < places; c += blockDim.x) cols[c] = 0.0f;
    __syncthreads();
  } else {
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int e = 0; e < W; ++e) acc[k][e] = 0.0f;
  }
  const auto weights = [&](int c0, float (&w)[W]) {
    if (CUT) {
#pragma unroll
      for (int e = 0; e < W; ++e) w[e] = ws[c0 + e + (c0 + e) / W];
    } else {
      load_weights<DT>(p.w, p.w_dt, p.w_offset, c0, n, weight_whole, w);
    }
  };
  int phase = 0;
  for (int64_t row = idle ? p.rows : group; row < p.rows; row += groups, phase ^= 1) {
    int64_t off[5];
    row_offsets(p.map, row, off);
    const RowCut cut = CUT ? row_cut<W>(p.dy, EB, off[0], n) : RowCut{0, n};
    const int edge = CUT ? cut.edge(threadIdx.x, n) : -1;
    const float r = p.rstd[row];
    uint4 yr[K], hr[K], sr[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c0 = cut.head + (int)(threadIdx.x + k * blockDim.x) * W;
      yr[k] = hr[k] = sr[k] = make_uint4(0, 0, 0, 0);
      if (c0 >= cut.end) continue;
      yr[k] = load16(reinterpret_cast<const char*>(p.dy) + (off[0] + c0) * EB);
      hr[k] = load16(reinterpret_cast<const char*>(p.h) + (off[1] + c0) * EB);
      if (p.dsum) sr[k] = load16(reinterpret_cast<const char*>(p.dsum) + (off[2] + c0) * EB);
    }
    float dot = 0.0f, ye = 0.0f, he = 0.0f, de = 0.0f, we = 0.0f;
    if (CUT && edge >= 0) {
      ye = load_plain(p.dy, DT, off[0] + edge);
      he = load_plain(p.h, DT, off[1] + edge) * r;
      if (p.dsum) de = load_plain(p.dsum, DT, off[2] + edge);
      we = ws[edge + edge / W];
      dot = ye * we * he;
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c0 = cut.head + (int)(threadIdx.x + k * blockDim.x) * W;
      if (c0 >= cut.end) continue;
      float y[W], h[W], w[W];
      unpack<DT>(yr[k], y);
      unpack<DT>(hr[k], h);
      weights(c0, w);
#pragma unroll
      for (int e = 0; e < W; ++e) dot = fmaf(y[e] * w[e], h[e] * r, dot);
    }
    group_sum(dot, red[phase]);
    if (CUT && blockDim.x == 32) __syncwarp();
    const float mean = __fdiv_rn(dot, (float)p.n);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c0 = cut.head + (int)(threadIdx.x + k * blockDim.x) * W;
      if (c0 >= cut.end) continue;
      float y[W], h[W], w[W], d[W];
      unpack<DT>(yr[k], y);
      unpack<DT>(hr[k], h);
      unpack<DT>(sr[k], d);
      weights(c0, w);
#pragma unroll
      for (int e = 0; e < W; ++e) {
        const float xh = h[e] * r;
        if (CUT) {
          const int at = c0 + e + (c0 + e) / W;
          if (p.dw) cols[at] = fmaf(y[e], xh, cols[at]);
        } else {
          acc[k][e] = fmaf(y[e], xh, acc[k][e]);
        }
        d[e] = fmaf(r, fmaf(-xh, mean, y[e] * w[e]), d[e]);
      }
      *reinterpret_cast<uint4*>(reinterpret_cast<char*>(p.dh) + (off[3] + c0) * EB) = pack<DT>(d);
      if constexpr (DROP != DROP_NONE) {
        drop_vec<DROP, !CUT, W>(p.drop, g, row * n + c0, d);
        *reinterpret_cast<uint4*>(reinterpret_cast<char*>(p.dx) + (off[4] + c0) * EB) = pack<DT>(d);
      }
    }
    if (CUT && edge >= 0) {
      if (p.dw) cols[edge + edge / W] = fmaf(ye, he, cols[edge + edge / W]);
      de = fmaf(r, fmaf(-he, mean, ye * we), de);
      store_from_f32(p.dh, DT, off[3] + edge, de);
      if constexpr (DROP != DROP_NONE) store_from_f32(p.dx, DT, off[4] + edge, drop1(p.drop, g, (uint64_t)(row * n + edge), de));
    }
  }
  allow_next();
  if (!p.dw) return;
  if (CUT) {  // the block's groups in order, as one share
    __syncthreads();
    float* const out = p.ws + (int64_t)blockIdx.x * n;
    for (int c = threadIdx.y * blockDim.x + threadIdx.x; c < n; c += blockDim.x * blockDim.y) {
      float sum = 0.0f;
      for (int y = 1; y <= (int)blockDim.y; ++y) sum += cut_shared[y * places + c + c / W];
      out[c] = sum;
    }
  } else if (!idle) {
    float* const out = p.ws + group * p.n;
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

// ---- gradient, rows streamed through shared memory ---------------------------------------------------------
// For many aligned rows, a fixed stride apart: persistent blocks, a row at a time; thread 0 keeps a ring of `stages` rows (dy, h and
// dsum) coming with bulk copies, so the loads never wait for the row's reduction. K vectors a thread.
// One barrier a row: it joins the warps' dot products, and behind it every thread has left the row
// before, whose stage is refilled then. Sums are formed with packed f32x2 instructions.
// Bound: HBM without dropout (8192 x 4096 bf16, 268 MB: 46 us alone, 47.5 a call with the join, 5.7 TB/s),
// the row's phases with it, as the masks are drawn by all warps after the row's barrier (336 MB in 70 us, 4.8 TB/s: multiplier
// 57%, ALU 45%, issue 57% busy).
constexpr int kMaxStages = 8;

template <int DT, int K, int DROP, int MAXT>
__global__ void __launch_bounds__(MAXT, MAXT == 512 ? 1 : K == 4 ? 2 : 3) norm_grad_stream_kernel(const __grid_constant__ NormGradPlan p, int stages, int weight_whole) {
  constexpr int W = kVec<DT>, EB = 16 / W, H = W / 2;
  extern __shared__ __align__(128) char ring[];
  __shared__ __align__(8) uint64_t full[kMaxStages];
  __shared__ float red[2][16];
  wait_for_last();
  const int n = (int)p.n, tid = threadIdx.x, warps = blockDim.x >> 5;
  const int row_bytes = n * EB, stage_bytes = row_bytes * (p.dsum ? 3 : 2);
  const int mine = (int)((p.rows - blockIdx.x + gridDim.x - 1) / gridDim.x);  // rows of this block
  const auto request = [&](int i) {
    const int s = i % stages;
    const int64_t row = (int64_t)blockIdx.x + (int64_t)i * gridDim.x;
    const uint32_t bar = smem_addr(&full[s]);
    char* const to = ring + (size_t)s * stage_bytes;
    mbar_arrive_expect_tx(bar, stage_bytes);
    bulk_load(to, reinterpret_cast<const char*>(p.dy) + row * p.map.stride[0][0] * EB, row_bytes, bar);
    bulk_load(to + row_bytes, reinterpret_cast<const char*>(p.h) + row * p.map.stride[1][0] * EB, row_bytes, bar);
    if (p.dsum) bulk_load(to + 2 * row_bytes, reinterpret_cast<const char*>(p.dsum) + row * p.map.stride[2][0] * EB, row_bytes, bar);
  };
  if (tid == 0) {
    for (int s = 0; s < stages; ++s) mbar_init(smem_addr(&full[s]), 1);
    fence_mbar_init();
  }
  __syncthreads();
  if (tid == 0)
    for (int i = 0; i < min(stages, mine); ++i) request(i);
  const Philox<DROP> g(p.drop);
  float2 acc[K][H];
  // the weights stay packed in registers where they are of the rows' type, and come from the caches otherwise
  const bool packed = p.w && p.w_dt == DT && weight_whole;
  uint4 wr[K];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int c0 = (int)(tid + k * blockDim.x) * W;
    wr[k] = packed && c0 < n ? load_kept(reinterpret_cast<const uint4*>(p.w) + c0 / W) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int e = 0; e < H; ++e) acc[k][e] = make_float2(0.0f, 0.0f);
  }
  const auto weights = [&](int k, float2 (&w)[H]) {
    if (packed) {
      unpack2<DT>(wr[k], w);
      if (p.w_offset != 0.0f) {
#pragma unroll
        for (int e = 0; e < H; ++e) w[e] = __fadd2_rn(w[e], make_float2(p.w_offset, p.w_offset));
      }
      return;
    }
    float f[W];
    load_weights<DT>(p.w, p.w_dt, p.w_offset, (int)(tid + k * blockDim.x) * W, n, weight_whole, f);
#pragma unroll
    for (int e = 0; e < H; ++e) w[e] = make_float2(f[2 * e], f[2 * e + 1]);
  };
  float r_next = p.rstd[blockIdx.x];
  for (int i = 0; i < mine; ++i) {
    const int64_t row = (int64_t)blockIdx.x + (int64_t)i * gridDim.x;
    const int s = i % stages;
    const float r = r_next;
    if (i + 1 < mine) r_next = p.rstd[row + gridDim.x];
    const bool arrived = mbar_wait(smem_addr(&full[s]), (i / stages) & 1);
    const char* const stage = ring + (size_t)s * stage_bytes;
    float2 dot2 = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int at = (int)(tid + k * blockDim.x) * 16;
      if (at >= row_bytes) continue;
      float2 y[H], h[H], w[H];
      unpack2<DT>(*reinterpret_cast<const uint4*>(stage + at), y);
      unpack2<DT>(*reinterpret_cast<const uint4*>(stage + row_bytes + at), h);
      weights(k, w);
#pragma unroll
      for (int e = 0; e < H; ++e) dot2 = __ffma2_rn(__fmul2_rn(y[e], w[e]), h[e], dot2);
    }
    const float part = warp_sum(dot2.x + dot2.y);
    if ((tid & 31) == 0) red[i & 1][tid >> 5] = part;
    if (!__syncthreads_and(arrived)) {  // a copy did not come: give up, when the others have come or their waits run out
      if (tid == 0) {
        record_fault(kFaultCopyTimeout);
        for (int j = i; j < min(i + stages - (i > 0 ? 1 : 0), mine); ++j) mbar_wait(smem_addr(&full[j % stages]), (j / stages) & 1);
      }
      __syncthreads();
      if (p.dw)
        for (int c = tid; c < n; c += blockDim.x) p.ws[(int64_t)blockIdx.x * n + c] = __int_as_float(0x7FC00000);
      return;
    }
    if (tid == 0 && i > 0 && i - 1 + stages < mine) request(i - 1 + stages);
    float dot = 0.0f;
    for (int q = 0; q < warps; ++q) dot += red[i & 1][q];
    // h holds xh = h r from here on; mean(g xh) = r sum(g h) / n
    const float mean = __fdiv_rn(dot * r, (float)n);
    const float2 r2 = make_float2(r, r), m2 = make_float2(-mean, -mean);
    char* const dh = reinterpret_cast<char*>(p.dh) + row * p.map.stride[3][0] * EB;
    char* const dx = reinterpret_cast<char*>(p.dx) + row * p.map.stride[4][0] * EB;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c0 = (int)(tid + k * blockDim.x) * W;
      if (c0 >= n) continue;
      float2 y[H], h[H], w[H];
      float d[W];
      unpack2<DT>(*reinterpret_cast<const uint4*>(stage + c0 * EB), y);
      unpack2<DT>(*reinterpret_cast<const uint4*>(stage + row_bytes + c0 * EB), h);
      weights(k, w);
      if (p.dsum) unpack<DT>(*reinterpret_cast<const uint4*>(stage + 2 * row_bytes + c0 * EB), d);
#pragma unroll
      for (int e = 0; e < H; ++e) {
        const float2 xh = __fmul2_rn(h[e], r2);
        acc[k][e] = __ffma2_rn(y[e], xh, acc[k][e]);
        const float2 t = __ffma2_rn(xh, m2, __fmul2_rn(y[e], w[e]));
        const float2 o = __ffma2_rn(t, r2, p.dsum ? make_float2(d[2 * e], d[2 * e + 1]) : make_float2(0.0f, 0.0f));
        d[2 * e] = o.x, d[2 * e + 1] = o.y;
      }
      *reinterpret_cast<uint4*>(dh + c0 * EB) = pack<DT>(d);
      if constexpr (DROP != DROP_NONE) {
        drop_vec<DROP, true, W>(p.drop, g, row * n + c0, d);
        *reinterpret_cast<uint4*>(dx + c0 * EB) = pack<DT>(d);
      }
    }
  }
  allow_next();
  if (!p.dw) return;
  float* const out = p.ws + (int64_t)blockIdx.x * n;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int c0 = (int)(tid + k * blockDim.x) * W;
    if (c0 >= n) continue;
#pragma unroll
    for (int q = 0; q < H; q += 2)
      *reinterpret_cast<float4*>(out + c0 + 2 * q) = make_float4(acc[k][q].x, acc[k][q].y, acc[k][q + 1].x, acc[k][q + 1].y);
  }
}

// dw[c] = sum of the groups' shares, in a fixed order: 32 columns a block, 32 threads a column (a thread a column took
// 9 us for 500 shares of 4096 columns, this takes 5). Blocks of 8 or 16 columns, for more blocks, are no faster.
__global__ void __launch_bounds__(1024) norm_grad_join_kernel(const float* ws, float* dw, int64_t n, int groups) {
  __shared__ float part[32][33];
  const int64_t c = (int64_t)blockIdx.x * 32 + threadIdx.x;
  float acc = 0.0f;
  follow();
  if (c < n) {
    const float* at = ws + (int64_t)threadIdx.y * n + c;
    const int64_t step = 32 * n;
    int k = threadIdx.y;
    for (; k + 96 < groups; k += 128, at += 4 * step) {
      float v[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = __ldcg(at + j * step);
#pragma unroll
      for (int j = 0; j < 4; ++j) acc += v[j];
    }
    float v[3];  // the last ones go out together too
#pragma unroll
    for (int j = 0; j < 3; ++j) v[j] = k + 32 * j < groups ? __ldcg(at + j * step) : 0.0f;
#pragma unroll
    for (int j = 0; j < 3; ++j) acc += v[j];
  }
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
  if (smem > 40 * 1024) {  // to the most that this library asks for, whatever the order of the calls
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 226 * 1024);
    if (e != cudaSuccess) return e;
  }
  int n = 0;
  e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, threads, smem);
  if (e != cudaSuccess) return e;
  if (cache.size() > 65536) cache.clear();
  *blocks = cache[key] = n > 0 ? n : 1;
  return cudaSuccess;
}

template <int DT, int K, int DROP, bool CUT>
cudaError_t run_norm_grad_row(const NormGradPlan& p, const RowShape& r, int whole, int64_t* groups, cudaStream_t s) {
  const auto kernel = norm_grad_row_kernel<DT, K, DROP, CUT>;
  const size_t smem = CUT ? (size_t)(p.dw ? r.ty + 1 : 1) * (p.n + p.n / kVec<DT> + 1) * 4 : 0;
  int per_sm = 1;
  const cudaError_t e = resident_blocks((const void*)kernel, r.tx * r.ty, smem, &per_sm);
  if (e != cudaSuccess) return e;
  // every group with the same number of rows, give or take one
  const int64_t most = std::min(norm_grad_partials(p.rows, p.n), (int64_t)device_sm_count() * per_sm * r.ty);
  const int64_t rows_each = (p.rows + most - 1) / most, count = (p.rows + rows_each - 1) / rows_each;
  const int64_t blocks = (count + r.ty - 1) / r.ty;
  *groups = CUT ? blocks : count;
  return launch_after(kernel, dim3((unsigned)blocks), dim3(r.tx, r.ty), smem, s, 1, p, whole, count);
}

template <int DT>
cudaError_t run_norm_grad(const NormGradPlan& p, const RowShape& r, bool cut, int whole, int64_t* groups, cudaStream_t s) {
#define HLO_CASE(KK, DD)                                                                                 \
  if (r.k == KK && p.drop.mode == DD)                                                                  \
  return cut ? run_norm_grad_row<DT, KK, DD, true>(p, r, whole, groups, s) : run_norm_grad_row<DT, KK, DD, false>(p, r, whole, groups, s)
  HLO_CASE(1, DROP_NONE);
  HLO_CASE(1, DROP_HOST);
  HLO_CASE(1, DROP_DEVICE);
  HLO_CASE(2, DROP_NONE);
  HLO_CASE(2, DROP_HOST);
  HLO_CASE(2, DROP_DEVICE);
  HLO_CASE(4, DROP_NONE);
  HLO_CASE(4, DROP_HOST);
  HLO_CASE(4, DROP_DEVICE);
  if constexpr (DT == F32) {  // 32 sums a thread, as with four vectors of 16 bits
    HLO_CASE(8, DROP_NONE);
    HLO_CASE(8, DROP_HOST);
    HLO_CASE(8, DROP_DEVICE);
  }
#undef HLO_CASE
  return cudaErrorInvalidValue;
}

template <int DT, int K, int DROP>
cudaError_t run_norm_grad_stream(const NormGradPlan& p, int threads, int stages, size_t smem, int whole, int64_t* groups, cudaStream_t s) {
  const auto kernel = threads <= 256 ? norm_grad_stream_kernel<DT, K, DROP, 256> : norm_grad_stream_kernel<DT, K, DROP, K == 4 ? 512 : 256>;
  int per_sm = 1;
  const cudaError_t e = resident_blocks((const void*)kernel, threads, smem, &per_sm);
  if (e != cudaSuccess) return e;
  const int64_t most = std::min(norm_grad_partials(p.rows, p.n), (int64_t)device_sm_count() * per_sm);
  const int64_t rows_each = (p.rows + most - 1) / most;
  *groups = (p.rows + rows_each - 1) / rows_each;
  return launch_after(kernel, dim3((unsigned)*groups), dim3(threads), smem, s, 1, p, stages, whole);
}

// The ring's shape for rows of `vectors` vectors; 0 stages: the rows do not fit.
struct RingShape {
  int k, threads, stages;
  size_t smem;
};
RingShape ring_shape(int64_t vectors, int arrays) {
  RingShape r = {};
  r.k = vectors > 512 ? 4 : vectors > 128 ? 2 : 1;
  r.threads = (int)((vectors + r.k - 1) / r.k + 31) / 32 * 32;
  const size_t stage = (size_t)vectors * 16 * arrays;
  // 768 threads an SM: 8192 x 4096 bf16 took 52 us when this was chosen (47.5 now), with 512 threads 58 us, with 256 85 us
  const int blocks = std::max(1, std::min(16, 768 / r.threads));
  const size_t room = (size_t)220 * 1024 / blocks - 1024;
  r.stages = (int)std::min<size_t>(kMaxStages, room / stage);
  if (r.stages < 2) r.stages = (int)std::min<size_t>(2, (size_t)224 * 1024 / stage);
  if (r.stages < 2 || r.threads > 512) r.stages = 0;
  r.smem = stage * r.stages;
  return r;
}

template <int DT>
cudaError_t run_norm_grad_ring(const NormGradPlan& p, const RingShape& r, int whole, int64_t* groups, cudaStream_t s) {
#define HLO_CASE(KK, DD) \
  if (r.k == KK && p.drop.mode == DD) return run_norm_grad_stream<DT, KK, DD>(p, r.threads, r.stages, r.smem, whole, groups, s)
  HLO_CASE(1, DROP_NONE);
  HLO_CASE(1, DROP_HOST);
  HLO_CASE(1, DROP_DEVICE);
  HLO_CASE(2, DROP_NONE);
  HLO_CASE(2, DROP_HOST);
  HLO_CASE(2, DROP_DEVICE);
  HLO_CASE(4, DROP_NONE);
  HLO_CASE(4, DROP_HOST);
  HLO_CASE(4, DROP_DEVICE);
#undef HLO_CASE
  return cudaErrorInvalidValue;
}

cudaError_t launch_norm_grad(const NormGradPlan& p, cudaStream_t s) {
  const int w = p.dt == F32 ? 4 : 8, eb = dt_bytes(p.dt);
  const void* const ptr[5] = {p.dy, p.h, p.dsum, p.dh, p.dx};
  const int ebs[5] = {eb, eb, eb, eb, eb};
  bool cut = false;
  const int64_t vectors = (p.n + w - 1) / w;
  const int max_k = p.dt == F32 ? 8 : 4;
  int64_t groups = norm_grad_partials(p.rows, p.n);
  if (vectors <= 512 * max_k && vectors_fit<5>(p.map, ptr, ebs, p.n, w, &cut)) {
    const RowShape r = row_shape(p.rows, vectors, max_k, 64);
    const int whole = p.w && (uintptr_t)p.w % 16 == 0;
    // the ring pays once its blocks have several rows each
    const RingShape ring = ring_shape(vectors, p.dsum ? 3 : 2);
    const bool stream = !cut && ring.stages > 0 && p.map.n <= 1 && p.rows >= 4 * device_sm_count();
    const cudaError_t e = stream ? (p.dt == F32    ? run_norm_grad_ring<F32>(p, ring, whole, &groups, s)
                                    : p.dt == BF16 ? run_norm_grad_ring<BF16>(p, ring, whole, &groups, s)
                                                   : run_norm_grad_ring<F16>(p, ring, whole, &groups, s))
                          : p.dt == F32    ? run_norm_grad<F32>(p, r, cut, whole, &groups, s)
                          : p.dt == BF16 ? run_norm_grad<BF16>(p, r, cut, whole, &groups, s)
                                         : run_norm_grad<F16>(p, r, cut, whole, &groups, s);
    if (e != cudaSuccess) return e;
  } else {
    if (p.dw) {
      const unsigned cols = (unsigned)((p.n + kAnyThreads - 1) / kAnyThreads);
      norm_grad_weight_any_kernel<<<dim3(cols, (unsigned)groups), kAnyThreads, 0, s>>>(p);
    }
    if (p.drop.mode == DROP_NONE) norm_grad_any_kernel<DROP_NONE><<<any_grid(p.rows), kAnyThreads, 0, s>>>(p);
    else if (p.drop.mode == DROP_HOST) norm_grad_any_kernel<DROP_HOST><<<any_grid(p.rows), kAnyThreads, 0, s>>>(p);
    else norm_grad_any_kernel<DROP_DEVICE><<<any_grid(p.rows), kAnyThreads, 0, s>>>(p);
  }
  if (!p.dw) return cudaGetLastError();
  return launch_after(norm_grad_join_kernel, dim3((unsigned)((p.n + 31) / 32)), dim3(32, 32), 0, s, 1, (const float*)p.ws, p.dw, p.n, (int)groups);
}

}  // namespace hlo
