// Attention over a paged cache (hlo_cache_attention): the choice of the kernel, the kernel for any type, size and
// alignment, and the join of tiles that several blocks worked on.
#include <algorithm>

#include "attend_work.cuh"

namespace hlo {

// ---- the join --------------------------------------------------------------------------------------------------
// Block (c, y) adds up the tile that block c of the attention began and did not finish, if there is one: a row at a time,
// its four warps taking every fourth block's share, with weights 2^(m_i - max m). The shares' sums are requested before
// their weights are known. Bound: the latency of two dependent loads, of the note and of what it points to.
template <int COLS>
__global__ void __launch_bounds__(128) attend_join_kernel(const __grid_constant__ AttendPlan p, int m, int cols) {
  __shared__ float part[4][COLS * 32];
  follow();
  const int4 share = p.shares[blockIdx.x];
  if (share.x < 0) return;
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  AttendItem it;
  it.b = share.x;
  it.head = share.y & 0xFFFF;
  it.tile = share.z;
  const int row0 = it.tile * m, rows = share.y >> 16;
  const int n = share.w - (int)blockIdx.x + 1;  // blocks
  const float none = __int_as_float(0xFF800000);
  const auto slot = [&](int i) { return i == 0 ? 2 * (int64_t)blockIdx.x + 1 : 2 * ((int64_t)blockIdx.x + i); };
  for (int r = blockIdx.y; r < rows; r += gridDim.y) {
    float acc[COLS], top = none, l = 0.0f;
#pragma unroll
    for (int j = 0; j < COLS; ++j) acc[j] = 0.0f;
    for (int i0 = 0; i0 < n; i0 += 32) {  // 32 blocks at a time, each warp eight of them
      float z[8][COLS];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int i = i0 + w + 4 * k;
#pragma unroll
        for (int j = 0; j < COLS; ++j)
          z[k][j] = i < n && lane + 32 * j < cols ? p.sums[(slot(i) * m + r) * cols + lane + 32 * j] : 0.0f;
      }
      const float2 s = i0 + lane < n ? p.stats[slot(i0 + lane) * m + r] : make_float2(none, 0.0f);
      float next = s.x;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) next = fmaxf(next, __shfl_xor_sync(0xffffffffu, next, o));
      next = fmaxf(next, top);
      const float base = next == none ? 0.0f : next;
      const float f = exp2f(s.x - base), old = exp2f(top - base);
      l = fmaf(l, old, warp_sum(f * s.y));
      top = next;
#pragma unroll
      for (int j = 0; j < COLS; ++j) acc[j] *= old;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float g = __shfl_sync(0xffffffffu, f, w + 4 * k);
        if (i0 + w + 4 * k < n) {
#pragma unroll
          for (int j = 0; j < COLS; ++j) acc[j] = fmaf(g, z[k][j], acc[j]);
        }
      }
    }
#pragma unroll
    for (int j = 0; j < COLS; ++j) part[w][lane + 32 * j] = acc[j];
    __syncthreads();
    const AttendRow at = attend_row(p, it, row0 + r);
    const float f = l == 0.0f ? 0.0f : p.value_scale / l;
    const int64_t to = it.b * p.out_stride[0] + at.token * p.out_stride[1] + at.head * p.out_stride[2];
    for (int c = threadIdx.x; c < p.dim; c += 128)
      store_from_f32(p.out, p.dt, to + c, l == 0.0f ? 0.0f : (part[0][c] + part[1][c] + part[2][c] + part[3][c]) * f);
    if (p.lse && threadIdx.x == 0) p.lse[((int64_t)it.b * p.m.seq + at.token) * p.heads + at.head] = attend_lse(top, l);
    __syncthreads();
  }
}

cudaError_t launch_attend_join(const AttendPlan& p, int m, int cols, int blocks, cudaStream_t s) {
  const int rows = (int)std::min<int64_t>({(int64_t)p.m.seq * p.group, m, 32});
  const auto kernel = cols <= 64 ? attend_join_kernel<2> : cols <= 128 ? attend_join_kernel<4> : attend_join_kernel<8>;
  return launch_after(kernel, dim3((unsigned)blocks, (unsigned)rows), dim3(128), 0, s, 1, p, m, cols);
}

// ---- any type, size and alignment ----------------------------------------------------------------------------------
// Tiles of 16 rows, 32 entries at a time, in f32 in shared memory. A warp has four rows: each lane one entry's four
// products; then a thread has one or two columns of all 16 rows. Entries that do not lie on 16-byte boundaries come here. Bound: the
// latency of its loads, element by element.
constexpr int kAnyRows = 16, kAnyKeys = 32;

__device__ __forceinline__ float attend_load(const void* p, int dt, int f8, int64_t i) {
  if (!f8) return load_plain(p, dt, i);
  const __half_raw h = __nv_cvt_fp8_to_halfraw(reinterpret_cast<const uint8_t*>(p)[i], __NV_E4M3);
  return __half2float(*reinterpret_cast<const __half*>(&h));
}

__global__ void __launch_bounds__(128) attend_any_kernel(const __grid_constant__ AttendPlan p) {
  extern __shared__ __align__(16) float mem[];
  __shared__ AttendScan scan;
  __shared__ float weight[kAnyRows][kAnyKeys];
  __shared__ float decay[kAnyRows];
  __shared__ float2 stat[kAnyRows];
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int pitch = (p.dim + 3) / 4 * 4 + 4;  // whole 16-byte vectors, neighbouring rows on different banks
  float *const qs = mem, *const ks = qs + kAnyRows * pitch, *const vs = ks + kAnyKeys * pitch;
  for (int i = tid; i < (kAnyRows + 2 * kAnyKeys) * pitch; i += 128) mem[i] = 0.0f;  // the columns behind dim stay 0
  wait_for_last();
  AttendShare share = attend_share<kAnyRows, kAnyKeys, 128>(p, scan);
  allow_next();  // every block runs from the start, so the join takes nobody's place
  int4 begun = make_int4(-1, 0, 0, 0);
  while (share.left > 0) {
    const AttendItem it = share.it;
    const int units = attend_units<kAnyRows, kAnyKeys>(p, it, it.tile);
    const int take = min(share.left, units - share.unit);
    const int row0 = it.tile * kAnyRows;
    const int rows = min(kAnyRows, it.count * p.group - row0);
    const int32_t* const table = p.m.table + it.b * p.m.table_stride;
    __syncthreads();
    for (int i = tid; i < kAnyRows * p.dim; i += 128) {
      const int r = i / p.dim, c = i - r * p.dim;
      float q = 0.0f;
      if (r < rows) {
        const AttendRow at = attend_row(p, it, row0 + r);
        q = load_plain(p.q, p.dt, it.b * p.q_stride[0] + at.token * p.q_stride[1] + at.head * p.q_stride[2] + c);
      }
      qs[r * pitch + c] = q;
    }
    float acc[2][kAnyRows], top[4], sum[4];
#pragma unroll
    for (int r = 0; r < kAnyRows; ++r) acc[0][r] = acc[1][r] = 0.0f;
#pragma unroll
    for (int r = 0; r < 4; ++r) top[r] = __int_as_float(0xFF800000), sum[r] = 0.0f;
    for (int u = share.unit; u < share.unit + take; ++u) {
      const int key0 = u * kAnyKeys, keys = min(kAnyKeys, it.total - key0);
      __syncthreads();  // the last entries have been read
      int page = -1, place = 0;
      if (lane < keys) cache_place(p.m, table, key0 + lane, &page, &place);
      for (int i = w; i < kAnyKeys; i += 4) {
        const int pg = __shfl_sync(0xffffffffu, page, i), pl = __shfl_sync(0xffffffffu, place, i);
        const int64_t ko = pg * p.k_stride[0] + pl * p.k_stride[1] + it.head * p.k_stride[2];
        const int64_t vo = pg * p.v_stride[0] + pl * p.v_stride[1] + it.head * p.v_stride[2];
        for (int c = lane; c < p.dim; c += 32) {
          ks[i * pitch + c] = pg < 0 ? 0.0f : attend_load(p.k, p.dt, p.f8, ko + c);
          vs[i * pitch + c] = pg < 0 ? 0.0f : attend_load(p.v, p.dt, p.f8, vo + c);
        }
      }
      __syncthreads();
      float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
      for (int c = 0; c < p.dim; c += 4) {
        const float4 k = *reinterpret_cast<const float4*>(ks + lane * pitch + c);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float4 q = *reinterpret_cast<const float4*>(qs + (4 * w + r) * pitch + c);
          s[r] = fmaf(q.x, k.x, fmaf(q.y, k.y, fmaf(q.z, k.z, fmaf(q.w, k.w, s[r]))));
        }
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = row0 + 4 * w + r;
        const bool seen = page >= 0 && 4 * w + r < rows && attend_sees(p, it, (int)((uint32_t)row / (uint32_t)p.group), key0 + lane);
        const float x = seen ? s[r] * p.score_scale : __int_as_float(0xFF800000);
        float most = x;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
        most = fmaxf(most, top[r]);
        const float base = most == __int_as_float(0xFF800000) ? 0.0f : most;
        const float e = seen ? exp2f(x - base) : 0.0f;
        const float d = exp2f(top[r] - base);
        sum[r] = fmaf(sum[r], d, warp_sum(e));
        top[r] = most;
        weight[4 * w + r][lane] = e;
        if (lane == 0) decay[4 * w + r] = d;
      }
      __syncthreads();
      // entries that some row does not see must not reach it, whatever they hold: their weight there is exactly 0
      const bool mixed = key0 + kAnyKeys > attend_open<kAnyRows>(p, it);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int c = tid + 128 * j;
        if (c >= p.dim) break;
#pragma unroll
        for (int r = 0; r < kAnyRows; ++r) acc[j][r] *= decay[r];
        for (int i = 0; i < kAnyKeys; ++i) {
          const float v = vs[i * pitch + c];
          if (mixed && !(fabsf(v) < __int_as_float(0x7F800000))) {
#pragma unroll
            for (int r = 0; r < kAnyRows; ++r)
              if (weight[r][i] != 0.0f) acc[j][r] = fmaf(weight[r][i], v, acc[j][r]);
          } else {
#pragma unroll
            for (int r = 0; r < kAnyRows; ++r) acc[j][r] = fmaf(weight[r][i], v, acc[j][r]);
          }
        }
      }
    }
    if (lane == 0) {
#pragma unroll
      for (int r = 0; r < 4; ++r) stat[4 * w + r] = make_float2(top[r], sum[r]);
    }
    __syncthreads();
    const bool begins = share.unit == 0, whole = begins && take == units;
    if (whole) {
      if (p.lse && tid < rows) {
        const AttendRow at = attend_row(p, it, row0 + tid);
        p.lse[((int64_t)it.b * p.m.seq + at.token) * p.heads + at.head] = attend_lse(stat[tid].x, stat[tid].y);
      }
    } else {
      const int64_t slot = attend_slot(begins);
      if (tid < kAnyRows) p.stats[slot * kAnyRows + tid] = stat[tid];
      if (begins) begun = attend_note(share, units, take, rows);
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int c = tid + 128 * j;
      if (c >= p.dim) break;
#pragma unroll
      for (int r = 0; r < kAnyRows; ++r) {
        if (r >= rows) continue;
        if (whole) {
          const AttendRow at = attend_row(p, it, row0 + r);
          const float l = stat[r].y;
          store_from_f32(p.out, p.dt, it.b * p.out_stride[0] + at.token * p.out_stride[1] + at.head * p.out_stride[2] + c,
                         l == 0.0f ? 0.0f : acc[j][r] * (p.value_scale / l));
        } else {
          p.sums[(attend_slot(begins) * (int64_t)kAnyRows + r) * p.dim + c] = acc[j][r];
        }
      }
    }
    share.left -= take;
    share.unit += take;
    if (share.left > 0 && share.unit == units) {
      share.unit = 0;
      if (!attend_next<kAnyRows>(p, share.it)) break;
    }
  }
  if (tid == 0) p.shares[blockIdx.x] = begun;
}

static size_t any_smem(int64_t dim) { return (kAnyRows + 2 * kAnyKeys) * ((dim + 3) / 4 * 4 + 4) * sizeof(float); }
static int any_blocks(int64_t dim) { return device_sm_count() * (int)std::min<size_t>(4, 200 * 1024 / (any_smem(dim) + 4096)); }

static cudaError_t run_any(AttendPlan& p, void* ws, cudaStream_t s) {
  const int blocks = any_blocks(p.dim);
  attend_layout(&p, ws, blocks, kAnyRows, p.dim);
  const size_t smem = any_smem(p.dim);
  if (smem > 40 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(attend_any_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 100 * 1024);
    if (e != cudaSuccess) return e;
  }
  const cudaError_t e = launch_after(attend_any_kernel, dim3((unsigned)blocks), dim3(128), smem, s, 1, p);
  return e == cudaSuccess ? launch_attend_join(p, kAnyRows, p.dim, blocks, s) : e;
}

// Whether entries can be copied 16 bytes at a time.
static bool aligned_entries(const AttendPlan& p) {
  const int64_t eb = p.f8 ? 1 : dt_bytes(p.dt);
  uintptr_t bits = (uintptr_t)p.k | (uintptr_t)p.v | (uintptr_t)(p.dim * eb);
  for (int d = 0; d < 3; ++d) bits |= (uintptr_t)(p.k_stride[d] * eb) | (uintptr_t)(p.v_stride[d] * eb);
  return bits % 16 == 0;
}

static int padded_columns(int64_t dim) { return dim <= 64 ? 64 : dim <= 128 ? 128 : 256; }

// Tiles of 256 rows on the fifth-generation tensor cores; heads of more than 128 elements have no place in tensor memory there.
// Codes have to be converted on their way: up to 128 rows it costs less to read them again for each 32 rows (32 sequences
// to 16384 entries of 8 key heads: 64 rows 372 us, in one tile 767; 96 rows 492, in one tile 793). bf16: 32 rows 133, 64 rows 163.
static bool many_rows(int64_t rows, int64_t dim, bool f8) { return rows > (f8 ? 128 : 32) && dim <= 128; }

size_t attend_workspace(int64_t batch, int64_t seq, int64_t heads, int64_t kv, int64_t dim) {
  const size_t any = attend_layout(nullptr, nullptr, any_blocks(dim), kAnyRows, (int)dim);
  const int64_t rows = seq * (heads / kv);
  if (many_rows(rows, dim, false)) return std::max(any, attend_layout(nullptr, nullptr, device_sm_count(), 256, padded_columns(dim)));
  return std::max(any, attend_layout(nullptr, nullptr, 2 * device_sm_count(), rows > 16 && dim <= 128 ? 32 : 16, padded_columns(dim)));
}

cudaError_t launch_attend(AttendPlan p, void* ws, cudaStream_t s) {
  if (p.m.pages == 0) {  // no page is there: copies of nothing get an address that is one
    p.k = p.v = ws;
    for (int d = 0; d < 3; ++d) p.k_stride[d] = p.v_stride[d] = 0;
  }
  if (!aligned_entries(p)) return run_any(p, ws, s);
  if (p.dt == F32) return p.f8 ? launch_attend_f32_f8(p, ws, s) : launch_attend_f32(p, ws, s);
  if (many_rows((int64_t)p.m.seq * p.group, p.dim, p.f8)) {
    if (p.dt == BF16) return p.f8 ? launch_attend_tile_bf16_f8(p, ws, s) : launch_attend_tile_bf16(p, ws, s);
    return p.f8 ? launch_attend_tile_f16_f8(p, ws, s) : launch_attend_tile_f16(p, ws, s);
  }
  if (p.dt == BF16) return p.f8 ? launch_attend_rows_bf16_f8(p, ws, s) : launch_attend_rows_bf16(p, ws, s);
  return p.f8 ? launch_attend_rows_f16_f8(p, ws, s) : launch_attend_rows_f16(p, ws, s);
}

}  // namespace hlo
