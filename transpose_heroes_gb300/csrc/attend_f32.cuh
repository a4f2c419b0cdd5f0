// Attention over a paged cache with f32 queries, over entries of f32 or f8E4M3FN: all products in f32 on the FMA pipe, since
// no matrix instruction keeps their 24 bits.
//
// As in attend_rows.cuh each of a block's four warps streams entries of its own through a private ring. A lane has DP / 32
// of the head's elements: of the queries and outputs of all MR rows in registers, of an entry from shared memory (without
// bank conflicts). The scores of 32 (entry, row) pairs are added up over the lanes at once: in five exchanges a lane gives
// away the half of its sums that the other lane is to end with, 31 in all, one a pair. Lane k MR + r then has the score of
// entry k and row r, and hands its weight to all when the values are added.
//
// Bound: HBM for 4 rows (64 sequences to 8192 entries, 2712 MB: 421 us, 95% of the copy rate); issue slots for more: 16 rows of 128
// take about 190 instructions an entry, of which 128 are FMAs (32 rows in two tiles over 16 sequences to 16384 entries: 940 us).
#pragma once
#include "attend_mma.cuh"

namespace hlo {

template <bool F8, int DP, int MR>
struct F32Shape {
  static constexpr int kRow = DP * (F8 ? 1 : 4);
  static constexpr int kKeys = F8 || DP <= 64 ? 16 : 8;
  static constexpr int kStage = 2 * kKeys * kRow;
  static constexpr int kStages = 3;
  static constexpr int kWarp = kStages * kStage > MR * (DP + 4) * 4 ? kStages * kStage : MR * (DP + 4) * 4;
  static constexpr int kPitch = DP + 4;
  static constexpr int kUnit = 4 * kKeys;
  static constexpr int kSmem = 4 * kWarp;
  static constexpr int kBlocks = kSmem <= 110 * 1024 ? 2 : 1;
};

// A lane's elements of an entry: 2 lane .. for heads of 64, else 4 lane .. of each 128.
template <bool F8, int DP>
__device__ __forceinline__ void f32_elements(const char* row, int lane, float (&v)[DP / 32]) {
#pragma unroll
  for (int g = 0; g < (DP + 127) / 128; ++g) {
    if constexpr (F8) {
      constexpr int n = DP == 64 ? 2 : 4;
      const uint32_t u = n == 2 ? *reinterpret_cast<const uint16_t*>(row + 2 * lane) : *reinterpret_cast<const uint32_t*>(row + 128 * g + 4 * lane);
#pragma unroll
      for (int k = 0; k < n; k += 2) {
        const uint32_t h = f16_of_codes(u >> (8 * k));
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
        v[4 * g + k] = f.x;
        v[4 * g + k + 1] = f.y;
      }
    } else if constexpr (DP == 64) {
      const float2 f = *reinterpret_cast<const float2*>(row + 8 * lane);
      v[0] = f.x, v[1] = f.y;
    } else {
      const float4 f = *reinterpret_cast<const float4*>(row + 512 * g + 16 * lane);
      v[4 * g] = f.x, v[4 * g + 1] = f.y, v[4 * g + 2] = f.z, v[4 * g + 3] = f.w;
    }
  }
}
template <int DP>
__device__ __forceinline__ int f32_column(int lane, int k) {
  return DP == 64 ? 2 * lane + k : 128 * (k >> 2) + 4 * lane + (k & 3);
}

template <bool F8, int DP, int MR>
__global__ void __launch_bounds__(128, F32Shape<F8, DP, MR>::kBlocks) attend_f32_kernel(const __grid_constant__ AttendPlan p, bool same_strides) {
  using S = F32Shape<F8, DP, MR>;
  constexpr int KT = S::kKeys, ROW = S::kRow, CH = ROW / 16, STAGES = S::kStages, EB = F8 ? 1 : 4, CL = DP / 32, KS = 32 / MR;
  extern __shared__ __align__(128) char ring[];
  __shared__ AttendScan scan;
  __shared__ float2 stat[4][MR];
  __shared__ uint32_t there[4][STAGES];
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  char* const mine = ring + w * S::kWarp;
  const uint32_t mine_at = attend_smem(mine);
  const float none = __int_as_float(0xFF800000);
  wait_for_last();
  AttendShare share = attend_share<MR, S::kUnit, 128>(p, scan);
  allow_next();  // every block runs from the start, so the join takes nobody's place
  int4 begun = make_int4(-1, 0, 0, 0);
  while (share.left > 0) {
    const AttendItem it = share.it;
    const int units = attend_units<MR, S::kUnit>(p, it, it.tile);
    const int take = min(share.left, units - share.unit);
    const int row0 = it.tile * MR, rows = min(MR, it.count * p.group - row0);
    const int32_t* const table = p.m.table + it.b * p.m.table_stride;
    const int first = share.unit * S::kUnit, end = min(it.total, first + take * S::kUnit);
    const int tiles = (max(0, end - first) + KT - 1) / KT, open = attend_open<MR>(p, it);
    const int n = (tiles - w + 3) / 4;
    const char* const kbase = reinterpret_cast<const char*>(p.k) + it.head * p.k_stride[2] * EB;
    const char* const vbase = reinterpret_cast<const char*>(p.v) + it.head * p.v_stride[2] * EB;
    int page = -1, place = 0;
    const auto look = [&](int i) {
      page = -1;
      const int e = first + (w + 4 * i) * KT + lane;
      if (i < n && lane < KT && e < end) page = cache_look(p.m, table, e, &place);
    };
    const auto request = [&](int i) {
      if (i < n) {
        const int s = i % STAGES;
        page = cache_page(p.m, page);
        const uint32_t given = __ballot_sync(0xffffffffu, page >= 0);
        if (lane == 0) there[w][s] = given;
        const int64_t ko = (page * p.k_stride[0] + place * p.k_stride[1]) * EB;
        const int64_t vo = same_strides ? ko : (page * p.v_stride[0] + place * p.v_stride[1]) * EB;
        const uint32_t to = mine_at + s * S::kStage;
#pragma unroll
        for (int c = 0; c < KT * CH / 32; ++c) {
          const int e = (c * 32 + lane) / CH, ch = (c * 32 + lane) % CH;
          const int64_t k = __shfl_sync(0xffffffffu, ko, e), v = same_strides ? k : __shfl_sync(0xffffffffu, vo, e);
          const bool ok = ch * 16 < p.dim * EB && (given >> e & 1);
          copy16(to + e * ROW + ch * 16, ok ? kbase + k + ch * 16 : kbase, ok);
          copy16(to + (KT + e) * ROW + ch * 16, ok ? vbase + v + ch * 16 : vbase, ok);
        }
      }
      copy_commit();
    };
    look(0);
#pragma unroll
    for (int i = 0; i < STAGES - 1; ++i) {
      request(i);
      look(i + 1);
    }
    float q[MR][CL], o[MR][CL];
#pragma unroll
    for (int r = 0; r < MR; ++r) {
      const AttendRow at = attend_row(p, it, row0 + r);
      const float* const from = reinterpret_cast<const float*>(p.q) + it.b * p.q_stride[0] + at.token * p.q_stride[1] + at.head * p.q_stride[2];
#pragma unroll
      for (int k = 0; k < CL; ++k) {
        const int c = f32_column<DP>(lane, k);
        q[r][k] = r < rows && c < p.dim ? from[c] : 0.0f;
        o[r][k] = 0.0f;
      }
    }
    const int my_row = lane % MR, my_key = lane / MR;  // of the pair whose score the lane ends with
    const int token = attend_row(p, it, row0 + my_row).token;
    float top = none, sum = 0.0f;
    bool some_cleared = false;
    for (int i = 0; i < n; ++i) {
      copy_wait<STAGES - 2>();
      __syncwarp();
      request(i + STAGES - 1);
      look(i + STAGES);
      const int s = i % STAGES, e0 = first + (w + 4 * i) * KT;
      const char* const ks = mine + s * S::kStage;
      const char* const vs = ks + KT * ROW;
      const uint32_t given = there[w][s];
      const bool hides = e0 + KT > open;
#pragma unroll 1
      for (int k0 = 0; k0 < KT; k0 += KS) {
        float z[32];
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          float v[CL];
          f32_elements<F8, DP>(ks + (k0 + k) * ROW, lane, v);
#pragma unroll
          for (int r = 0; r < MR; ++r) {
            float x = 0.0f;
#pragma unroll
            for (int c = 0; c < CL; ++c) x = fmaf(q[r][c], v[c], x);
            z[k * MR + r] = x;
          }
        }
#pragma unroll
        for (int h = 16; h >= 1; h /= 2) {
          const bool upper = lane & h;
#pragma unroll
          for (int j = 0; j < h; ++j) {
            const float a = z[j], b = z[j + h];
            z[j] = (upper ? b : a) + __shfl_xor_sync(0xffffffffu, upper ? a : b, h);
          }
        }
        const int e = k0 + my_key;
        bool sees = given >> e & 1;
        if (hides && sees) sees = my_row < rows && attend_sees(p, it, token, e0 + e);
        const float x = sees ? z[0] * p.score_scale : none;
        float most = x;
#pragma unroll
        for (int h = MR; h < 32; h *= 2) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, h));
        if (__any_sync(0xffffffffu, most > top + 8.0f)) {
          const float next = fmaxf(top, most);
          const float f = next == top ? 1.0f : exp2f(top - next);
          top = next;
          sum *= f;
#pragma unroll
          for (int r = 0; r < MR; ++r) {
            const float g = __shfl_sync(0xffffffffu, f, r);
#pragma unroll
            for (int c = 0; c < CL; ++c) o[r][c] *= g;
          }
        }
        const float weight = exp2f(x - (top == none ? 0.0f : top));
        sum += weight;
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          float v[CL];
          f32_elements<F8, DP>(vs + (k0 + k) * ROW, lane, v);
          if (hides) {
#pragma unroll
            for (int c = 0; c < CL; ++c)
              if (!(fabsf(v[c]) < __int_as_float(0x7F800000))) v[c] = 0.0f, some_cleared = true;
          }
#pragma unroll
          for (int r = 0; r < MR; ++r) {
            const float g = __shfl_sync(0xffffffffu, weight, k * MR + r);
#pragma unroll
            for (int c = 0; c < CL; ++c) o[r][c] = fmaf(g, v[c], o[r][c]);
          }
        }
      }
    }
    copy_wait<0>();
    __syncwarp();
#pragma unroll
    for (int h = MR; h < 32; h *= 2) sum += __shfl_xor_sync(0xffffffffu, sum, h);
    if (lane < MR) stat[w][lane] = make_float2(top, sum);
    float* const part = reinterpret_cast<float*>(mine);
#pragma unroll
    for (int r = 0; r < MR; ++r)
#pragma unroll
      for (int k = 0; k < CL; ++k) part[r * S::kPitch + f32_column<DP>(lane, k)] = o[r][k];
    const bool cleared = __syncthreads_or(some_cleared);
    const bool begins = share.unit == 0, whole = begins && take == units;
    const int64_t slot = attend_slot(begins);
    const int from = open <= first ? first : first + (open - first) / KT * KT;
    for (int i = tid; i < rows * DP; i += 128) {
      const int r = i / DP, c = i - r * DP;
      const float t = fmaxf(fmaxf(stat[0][r].x, stat[1][r].x), fmaxf(stat[2][r].x, stat[3][r].x));
      const float base = t == none ? 0.0f : t;
      float l = 0.0f, y = 0.0f;
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const float f = exp2f(stat[v][r].x - base);
        l = fmaf(f, stat[v][r].y, l);
        y = fmaf(f, *reinterpret_cast<const float*>(ring + v * S::kWarp + (r * S::kPitch + c) * 4), y);
      }
      const AttendRow at = attend_row(p, it, row0 + r);
      if (cleared && c < p.dim) y += cleared_values<F8>(p, it, at.token, from, end, c);
      if (!whole) {
        p.sums[(slot * MR + r) * DP + c] = y;
        if (c == 0) p.stats[slot * MR + r] = make_float2(t, l);
        continue;
      }
      if (p.lse && c == 0) p.lse[((int64_t)it.b * p.m.seq + at.token) * p.heads + at.head] = attend_lse(t, l);
      if (c < p.dim)
        reinterpret_cast<float*>(p.out)[it.b * p.out_stride[0] + at.token * p.out_stride[1] + at.head * p.out_stride[2] + c] =
            l == 0.0f ? 0.0f : y * (p.value_scale / l);
    }
    if (!whole && begins) begun = attend_note(share, units, take, rows);
    __syncthreads();
    share.left -= take;
    share.unit += take;
    if (share.left > 0 && share.unit == units) {
      share.unit = 0;
      if (!attend_next<MR>(p, share.it)) break;
    }
  }
  if (tid == 0) p.shares[blockIdx.x] = begun;
}

template <bool F8, int DP, int MR>
cudaError_t run_attend_f32(AttendPlan& p, void* ws, cudaStream_t s) {
  using S = F32Shape<F8, DP, MR>;
  const int blocks = device_sm_count() * S::kBlocks;
  attend_layout(&p, ws, blocks, MR, DP);
  bool same = true;
  for (int d = 0; d < 2; ++d) same = same && p.k_stride[d] == p.v_stride[d];
  const auto kernel = attend_f32_kernel<F8, DP, MR>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
  if (e != cudaSuccess) return e;
  e = launch_after(kernel, dim3((unsigned)blocks), dim3(128), S::kSmem, s, 1, p, same);
  return e == cudaSuccess ? launch_attend_join(p, MR, DP, blocks, s) : e;
}

// Tiles of 4, 8 or 16 rows (8 at most for heads of more than 128 elements, for the registers' sake).
template <bool F8>
cudaError_t run_attend_f32_type(AttendPlan& p, void* ws, cudaStream_t s) {
  const int64_t rows = (int64_t)p.m.seq * p.group;
#define HLO_CASE(DP, MR) return run_attend_f32<F8, DP, MR>(p, ws, s)
  if (p.dim > 128) {
    if (rows <= 4) HLO_CASE(256, 4);
    HLO_CASE(256, 8);
  }
  if (p.dim > 64) {
    if (rows <= 4) HLO_CASE(128, 4);
    if (rows <= 8) HLO_CASE(128, 8);
    HLO_CASE(128, 16);
  }
  if (rows <= 4) HLO_CASE(64, 4);
  if (rows <= 8) HLO_CASE(64, 8);
  HLO_CASE(64, 16);
#undef HLO_CASE
}

}  // namespace hlo
