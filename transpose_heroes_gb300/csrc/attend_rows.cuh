// Attention over a paged cache for few rows a key head (single tokens, small trees), on the tensor cores by mma.sync.
//
// Mathematics: the softmax's running maximum and sum. Each of a block's four warps streams entries of its own (KT at a
// time through a private ring of asynchronous copies, so no barrier stands in the loop) for all of the tile's 16 MT
// rows, and holds its own maximum m, sum l and output o; at the stretch's end the four are added up with weights
// 2^(m_w - m). m moves only where a score exceeds it by 2^8: until then the weights are at most 256, exact in f32 sums and
// no worse rounded, and o need not be rescaled.
//
// Bound: HBM. Each entry is read once and multiplied by at most 32 rows (32 flops a byte): mma.sync is enough (a
// quarter of its rate), and needs no accumulators in tensor memory, whose tiles of 128 rows would be mostly empty. bf16, 8 key
// heads of 128, 4 query heads each: 64 sequences to 8192 entries (1356 MB) 210 us, 95% of the copy rate; 32 rows (16 sequences
// to 16384, 8 new tokens, 700 MB) 133 us, 77%. Over codes the conversions bound it: 134 us for those 64 sequences' 679 MB, 198 us for
// 32 rows of 687 MB, where two warps a scheduler issue 0.3 instructions a cycle, waiting for one another's results.
//
// An 8-bit cache is converted to f16 in registers, which holds its codes exactly: ldmatrix hands a thread four neighbouring
// codes of a key, so the products run over the head's elements in an order of their own, which the queries' registers
// follow; of values, a byte permutation pairs the codes of two entries. bf16 queries become f16 after a power of two has
// brought each row's greatest element to 2^14: elements down to 2^-28 of it keep all their bits.
#pragma once
#include "attend_mma.cuh"

namespace hlo {

template <bool F8, int DP, int MT>
struct RowsShape {
  static constexpr int kRow = DP * (F8 ? 1 : 2);                 // bytes of an entry in the ring
  static constexpr int kKeys = F8 || DP <= 64 ? 32 : 16;         // of a warp's stage
  static constexpr int kStage = 2 * kKeys * kRow;                // keys, then values
  static constexpr int kStages = kStage <= 4096 ? 5 : 3;
  static constexpr int kWarp = kStages * kStage;                 // of each warp
  static constexpr int kPitch = DP + 4;                          // of the rows that the warps add up (f32)
  static constexpr int kRows = 16 * MT, kUnit = 4 * kKeys;
  static_assert(kRows * kPitch * 4 <= kWarp, "a warp's output takes the place of its ring");
  static constexpr int kQueries = MT > 1 ? kRows * (DP * 2 + 16) : 0;  // queries in shared memory: rows 16 bytes apart in the banks
  static constexpr int kSmem = 4 * kWarp + kQueries;
  static constexpr int kBlocks = kSmem <= 110 * 1024 ? 2 : 1;    // an SM
};

// Where 16-byte chunk c of entry r lies in its row: ldmatrix reads eight entries' same chunk, and they fall on different banks.
template <int ROW>
__device__ __forceinline__ int rows_chunk(int r, int c) {
  return ROW >= 128 ? c ^ (r & 7) : c ^ ((r >> 1) & 3);
}

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at)
               : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at)
               : "memory");
}
template <bool BF>
__device__ __forceinline__ void mma16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (BF)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The 16-bit elements c and c + 1 of a query row (zeros where the row or the columns are none).
__device__ __forceinline__ uint32_t query_pair(const uint16_t* row, int c, int dim, bool whole) {
  if (!row || c >= dim) return 0;
  if (whole) return *reinterpret_cast<const uint32_t*>(row + c);
  return (uint32_t)row[c] | (uint32_t)row[c + 1] << 16;
}

template <int DT, bool F8, int DP, int MT>
__global__ void __launch_bounds__(128, RowsShape<F8, DP, MT>::kBlocks)
    attend_rows_kernel(const __grid_constant__ AttendPlan p, bool same_strides, bool q_words, bool out_vectors) {
  using S = RowsShape<F8, DP, MT>;
  constexpr bool BF = DT == BF16 && !F8;  // the products' type
  constexpr int KT = S::kKeys, ROW = S::kRow, CH = ROW / 16, STAGES = S::kStages, NT = KT / 8;
  extern __shared__ __align__(128) char ring[];
  __shared__ AttendScan scan;
  __shared__ float2 stat[4][S::kRows];
  __shared__ uint32_t there[4][STAGES];  // which of a stage's entries exist
  __shared__ float row_unit[S::kRows];
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5, g = lane >> 2, quad = lane & 3;
  char* const mine = ring + w * S::kWarp;
  const uint32_t mine_at = attend_smem(mine);
  wait_for_last();
  AttendShare share = attend_share<S::kRows, S::kUnit, 128>(p, scan);
  allow_next();  // every block runs from the start, so the join takes nobody's place
  int4 begun = make_int4(-1, 0, 0, 0);
  constexpr int EB = F8 ? 1 : 2;
  while (share.left > 0) {
    const AttendItem it = share.it;
    const int units = attend_units<S::kRows, S::kUnit>(p, it, it.tile);
    const int take = min(share.left, units - share.unit);
    const int row0 = it.tile * S::kRows;
    const int rows = min(S::kRows, it.count * p.group - row0);
    const int32_t* const table = p.m.table + it.b * p.m.table_stride;
    const int first = share.unit * S::kUnit, end = min(it.total, first + take * S::kUnit);
    const int tiles = (max(0, end - first) + KT - 1) / KT, open = attend_open<S::kRows>(p, it);
    const int n = (tiles - w + 3) / 4;  // of this warp: w, w + 4, ...
    const char* const kbase = reinterpret_cast<const char*>(p.k) + it.head * p.k_stride[2] * EB;
    const char* const vbase = reinterpret_cast<const char*>(p.v) + it.head * p.v_stride[2] * EB;

    // the page and place of the lane's entry of tile i, whose copies are requested a turn later
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
        const int ch = lane % CH;
        const bool column = ch * 16 < p.dim * EB;
#pragma unroll
        for (int c = 0; c < KT * CH / 32; ++c) {
          const int e = c * (32 / CH) + lane / CH;
          const int64_t k = __shfl_sync(0xffffffffu, ko, e), v = same_strides ? k : __shfl_sync(0xffffffffu, vo, e);
          const bool ok = column && (given >> e & 1);
          const uint32_t at = to + e * ROW + rows_chunk<ROW>(e, ch) * 16;
          copy16(at, ok ? kbase + k + ch * 16 : kbase, ok);
          copy16(at + KT * ROW, ok ? vbase + v + ch * 16 : vbase, ok);
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

    // The queries, as the products' left operands: in registers for 16 rows; for 32 in shared memory, in the same order, since
    // their 64 registers are wanted for the products in flight (32 rows of 128 over codes, 687 MB: 198 us, 259 with all in registers, of which some were spilled).
    constexpr bool kept = MT == 1;
    uint32_t q[MT][kept ? DP / 16 : 1][4];
    float unit[MT][2];  // a row's scores in units of a factor 2
    int token[MT][2];
    constexpr int kPitchQ = DP * 2 + 16;
    char* const q_rows = ring + 4 * S::kWarp;
    // a row's scale over codes: 2^e <= most < 2^(e + 1), for most of at least 2^-100 (smaller rows' scores vanish all the same)
    const auto scaled = [&](uint32_t (&v)[DP / 16][2]) {
      float most = 0.0f;
#pragma unroll
      for (int c = 0; c < DP / 16; ++c)
#pragma unroll
        for (int k = 0; k < 2; ++k) most = fmaxf(most, fmaxf(fabsf(__uint_as_float(v[c][k] << 16)), fabsf(__uint_as_float(v[c][k] & 0xFFFF0000u))));
      most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 1));
      most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 2));
      const int e = max((int)(__float_as_uint(most) >> 23) - 127, -100);
      const float up = __uint_as_float((uint32_t)(127 + 14 - e) << 23);
#pragma unroll
      for (int c = 0; c < DP / 16; ++c)
#pragma unroll
        for (int k = 0; k < 2; ++k) v[c][k] = pack_pair<false>(__uint_as_float(v[c][k] << 16) * up, __uint_as_float(v[c][k] & 0xFFFF0000u) * up);
      return __uint_as_float((uint32_t)(127 - 14 + e) << 23);
    };
    const auto load_row = [&](int r, uint32_t (&v)[DP / 16][2]) {  // a lane's part of row r; what its scores are multiplied by
      const AttendRow at = attend_row(p, it, row0 + r);
      const uint16_t* const row =
          r < rows ? reinterpret_cast<const uint16_t*>(p.q) + it.b * p.q_stride[0] + at.token * p.q_stride[1] + at.head * p.q_stride[2] : nullptr;
#pragma unroll
      for (int c = 0; c < DP / 16; ++c) {
        v[c][0] = query_pair(row, 16 * c + (F8 ? 4 * quad : 2 * quad), p.dim, q_words);
        v[c][1] = query_pair(row, 16 * c + (F8 ? 4 * quad + 2 : 2 * quad + 8), p.dim, q_words);
      }
      if constexpr (DT == BF16 && F8) return p.score_scale * scaled(v);
      return p.score_scale;
    };
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h) token[m][h] = attend_row(p, it, row0 + 16 * m + g + 8 * h).token;
    if constexpr (kept) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t v[DP / 16][2];
        unit[0][h] = load_row(g + 8 * h, v);
#pragma unroll
        for (int c = 0; c < DP / 16; ++c) q[0][c][h] = v[c][0], q[0][c][h + 2] = v[c][1];
      }
    } else {  // each warp brings 4 MT rows
#pragma unroll
      for (int k = 0; k < S::kRows / 32; ++k) {
        uint32_t v[DP / 16][2];
        const int r = 8 * (w + 4 * k) + g;
        const float u = load_row(r, v);
        if (quad == 0) row_unit[r] = u;
#pragma unroll
        for (int c = 0; c < DP / 16; ++c) {
          *reinterpret_cast<uint32_t*>(q_rows + r * kPitchQ + 32 * c + 4 * quad) = v[c][0];
          *reinterpret_cast<uint32_t*>(q_rows + r * kPitchQ + 32 * c + 16 + 4 * quad) = v[c][1];
        }
      }
      __syncthreads();
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) unit[m][h] = row_unit[16 * m + g + 8 * h];
    }
    const uint32_t q_lane = attend_smem(q_rows) + ((lane & 7) + ((lane >> 3) & 1) * 8) * kPitchQ + (lane >> 4) * 16;

    float o[MT][DP / 8][4], top[MT][2], sum[MT][2];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
#pragma unroll
      for (int c = 0; c < DP / 8; ++c) o[m][c][0] = o[m][c][1] = o[m][c][2] = o[m][c][3] = 0.0f;
      top[m][0] = top[m][1] = __int_as_float(0xFF800000);
      sum[m][0] = sum[m][1] = 0.0f;
    }
    bool some_cleared = false;

    for (int i = 0; i < n; ++i) {
      copy_wait<STAGES - 2>();
      __syncwarp();
      request(i + STAGES - 1);
      look(i + STAGES);
      const int s = i % STAGES, e0 = first + (w + 4 * i) * KT;
      const uint32_t ks = mine_at + s * S::kStage, vs = ks + KT * ROW;
      const uint32_t given = there[w][s];
      const bool hides = e0 + KT > open;  // some rows may not see all of it
      float x[MT][NT][4];
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int t = 0; t < NT; ++t) x[m][t][0] = x[m][t][1] = x[m][t][2] = x[m][t][3] = 0.0f;
#pragma unroll
      for (int c = 0; c < DP / 16; ++c) {
        uint32_t b[4], a[MT][4];
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          if constexpr (kept) {
#pragma unroll
            for (int k = 0; k < 4; ++k) a[m][k] = q[m][c][k];
          } else {
            ldmatrix4(a[m], q_lane + 16 * m * kPitchQ + 32 * c);
          }
        }
        if constexpr (F8) {
          ldmatrix4(b, ks + lane * ROW + rows_chunk<ROW>(lane, c) * 16);
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            const uint32_t b0 = f16_of_codes(b[t]), b1 = f16_of_codes(b[t] >> 16);
#pragma unroll
            for (int m = 0; m < MT; ++m) mma16<BF>(x[m][t], a[m], b0, b1);
          }
        } else {
#pragma unroll
          for (int k = 0; k < KT / 16; ++k) {
            const int r = 16 * k + (lane & 7) + (lane >> 4) * 8;
            ldmatrix4(b, ks + r * ROW + rows_chunk<ROW>(r, 2 * c + ((lane >> 3) & 1)) * 16);
#pragma unroll
            for (int m = 0; m < MT; ++m) {
              mma16<BF>(x[m][2 * k], a[m], b[0], b[1]);
              mma16<BF>(x[m][2 * k + 1], a[m], b[2], b[3]);
            }
          }
        }
      }
      if (hides || given != (KT == 32 ? 0xFFFFFFFFu : 0xFFFFu)) {
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int e = 8 * t + 2 * quad + (k & 1);
              if (!(given >> e & 1) || 16 * m + g + 8 * (k >> 1) >= rows || !attend_sees(p, it, token[m][k >> 1], e0 + e))
                x[m][t][k] = __int_as_float(0xFF800000);
            }
        if (hides) {
          bool any = false;
          for (int k = lane; k < KT * CH; k += 32) any |= clear_vector<F8, DT == BF16>(reinterpret_cast<uint4*>(mine + s * S::kStage + KT * ROW) + k);
          some_cleared |= any;
          __syncwarp();
        }
      }
      float most[MT][2];
      bool moves = false;
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float y = fmaxf(x[m][0][2 * h], x[m][0][2 * h + 1]);
#pragma unroll
          for (int t = 1; t < NT; ++t) y = fmaxf(y, fmaxf(x[m][t][2 * h], x[m][t][2 * h + 1]));
          y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 1));
          y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 2));
          most[m][h] = y * unit[m][h];
          moves |= most[m][h] > top[m][h] + 8.0f;
        }
      if (__any_sync(0xffffffffu, moves)) {
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float next = fmaxf(top[m][h], most[m][h]);
            const float f = next == top[m][h] ? 1.0f : exp2_fast(top[m][h] - next);
            top[m][h] = next;
            sum[m][h] *= f;
#pragma unroll
            for (int c = 0; c < DP / 8; ++c) {
              o[m][c][2 * h] *= f;
              o[m][c][2 * h + 1] *= f;
            }
          }
      }
      uint32_t pw[MT][NT][2];  // the weights, as the second products' left operands
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float base = top[m][h] == __int_as_float(0xFF800000) ? 0.0f : top[m][h];
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            const float a = exp2_fast(fmaf(x[m][t][2 * h], unit[m][h], -base)), b = exp2_fast(fmaf(x[m][t][2 * h + 1], unit[m][h], -base));
            sum[m][h] += a + b;
            pw[m][t][h] = pack_pair<BF>(a, b);
          }
        }
#pragma unroll
      for (int k = 0; k < KT / 16; ++k) {
#pragma unroll
        for (int c = 0; c < DP / (F8 ? 32 : 16); ++c) {
          uint32_t b[4];
          const int r = 16 * k + (lane & 15);
          ldmatrix4_trans(b, vs + r * ROW + rows_chunk<ROW>(r, 2 * c + (lane >> 4)) * 16);
          if constexpr (F8) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {  // 16-byte chunk 2 c + j: its even and its odd elements
              const uint32_t u = __byte_perm(b[2 * j], 0, 0x3120), v = __byte_perm(b[2 * j + 1], 0, 0x3120);
              const uint32_t e0_ = f16_of_codes(u), e1_ = f16_of_codes(v), o0_ = f16_of_codes(u >> 16), o1_ = f16_of_codes(v >> 16);
#pragma unroll
              for (int m = 0; m < MT; ++m) {
                const uint32_t a[4] = {pw[m][2 * k][0], pw[m][2 * k][1], pw[m][2 * k + 1][0], pw[m][2 * k + 1][1]};
                mma16<BF>(o[m][4 * c + 2 * j], a, e0_, e1_);
                mma16<BF>(o[m][4 * c + 2 * j + 1], a, o0_, o1_);
              }
            }
          } else {
#pragma unroll
            for (int m = 0; m < MT; ++m) {
              const uint32_t a[4] = {pw[m][2 * k][0], pw[m][2 * k][1], pw[m][2 * k + 1][0], pw[m][2 * k + 1][1]};
              mma16<BF>(o[m][2 * c], a, b[0], b[1]);
              mma16<BF>(o[m][2 * c + 1], a, b[2], b[3]);
            }
          }
        }
      }
    }

    // the warps' outputs, in the place of their rings
    copy_wait<0>();
    __syncwarp();
    float* const part = reinterpret_cast<float*>(mine);
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = 16 * m + g + 8 * h;
        float l = sum[m][h];
        l += __shfl_xor_sync(0xffffffffu, l, 1);
        l += __shfl_xor_sync(0xffffffffu, l, 2);
        if (quad == 0) stat[w][r] = make_float2(top[m][h], l);
#pragma unroll
        for (int c = 0; c < DP / 16; ++c) {
          if constexpr (F8) {
            *reinterpret_cast<float4*>(part + r * S::kPitch + 16 * c + 4 * quad) =
                make_float4(o[m][2 * c][2 * h], o[m][2 * c + 1][2 * h], o[m][2 * c][2 * h + 1], o[m][2 * c + 1][2 * h + 1]);
          } else {
            *reinterpret_cast<float2*>(part + r * S::kPitch + 16 * c + 2 * quad) = make_float2(o[m][2 * c][2 * h], o[m][2 * c][2 * h + 1]);
            *reinterpret_cast<float2*>(part + r * S::kPitch + 16 * c + 8 + 2 * quad) = make_float2(o[m][2 * c + 1][2 * h], o[m][2 * c + 1][2 * h + 1]);
          }
        }
      }
    const bool cleared = __syncthreads_or(some_cleared);
    const bool begins = share.unit == 0, whole = begins && take == units;
    const int64_t slot = attend_slot(begins);
    for (int i = tid; i < rows * (DP / 4); i += 128) {
      const int r = i / (DP / 4), c = 4 * (i - r * (DP / 4));
      const float t = fmaxf(fmaxf(stat[0][r].x, stat[1][r].x), fmaxf(stat[2][r].x, stat[3][r].x));
      const float base = t == __int_as_float(0xFF800000) ? 0.0f : t;
      float l = 0.0f;
      float4 y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const float f = exp2_fast(stat[v][r].x - base);
        const float4 z = *reinterpret_cast<const float4*>(ring + v * S::kWarp + (r * S::kPitch + c) * 4);
        l = fmaf(f, stat[v][r].y, l);
        y = make_float4(fmaf(f, z.x, y.x), fmaf(f, z.y, y.y), fmaf(f, z.z, y.z), fmaf(f, z.w, y.w));
      }
      const AttendRow at = attend_row(p, it, row0 + r);
      if (cleared && c < p.dim) {
        const int from = open <= first ? first : first + (open - first) / KT * KT;
        y.x += cleared_values<F8>(p, it, at.token, from, end, c);
        y.y += cleared_values<F8>(p, it, at.token, from, end, c + 1);
        y.z += cleared_values<F8>(p, it, at.token, from, end, c + 2);
        y.w += cleared_values<F8>(p, it, at.token, from, end, c + 3);
      }
      if (!whole) {
        *reinterpret_cast<float4*>(p.sums + (slot * S::kRows + r) * DP + c) = y;
        if (c == 0) p.stats[slot * S::kRows + r] = make_float2(t, l);
        continue;
      }
      if (p.lse && c == 0) p.lse[((int64_t)it.b * p.m.seq + at.token) * p.heads + at.head] = attend_lse(t, l);
      if (c >= p.dim) continue;
      const float f = l == 0.0f ? 0.0f : p.value_scale / l;
      if (l == 0.0f) y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      uint16_t* const to = reinterpret_cast<uint16_t*>(p.out) + it.b * p.out_stride[0] + at.token * p.out_stride[1] + at.head * p.out_stride[2] + c;
      const uint32_t lo = pack_pair<DT == BF16>(y.x * f, y.y * f), hi = pack_pair<DT == BF16>(y.z * f, y.w * f);
      if (out_vectors) {
        *reinterpret_cast<uint2*>(to) = make_uint2(lo, hi);
      } else {
        to[0] = (uint16_t)lo;
        to[1] = (uint16_t)(lo >> 16);
        to[2] = (uint16_t)hi;
        to[3] = (uint16_t)(hi >> 16);
      }
    }
    if (!whole && begins) begun = attend_note(share, units, take, rows);
    __syncthreads();
    share.left -= take;
    share.unit += take;
    if (share.left > 0 && share.unit == units) {
      share.unit = 0;
      if (!attend_next<S::kRows>(p, share.it)) break;
    }
  }
  if (tid == 0) p.shares[blockIdx.x] = begun;
}

template <int DT, bool F8, int DP, int MT>
cudaError_t run_attend_rows(AttendPlan& p, void* ws, cudaStream_t s) {
  using S = RowsShape<F8, DP, MT>;
  const int blocks = device_sm_count() * S::kBlocks;
  attend_layout(&p, ws, blocks, S::kRows, DP);
  bool same = true, words = (uintptr_t)p.q % 4 == 0, vectors = (uintptr_t)p.out % 8 == 0;
  for (int d = 0; d < 2; ++d) same = same && p.k_stride[d] == p.v_stride[d];
  for (int d = 0; d < 3; ++d) {
    words = words && p.q_stride[d] % 2 == 0;
    vectors = vectors && p.out_stride[d] % 4 == 0;
  }
  const auto kernel = attend_rows_kernel<DT, F8, DP, MT>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
  if (e != cudaSuccess) return e;
  e = launch_after(kernel, dim3((unsigned)blocks), dim3(128), S::kSmem, s, 1, p, same, words, vectors);
  return e == cudaSuccess ? launch_attend_join(p, S::kRows, DP, blocks, s) : e;
}

// Tiles of 16 rows, or of 32 where the rows are more and 32 rows' outputs fit the registers (128 columns).
template <int DT, bool F8>
cudaError_t run_attend_rows_type(AttendPlan& p, void* ws, cudaStream_t s) {
  const bool more = (int64_t)p.m.seq * p.group > 16;
  if (p.dim <= 64) return more ? run_attend_rows<DT, F8, 64, 2>(p, ws, s) : run_attend_rows<DT, F8, 64, 1>(p, ws, s);
  if (p.dim <= 128) return more ? run_attend_rows<DT, F8, 128, 2>(p, ws, s) : run_attend_rows<DT, F8, 128, 1>(p, ws, s);
  return run_attend_rows<DT, F8, 256, 1>(p, ws, s);
}

}  // namespace hlo
