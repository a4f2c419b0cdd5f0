// Attention over a paged cache for many rows a key head (prompts, large trees), on the fifth-generation tensor cores.
//
// A block has 256 rows of one key head as two tiles of 128, and streams the entries in tiles of 128 through a ring in
// shared memory; each tile is multiplied with both. Sixteen warps in four groups:
//   groups 0, 1   the softmax of tile 0 and tile 1, a row a thread: scores from tensor memory into registers, running maximum
//                 and sum, weights back into tensor memory in the scores' place, where the second product takes them from
//   group 2       brings keys and values (in the products' 128-byte swizzle), and looks through values that a mask may hide
//   group 3       one warp issues the products: while one tile's softmax runs, the other tile's products do; one brings queries
// Tensor memory: scores 128 columns and outputs DP columns for each tile. The maximum moves only where a score exceeds it
// by 2^8; then the group rescales its outputs there. No product of its tile runs then: the scores' arrival implies that the
// product before has ended, and the next one waits for the weights.
// Order of the products: S0(0) S1(0) | V0(0) S0(1) V1(0) S1(1) | ... : a tile's next scores follow its weights' product, so
// they may overwrite the weights.
//
// Entries arrive by tensor copies, one warp requesting a box of a page a lane, where pages hold whole boxes of 8 to 128 entries;
// queries too, where the group divides the tile. Other pages and strides take 16-byte copies by four warps, codes go
// through registers, where they become f16.
//
// Bound, by cycles that the groups counted at prompts of 4096 tokens (8 key heads of 128, 4 query heads each): a pair of tiles
// takes about 4000 cycles, of which its four products need 2048. A tile's softmax takes 2200 (scores and maximum 800, exponentials
// 1250, the rest the weights' way back) and its two products 1024 behind one another, so the two tiles' alternation is
// limited by one tile's chain. At the end of a stretch of tiles the results' way out costs 5500 cycles. 4 prompts: 667 us, 824
// TFLOP/s, 43% of the library's bf16 product; trees of 48 nodes (192 rows) over 16 x 16384 entries, 708 MB: 205 us, 51% of the copy rate.
// Before: one thread of a diverged warp issued the products (905 us), 16-byte copies brought everything (900), the queries came
// behind the last tile's values (789), all tiles were looked through and masked (1401).
//
// Infinite and NaN values in tiles that a mask cuts are cleared by the copying warps before the products see them, and added
// again for the rows that see them (cleared_values). Every wait is bounded: when one runs out, the block records the fault,
// stops, waits for its copies and products, frees its tensor memory and leaves its rows unwritten.
#pragma once
#include "async_copy.cuh"
#include "attend_mma.cuh"

namespace hlo {

template <int DP>
struct TileShape {
  static constexpr int kRows = 256, kKeys = 128;
  static constexpr int kPanel = 128 * 128;                // 128 rows of 64 16-bit elements
  static constexpr int kTile = kPanel * (DP / 64);        // queries of a tile, or a slot of the ring
  static constexpr int kSlots = DP == 64 ? 8 : 4;
  static constexpr int kStaging = 32 * 64;                // of a softmax warp: 64 bytes of each of its rows
  static constexpr int kSmem = (2 + kSlots) * kTile + 8 * kStaging + 1024;  // and what rounding the base up to 1024 takes
  static constexpr int kThreads = 512;
  static constexpr int kScores = 128;                     // columns; tile s: scores at 128 s, outputs at 256 + DP s
};

struct TileBarriers {
  uint64_t kv_full[8], kv_empty[8], landed[8], cleaned, q_full, q_empty, s_full[2], p_full[2], o_full[2], drained;
};

// The cache as the tensor copies see it: [pages, kv, page_size, dim], boxes of `rows` entries by 64 elements.
struct TileMaps {
  CUtensorMap k, v;
  CUtensorMap q;  // [batch, seq, heads, dim], boxes of a tile's tokens and the group's heads, where a group divides the tile
  int rows;
  int queries;    // whether q is there
};

__device__ __forceinline__ void tile_copy(uint32_t to, const CUtensorMap* map, int x, int place, int head, int page, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(to),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(place), "r"(head), "r"(page), "r"(bar)
      : "memory");
}

__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
// Whether phase `parity` has ended, without waiting.
__device__ __forceinline__ bool mbar_done(uint32_t bar, uint32_t parity) {
  uint32_t done;
  asm volatile("{ .reg .pred P; mbarrier.test_wait.parity.shared::cta.b64 P, [%1], %2; selp.u32 %0, 1, 0, P; }" : "=r"(done) : "r"(bar), "r"(parity) : "memory");
  return done != 0;
}
// Arrives when all products that the leader has issued have ended.
__device__ __forceinline__ void tile_commit(uint32_t leader, uint32_t bar) {
  asm volatile("{ .reg .pred q; setp.ne.u32 q, %1, 0; @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0]; }" ::"r"(bar),
               "r"(leader)
               : "memory");
}
__device__ __forceinline__ void tile_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tile_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// d (+)= a b, issued by the leader of a converged warp. Operands in shared memory by descriptor; a also in tensor memory.
__device__ __forceinline__ void tile_mma(uint32_t leader, uint32_t d, uint64_t a, uint64_t b, uint32_t what, bool add) {
  asm volatile(
      "{ .reg .pred p, q; setp.ne.u32 q, %5, 0; setp.ne.u32 p, %4, 0; @q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p; }" ::"r"(d), "l"(a),
      "l"(b), "r"(what), "r"((uint32_t)add), "r"(leader)
      : "memory");
}
__device__ __forceinline__ void tile_mma_weights(uint32_t leader, uint32_t d, uint32_t a, uint64_t b, uint32_t what, bool add) {
  asm volatile(
      "{ .reg .pred p, q; setp.ne.u32 q, %5, 0; setp.ne.u32 p, %4, 0; @q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p; }" ::"r"(d), "r"(a),
      "l"(b), "r"(what), "r"((uint32_t)add), "r"(leader)
      : "memory");
}

// A matrix in panels of 64 elements (128 bytes, swizzled) by rows: groups of 8 rows 1024 bytes apart, panels `panel` apart
// (used where the rows are the products' inner dimension).
__device__ __forceinline__ uint64_t tile_descriptor(uint32_t at, uint32_t panel) {
  return (uint64_t)((at >> 4) & 0x3FFF) | (uint64_t)((panel >> 4) & 0x3FFF) << 16 | (uint64_t)(1024 >> 4) << 32 | (uint64_t)1 << 46 |
         (uint64_t)2 << 61;
}

__device__ __forceinline__ void tile_load32(uint32_t (&r)[32], uint32_t at) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, "
      "%20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]),
        "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]),
        "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]),
        "=r"(r[31])
      : "r"(at));
}
__device__ __forceinline__ void tile_load16(uint32_t (&r)[16], uint32_t at) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]),
        "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(at));
}
__device__ __forceinline__ void tile_store16(uint32_t at, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(at), "r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]),
      "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tile_wait_loads() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tile_wait_stores() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Which of the 32 entries from `e` on a row's token sees (bit i: entry e + i), by the mask alone.
__device__ __forceinline__ uint32_t tile_sees(const AttendPlan& p, const AttendItem& it, int token, int e) {
  const int u = e - it.length;  // the first one among the new tokens
  if (!p.mask) {
    const int n = token + 1 - u;  // it sees the first n
    return n >= 32 ? 0xFFFFFFFFu : n <= 0 ? 0u : (1u << n) - 1;
  }
  if (u <= -32) return 0xFFFFFFFFu;
  const uint32_t* const row = p.mask + it.b * p.mask_stride[0] + token * p.mask_stride[1];
  const int words = (p.m.seq + 31) >> 5;
  if (u < 0) return (row[0] << -u) | ((1u << -u) - 1);
  const int k = u >> 5;
  const uint32_t lo = k < words ? row[k] : 0u, hi = k + 1 < words ? row[k + 1] : 0u;
  return __funnelshift_r(lo, hi, u & 31);
}

template <int DT, bool F8, int DP, bool TMA>
__global__ void __launch_bounds__(512, 1) attend_tile_kernel(const __grid_constant__ AttendPlan p, const __grid_constant__ TileMaps maps, bool same_strides,
                                                             bool q_vectors, bool out_vectors) {
  using S = TileShape<DP>;
  constexpr bool BF = DT == BF16 && !F8;  // the products' type
  constexpr int SLOTS = S::kSlots, CH = DP / 8;  // 16-byte chunks of a row
  constexpr int kCleared = TMA ? 32 : S::kKeys;  // entries that are looked through at once
  extern __shared__ char raw[];
  __shared__ __align__(8) TileBarriers bars;
  __shared__ AttendScan scan;
  __shared__ uint32_t tmem_at;
  __shared__ __align__(16) uint32_t there[8][4];  // there: which of a tile's entries exist
  __shared__ float row_unit[2][S::kRows];    // a row's scores in units of a factor 2 (bf16 queries over codes)
  __shared__ int cleared[4];                 // the item whose values were cleared, by the item's number mod 4
  __shared__ volatile int dead;
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  char* const base = raw + ((1024 - (attend_smem(raw) & 1023)) & 1023);
  const uint32_t q_at = attend_smem(base), ring_at = q_at + 2 * S::kTile;
  const auto bar = [&](const uint64_t& b) { return smem_addr(&b); };
  if (tid == 0) {
    for (int i = 0; i < SLOTS; ++i) {
      mbar_init(bar(bars.kv_full[i]), TMA ? 1 : 128);
      mbar_init(bar(bars.kv_empty[i]), 1);
      mbar_init(bar(bars.landed[i]), 1);
    }
    mbar_init(bar(bars.cleaned), 96);
    mbar_init(bar(bars.q_full), TMA ? maps.queries ? 1 : 96 : 128);
    mbar_init(bar(bars.q_empty), 1);
    for (int s = 0; s < 2; ++s) {
      mbar_init(bar(bars.s_full[s]), 1);
      mbar_init(bar(bars.p_full[s]), 4);
      mbar_init(bar(bars.o_full[s]), 1);
    }
    mbar_init(bar(bars.drained), 1);
    fence_mbar_init();
    dead = 0;
  }
  if (tid < 4) cleared[tid] = -1;
  wait_for_last();
  if (w == 12) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(attend_smem(&tmem_at)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    tile_fence_before();
  }
  AttendShare share = attend_share<S::kRows, S::kKeys, S::kThreads>(p, scan);
  __syncthreads();
  tile_fence_after();
  const uint32_t tmem = 0;  // all 512 columns: they begin at column 0
  int4 begun = make_int4(-1, 0, 0, 0);
  int item = 0;
  uint32_t tile0 = 0;  // tiles of entries before this stretch's
  // Waits for a phase; false when the wait ran out (the other groups' waits then run out too).
  const auto wait = [&](const uint64_t& b, uint32_t parity) {
    if (mbar_wait(bar(b), parity & 1)) return true;
    dead = 1;
    record_fault(kFaultCopyTimeout);
    return false;
  };
  // The same for a whole warp.
  const auto wait_all = [&](const uint64_t& b, uint32_t parity) { return __all_sync(0xffffffffu, wait(b, parity)); };
  // What a stretch of a tile is to every group.
  struct Part {
    int first, end, tiles, rows, units, take, open, row0;
  };
  const auto part_of = [&](const AttendShare& s) {
    Part a;
    a.units = attend_units<S::kRows, S::kKeys>(p, s.it, s.it.tile);
    a.take = min(s.left, a.units - s.unit);
    a.row0 = s.it.tile * S::kRows;
    a.rows = min(S::kRows, s.it.count * p.group - a.row0);
    a.first = s.unit * S::kKeys;
    a.open = attend_open<S::kRows>(p, s.it);
    a.end = min(s.it.total, a.first + a.take * S::kKeys);
    a.tiles = (max(0, a.end - a.first) + S::kKeys - 1) / S::kKeys;
    return a;
  };
  const auto advance = [&](AttendShare& s, const Part& a) {
    s.left -= a.take;
    s.unit += a.take;
    ++item;
    tile0 += a.tiles;
    if (s.left > 0 && s.unit == a.units) {
      s.unit = 0;
      if (!attend_next<S::kRows>(p, s.it)) s.left = 0;
    }
  };

  if (w < 8) {
    // ---- the softmax ----------------------------------------------------------------------------------------
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(F8 ? 160 : 168));
    const int s = w >> 2, r = tid & 127;
    const uint32_t lanes = (uint32_t)(32 * (w & 3)) << 16;
    const uint32_t scores = tmem + lanes + S::kScores * s, outs = tmem + lanes + 256 + DP * s;
    uint32_t seen_scores = 0, seen_outs = 0;  // phases
    while (share.left > 0) {
      const Part a = part_of(share);
      const AttendItem& it = share.it;
      const bool live = a.rows > 128 * s;
      if (live) {
        const int row = 128 * s + r;
        const bool mine = row < a.rows;
        const AttendRow at = attend_row(p, it, a.row0 + row);
        float unit = p.score_scale, top = __int_as_float(0xFF800000), sum = 0.0f;
        for (int j = 0; j < a.tiles; ++j) {
          if (!wait_all(bars.s_full[s], seen_scores)) goto done;
          ++seen_scores;
          tile_fence_after();
          if (DT == BF16 && F8 && j == 0) unit = row_unit[item & 1][row];
          const int e0 = a.first + j * S::kKeys;
          const uint4 given = *reinterpret_cast<const uint4*>(there[(tile0 + j) & 7]);
          const bool hides = e0 + S::kKeys > a.open, cut = hides || (given.x & given.y & given.z & given.w) != 0xFFFFFFFFu;
          uint32_t x[4][32];
          float m[4];
          tile_load32(x[0], scores);
#pragma unroll
          for (int c = 0; c < 4; ++c) {  // a quarter's maximum while the next one comes
            tile_wait_loads();
            if (c < 3) tile_load32(x[c + 1], scores + 32 * (c + 1));
            if (cut) {
              uint32_t see = c == 0 ? given.x : c == 1 ? given.y : c == 2 ? given.z : given.w;
              if (hides && mine) see &= tile_sees(p, it, at.token, e0 + 32 * c);
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (!(see >> i & 1)) x[c][i] = 0xFF800000u;
            }
            float u = __uint_as_float(x[c][0]), v = __uint_as_float(x[c][1]);
#pragma unroll
            for (int i = 2; i < 32; i += 2) {
              u = fmaxf(u, __uint_as_float(x[c][i]));
              v = fmaxf(v, __uint_as_float(x[c][i + 1]));
            }
            m[c] = fmaxf(u, v);
          }
          const float most = fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3])) * unit;
          if (__any_sync(0xffffffffu, most > top + 8.0f)) {
            const float next = fmaxf(top, most);
            const float f = next == top ? 1.0f : exp2_fast(top - next);
            top = next;
            sum *= f;
            if (j > 0) {
#pragma unroll
              for (int c = 0; c < DP; c += 16) {
                uint32_t o[16];
                tile_load16(o, outs + c);
                tile_wait_loads();
#pragma unroll
                for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                tile_store16(outs + c, o);
              }
            }
          }
          const float low = top == __int_as_float(0xFF800000) ? 0.0f : -top;
          float2 total[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t weights[16];
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
              const float2 y = __ffma2_rn(make_float2(__uint_as_float(x[c][i]), __uint_as_float(x[c][i + 1])), make_float2(unit, unit),
                                          make_float2(low, low));
              const float2 e = make_float2(exp2_fast(y.x), exp2_fast(y.y));
              total[(i >> 1) & 1] = __fadd2_rn(total[(i >> 1) & 1], e);
              weights[i / 2] = pack_pair<BF>(e.x, e.y);
            }
            tile_store16(scores + 16 * c, weights);
          }
          sum += (total[0].x + total[0].y) + (total[1].x + total[1].y);
          tile_wait_stores();
          tile_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(bars.p_full[s]));
        }
        if (a.tiles > 0) {
          if (!wait_all(bars.o_full[s], seen_outs)) goto done;
          ++seen_outs;
          tile_fence_after();
        }
        const bool begins = share.unit == 0, whole = begins && a.take == a.units;
        const int64_t slot = attend_slot(begins) * (int64_t)S::kRows + row;
        const bool again = a.tiles > 0 && cleared[item & 3] == item;
        const int from = a.open <= a.first ? a.first : a.first + (a.open - a.first) / kCleared * kCleared;
        const float f = sum == 0.0f ? 0.0f : p.value_scale / sum;  // rows that saw nothing have outputs of 0
        if (mine && whole && p.lse) p.lse[((int64_t)it.b * p.m.seq + at.token) * p.heads + at.head] = attend_lse(top, sum);
        if (mine && !whole) p.stats[slot] = make_float2(top, sum);
        // 64 bytes of each row at a time (32 elements of out, or 16 sums) through shared memory, so that a warp's stores fill whole
        // sectors
        char* const staging = base + (2 + SLOTS) * S::kTile + w * S::kStaging;
        const auto staged = [&](int row, int c) { return reinterpret_cast<uint4*>(staging + row * 64 + (c ^ ((row >> 1) & 3)) * 16); };
        const uint32_t given = __ballot_sync(0xffffffffu, mine);
        char* const to = whole ? reinterpret_cast<char*>(reinterpret_cast<uint16_t*>(p.out) + it.b * p.out_stride[0] + at.token * p.out_stride[1] +
                                                         at.head * p.out_stride[2])
                               : reinterpret_cast<char*>(p.sums + slot * DP);
        const int step = whole ? 32 : 16, columns = whole ? p.dim : DP, piece = lane & 3;
        char* at_other[4];
        bool stores[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int other = 8 * i + (lane >> 2);
          at_other[i] = reinterpret_cast<char*>(__shfl_sync(0xffffffffu, (unsigned long long)to, other)) + 16 * piece;
          stores[i] = given >> other & 1;
        }
#pragma unroll 1
        for (int c = 0; c < DP; c += step) {
          uint32_t h[16];
          if (a.tiles == 0) {
#pragma unroll
            for (int i = 0; i < 16; ++i) h[i] = 0;
          } else if (whole) {
            uint32_t o[32];
            tile_load32(o, outs + c);
            tile_wait_loads();
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float2 y = __fmul2_rn(make_float2(__uint_as_float(o[2 * i]), __uint_as_float(o[2 * i + 1])), make_float2(f, f));
              h[i] = pack_pair<DT == BF16>(y.x, y.y);
            }
          } else {
            tile_load16(h, outs + c);
            tile_wait_loads();
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) *staged(lane, i) = make_uint4(h[4 * i], h[4 * i + 1], h[4 * i + 2], h[4 * i + 3]);
          if (again && mine) {  // scaling does not change what is infinite or NaN
#pragma unroll 1
            for (int i = 0; i < step; ++i) {
              if (c + i >= p.dim) break;
              const float v = cleared_values<F8>(p, it, at.token, from, a.end, c + i);
              if (v == 0.0f) continue;
              void* const element = reinterpret_cast<char*>(staged(lane, whole ? i >> 3 : i >> 2)) + (whole ? 2 * (i & 7) : 4 * (i & 3));
              if (whole) store_from_f32(element, DT, 0, load_plain(element, DT, 0) + v);
              else *reinterpret_cast<float*>(element) += v;
            }
          }
          __syncwarp();
          const bool column = c + piece * (step / 4) < columns;
          if (out_vectors || !whole) {
            uint4 z[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) z[i] = *staged(8 * i + (lane >> 2), piece);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              if (column && stores[i]) *reinterpret_cast<uint4*>(at_other[i]) = z[i];
              at_other[i] += 64;
            }
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
#pragma unroll 1
              for (int k = 0; k < 8; ++k)
                if (column && stores[i]) reinterpret_cast<uint16_t*>(at_other[i])[k] = reinterpret_cast<const uint16_t*>(staged(8 * i + (lane >> 2), piece))[k];
              at_other[i] += 64;
            }
          }
          __syncwarp();
        }
        if (begins && !whole) begun = attend_note(share, a.units, a.take, a.rows);
        tile_fence_before();
      }
      advance(share, a);
    }
  } else if (w < 12) {
    // ---- the copies -----------------------------------------------------------------------------------------
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(F8 ? 120 : 104));
    constexpr int EB = F8 ? 1 : 2;
    const int pw = w - 8, ch = lane % CH;
    uint32_t slots = 0;                  // slots filled so far
    uint32_t q_loads = 0;
    // chunk `c` of row r of a tile of 128 rows
    const auto chunk_at = [&](uint32_t tile, int r, int c) { return tile + (c >> 3) * S::kPanel + r * 128 + ((c & 7) ^ (r & 7)) * 16; };
    // 8 elements of a query row that cannot be copied as they are
    const auto put_query = [&](uint32_t to, const uint16_t* from, bool ok, int row) {
      uint32_t v[4] = {0, 0, 0, 0};
      if (ok && q_vectors) {
        const uint4 u = *reinterpret_cast<const uint4*>(from);
        v[0] = u.x, v[1] = u.y, v[2] = u.z, v[3] = u.w;
      } else if (ok) {
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = (uint32_t)from[2 * k] | (uint32_t)from[2 * k + 1] << 16;
      }
      if constexpr (DT == BF16 && F8) {  // as in attend_rows_kernel: a power of two takes the row's greatest element to 2^14
        float most = 0.0f;
#pragma unroll
        for (int k = 0; k < 4; ++k) most = fmaxf(most, fmaxf(fabsf(__uint_as_float(v[k] << 16)), fabsf(__uint_as_float(v[k] & 0xFFFF0000u))));
#pragma unroll
        for (int x = 1; x < CH; x *= 2) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, x));
        const int ex = max((int)(__float_as_uint(most) >> 23) - 127, -100);
        const float up = __uint_as_float((uint32_t)(127 + 14 - ex) << 23);
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = pack_pair<false>(__uint_as_float(v[k] << 16) * up, __uint_as_float(v[k] & 0xFFFF0000u) * up);
        if (ch == 0) row_unit[item & 1][row] = p.score_scale * __uint_as_float((uint32_t)(127 - 14 + ex) << 23);
      }
      *reinterpret_cast<uint4*>(base + (to - q_at)) = make_uint4(v[0], v[1], v[2], v[3]);
    };
    // requests 32 rows of the queries: rows 32 k ..
    const auto put_queries = [&](const Part& a, const AttendItem& it, int k) {
      const int mine = 32 * k + lane;
      const AttendRow at = attend_row(p, it, a.row0 + mine);
      const int64_t off = mine < a.rows ? it.b * p.q_stride[0] + at.token * p.q_stride[1] + at.head * p.q_stride[2] : -1;
      const uint32_t tile = q_at + (k >> 2) * S::kTile;
      const bool plain = !(DT == BF16 && F8) && q_vectors;
#pragma unroll 8
      for (int i = 0; i < CH; ++i) {
        const int e = i * (32 / CH) + lane / CH, r = 32 * (k & 3) + e;
        const int64_t o = __shfl_sync(0xffffffffu, off, e);
        const uint16_t* const from = reinterpret_cast<const uint16_t*>(p.q) + (o < 0 ? 0 : o + 8 * ch);
        const bool ok = o >= 0 && 8 * ch < p.dim;
        const uint32_t to = chunk_at(tile, r, ch);
        if (plain) copy16(to, ok ? (const void*)from : p.q, ok);
        else put_query(to, from, ok, 32 * k + e);
      }
    };
    if constexpr (TMA) {
      if (w == 8) {
        // one warp requests the tiles, a box of entries a lane
        const int boxes = S::kKeys / maps.rows;
        uint32_t turns = 0, through = 0;  // a bit a slot: phases of `landed`; whether the last copy went to `landed`
        while (share.left > 0) {
          const Part a = part_of(share);
          const AttendItem& it = share.it;
          const int32_t* const table = p.m.table + it.b * p.m.table_stride;
          int page = -1, place = 0;
          const auto look = [&](int j) {
            page = -1;
            const int e = a.first + j * S::kKeys + lane * maps.rows;
            if (lane < boxes && e < a.end) page = cache_look(p.m, table, e, &place);
          };
          if (a.tiles > 0) look(0);
          for (int j = 0; j < a.tiles; ++j) {
            const int pg = cache_page(p.m, page), pl = place;
            look(j + 1);
            uint32_t given[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int e = 32 * k + lane;
              given[k] = __ballot_sync(0xffffffffu, __shfl_sync(0xffffffffu, pg, e / maps.rows) >= 0 && a.first + j * S::kKeys + e < a.end);
            }
#pragma unroll
            for (int side = 0; side < 2; ++side) {
              const int slot = slots % SLOTS;
              if (slots >= SLOTS && !wait_all(bars.kv_empty[slot], slots / SLOTS - 1)) goto gone;
              ++slots;
              // values that some row may not see are looked through first
              const bool look_through = side && a.first + (j + 1) * S::kKeys > a.open;
              if (look_through) turns ^= 1u << slot;
              through = (through & ~(1u << slot)) | (uint32_t)look_through << slot;
              const uint32_t b = look_through ? bar(bars.landed[slot]) : bar(bars.kv_full[slot]);
              if (lane == 0) {
                if (side == 0) {
#pragma unroll
                  for (int k = 0; k < 4; ++k) there[(tile0 + j) & 7][k] = given[k];
                }
                mbar_arrive_expect_tx(b, S::kTile);
              }
              __syncwarp();
              if (lane < boxes) {  // a page that is not there lies behind the last one: zeros
                const uint32_t to = ring_at + slot * S::kTile + lane * maps.rows * 128;
#pragma unroll
                for (int c = 0; c < DP / 64; ++c)
                  tile_copy(to + c * S::kPanel, side ? &maps.v : &maps.k, 64 * c, pl, it.head, pg < 0 ? (int)p.m.pages : pg, b);
              }
            }
          }
          advance(share, a);
        }
      gone:
        if (dead) {  // given up: the copies on their way still have to come
          for (uint32_t k = 0; k < min(slots, (uint32_t)SLOTS); ++k)
            mbar_wait((through >> k & 1) ? bar(bars.landed[k]) : bar(bars.kv_full[k]), (through >> k & 1) ? (turns >> k & 1) ^ 1 : (slots - 1 - k) / SLOTS & 1);
        }
      } else {
        // the others bring the queries, and look through values
        uint32_t turns = 0, joins = 0;  // phases of `landed`, a bit a slot, and of `cleaned`
        while (share.left > 0) {
          const Part a = part_of(share);
          if (a.tiles > 0) {
            if (!maps.queries) {
              if (q_loads > 0 && !wait_all(bars.q_empty, q_loads - 1)) goto done;
              ++q_loads;
              for (int k = w - 9; k < (a.rows > 128 ? 8 : 4); k += 3) put_queries(a, share.it, k);
              copy_commit();
              copy_wait<0>();
              fence_proxy_async();
              mbar_arrive(bar(bars.q_full));
            }
            for (int j = max(0, (a.open - a.first) / S::kKeys); j < a.tiles; ++j) {
              const int slot = (slots + 2 * j + 1) % SLOTS;
              if (!wait_all(bars.landed[slot], turns >> slot)) goto done;
              turns ^= 1u << slot;
              const int given = min(S::kKeys, a.end - (a.first + j * S::kKeys));  // entries behind them are other sequences', or nobody's
              bool any = false;
              // 32 rows a warp, from those on that some row of the queries may not see
              const int block0 = max(0, (a.open - a.first) - j * S::kKeys) / 32;
              for (int k = block0 + w - 9; k < 4; k += 3) {
                char* const rows = base + (ring_at - q_at) + slot * S::kTile + (ch >> 3) * S::kPanel + k * 4096 + (lane / CH) * 128;
                const int left = given - 32 * k - lane / CH;
                constexpr int step = 32 / CH;
                uint32_t bad = 0;
#pragma unroll
                for (int i = 0; i < CH; ++i) {
                  const uint4 v = *reinterpret_cast<const uint4*>(rows + i * step * 128 + ((ch & 7) ^ ((i * step + lane / CH) & 7)) * 16);
                  bad |= wants_clearing<false, BF>(v) || i * step >= left;
                }
                if (bad) {
#pragma unroll 1
                  for (int i = 0; i < CH; ++i) {
                    uint4* const at = reinterpret_cast<uint4*>(rows + i * step * 128 + ((ch & 7) ^ ((i * step + lane / CH) & 7)) * 16);
                    if (i * step >= left) *at = make_uint4(0, 0, 0, 0);
                    else any |= clear_vector<false, BF>(at);
                  }
                }
              }
              if (any) cleared[item & 3] = item;
              fence_proxy_async();
              mbar_arrive(bar(bars.cleaned));
              if (w == 9) {
                if (!wait_all(bars.cleaned, joins)) goto done;
                if (lane == 0) mbar_arrive(bar(bars.kv_full[slot]));
              }
              ++joins;
            }
            slots += 2 * a.tiles;
          }
          advance(share, a);
        }
      }
    } else {
    // copies in flight: the barriers of the last two groups, and whether a group's values have to be looked through
    uint32_t pending[2] = {0, 0}, look_through[2] = {0, 0};
    int look_item[2] = {0, 0};
    const bool one_page = p.dim == DP && p.m.page_size % 32 == 0;  // the 32 entries of a warp lie in one page, `step` bytes apart
    const int64_t step[2] = {p.k_stride[1] * EB, p.v_stride[1] * EB};
    const auto land = [&](int k) {  // group k has come
      if (!pending[k]) return;
      if (look_through[k]) {
        bool any = false;
#pragma unroll 1
        for (int i = 0; i < CH; ++i) {
          const int r = 32 * pw + i * (32 / CH) + lane / CH;
          any |= clear_vector<false, BF>(reinterpret_cast<uint4*>(base + (chunk_at(look_through[k], r, ch) - q_at)));
        }
        if (any) cleared[look_item[k] & 3] = look_item[k];
      }
      fence_proxy_async();
      mbar_arrive(pending[k]);
      pending[k] = 0;
    };
    const auto sent = [&](uint32_t b, uint32_t look, int number) {  // a group's copies have been requested
      copy_commit();
      if (pending[0]) {
        copy_wait<2>();
        land(0);
      }
      pending[0] = pending[1];
      look_through[0] = look_through[1];
      look_item[0] = look_item[1];
      pending[1] = b;
      look_through[1] = look;
      look_item[1] = number;
    };
    const auto flush = [&] {
      copy_wait<0>();
      land(0);
      land(1);
    };
    while (share.left > 0) {
      const Part a = part_of(share);
      const AttendItem& it = share.it;
      if (a.tiles > 0) {
        const int32_t* const table = p.m.table + it.b * p.m.table_stride;
        int page = -1, place = 0;
        const auto look = [&](int j) {
          page = -1;
          const int e = a.first + j * S::kKeys + 32 * pw + lane;
          if (e < a.end) page = cache_look(p.m, table, e, &place);
        };
        look(0);
        // the queries, whose place the last stretch's products leave late: behind the first keys
        const auto queries = [&] {
          if (q_loads > 0) {
            if (!__all_sync(0xffffffffu, mbar_done(bar(bars.q_empty), (q_loads - 1) & 1))) flush();
            if (!wait_all(bars.q_empty, q_loads - 1)) return false;
          }
          ++q_loads;
          for (int k = pw; k < (a.rows > 128 ? 8 : 4); k += 4) put_queries(a, share.it, k);
          sent(bar(bars.q_full), 0, item);
          return true;
        };
        // keys and values
        const char* const kbase = reinterpret_cast<const char*>(p.k) + it.head * p.k_stride[2] * EB;
        const char* const vbase = reinterpret_cast<const char*>(p.v) + it.head * p.v_stride[2] * EB;
        if constexpr (F8) {
          // 16 codes become two chunks of f16 on their way through registers: while a tile's keys are converted its values are
          // coming, and then the next tile's keys
          constexpr int CC = DP / 16;
          const int cc = lane % CC;
          const bool column = 16 * cc < p.dim;
          uint32_t given = 0;
          int64_t ko = 0, vo = 0;
          const auto resolve = [&](int j) {
            page = cache_page(p.m, page);
            given = __ballot_sync(0xffffffffu, page >= 0);
            ko = page * p.k_stride[0] + place * p.k_stride[1];
            vo = same_strides ? ko : page * p.v_stride[0] + place * p.v_stride[1];
            look(j + 1);
          };
          const auto fetch = [&](uint4 (&v)[CC], const char* from, int64_t off) {
#pragma unroll
            for (int i = 0; i < CC; ++i) {
              const int e = i * (32 / CC) + lane / CC;
              const int64_t o = __shfl_sync(0xffffffffu, off, e);
              v[i] = column && (given >> e & 1) ? *reinterpret_cast<const uint4*>(from + o + cc * 16) : make_uint4(0, 0, 0, 0);
            }
          };
          const auto put = [&](const uint4 (&v)[CC], bool look_through) {
            const int slot = slots % SLOTS;
            if (slots >= SLOTS && !wait_all(bars.kv_empty[slot], slots / SLOTS - 1)) return false;
            ++slots;
            const uint32_t tile = ring_at + slot * S::kTile;
            bool any = false;
#pragma unroll
            for (int i = 0; i < CC; ++i) {
              const int r = 32 * pw + i * (32 / CC) + lane / CC;
              uint32_t u[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
              if (look_through && wants_clearing<true, false>(v[i])) {
#pragma unroll
                for (int k = 0; k < 4; ++k) any |= clear_word<true, false>(u[k]);
              }
#pragma unroll
              for (int k = 0; k < 2; ++k)
                *reinterpret_cast<uint4*>(base + (chunk_at(tile, r, 2 * cc + k) - q_at)) =
                    make_uint4(f16_of_codes(u[2 * k]), f16_of_codes(u[2 * k] >> 16), f16_of_codes(u[2 * k + 1]), f16_of_codes(u[2 * k + 1] >> 16));
            }
            if (any) cleared[item & 3] = item;
            fence_proxy_async();
            mbar_arrive(bar(bars.kv_full[slot]));
            return true;
          };
          uint4 keys[CC], values[CC];
          resolve(0);
          fetch(keys, kbase, ko);
          fetch(values, vbase, vo);
          for (int j = 0; j < a.tiles; ++j) {
            if (lane == 0) there[(tile0 + j) & 7][pw] = given;
            if (!put(keys, false)) goto done;
            if (j == 0) {
              if (!queries()) goto done;
              flush();
            }
            const bool more = j + 1 < a.tiles;
            if (more) {
              resolve(j + 1);
              fetch(keys, kbase, ko);
            }
            if (!put(values, a.first + (j + 1) * S::kKeys > a.open)) goto done;
            if (more) fetch(values, vbase, vo);
          }
        } else {
        for (int j = 0; j < a.tiles; ++j) {
          page = cache_page(p.m, page);
          const uint32_t given = __ballot_sync(0xffffffffu, page >= 0);
          if (lane == 0) there[(tile0 + j) & 7][pw] = given;
          int64_t off[2];
          off[0] = (page * p.k_stride[0] + place * p.k_stride[1]) * EB;
          off[1] = same_strides ? off[0] : (page * p.v_stride[0] + place * p.v_stride[1]) * EB;
          look(j + 1);
          const bool hides = a.first + (j + 1) * S::kKeys > a.open;
#pragma unroll
          for (int side = 0; side < 2; ++side) {
            if (j == 0 && side == 1 && !queries()) goto done;
            const int slot = slots % SLOTS;
            if (slots >= SLOTS) {
              // what is on its way is announced before the warp waits: the products may need it to free the slot
              if (!__all_sync(0xffffffffu, mbar_done(bar(bars.kv_empty[slot]), (slots / SLOTS - 1) & 1))) flush();
              if (!wait_all(bars.kv_empty[slot], slots / SLOTS - 1)) goto done;
            }
            ++slots;
            const uint32_t tile = ring_at + slot * S::kTile;
            const char* const from = side ? vbase : kbase;
            {
              // row e = i (32 / CH) + lane / CH of the warp's 32: its place in shared memory repeats every CH / 4 steps, but for the step
              const bool column = 8 * ch < p.dim;
              uint32_t to[CH / 4];
#pragma unroll
              for (int i = 0; i < CH / 4; ++i) to[i] = chunk_at(tile, 32 * pw + i * (32 / CH) + lane / CH, ch);
              if (one_page && given == 0xFFFFFFFFu && column) {
                const char* at = from + __shfl_sync(0xffffffffu, off[side], 0) + step[side] * (lane / CH) + ch * 16;
#pragma unroll
                for (int i = 0; i < CH; ++i) {
                  copy16(to[i % (CH / 4)] + (i / (CH / 4)) * 1024, at, true);
                  at += step[side] * (32 / CH);
                }
              } else {
#pragma unroll
                for (int i = 0; i < CH; ++i) {
                  const int e = i * (32 / CH) + lane / CH;
                  const int64_t o = __shfl_sync(0xffffffffu, off[side], e);
                  const bool ok = column && (given >> e & 1);
                  copy16(to[i % (CH / 4)] + (i / (CH / 4)) * 1024, ok ? from + o + ch * 16 : from, ok);
                }
              }
              sent(bar(bars.kv_full[slot]), side && hides ? tile : 0, item);
            }
          }
        }
        }
      }
      advance(share, a);
    }
    flush();
    }
  } else {
    // ---- the products ---------------------------------------------------------------------------------------
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    if (w == 12) {  // one thread issues, but the warp stays together: descriptors are then the same for all of it
      constexpr uint32_t type = BF ? 1 : 0;
      constexpr uint32_t common = 1u << 4 | type << 7 | type << 10 | (128u >> 4) << 24;
      constexpr uint32_t score_what = common | (uint32_t)(S::kKeys >> 3) << 17, out_what = common | 1u << 16 | (uint32_t)(DP >> 3) << 17;
      // descriptors of addresses further on: the address' field, in units of 16 bytes, grows (it has room for all of shared memory)
      const uint64_t q_d = tile_descriptor(q_at, S::kPanel), ring_d = tile_descriptor(ring_at, S::kPanel);
      uint32_t leader;
      asm volatile("{ .reg .pred q; elect.sync _|q, 0xFFFFFFFF; selp.u32 %0, 1, 0, q; }" : "=r"(leader));
      uint32_t slots = 0, q_loads = 0, weights[2] = {0, 0};
      bool ok = true;
      while (ok && share.left > 0) {
        const Part a = part_of(share);
        const int live = a.rows > 128 ? 2 : 1;
        if (a.tiles > 0) {
          ok = wait_all(bars.q_full, q_loads++);
          // the product of the weights with the values of slot number v, of which the first tile's begins the sum
          const auto second = [&](int s, uint32_t v, bool add) {
            ok = wait_all(bars.p_full[s], weights[s]++) && wait_all(bars.kv_full[v % SLOTS], v / SLOTS);
            if (!ok) return;
            tile_fence_after();
            const uint64_t values = ring_d + (v % SLOTS) * (S::kTile >> 4);
#pragma unroll
            for (int k = 0; k < S::kKeys / 16; ++k)
              tile_mma_weights(leader, tmem + 256 + DP * s, tmem + S::kScores * s + 8 * k, values + k * (2048 >> 4), out_what, add || k > 0);
          };
          for (int j = 0; ok && j < a.tiles; ++j) {
            const uint32_t k0 = slots + 2 * j;
            ok = wait_all(bars.kv_full[k0 % SLOTS], k0 / SLOTS);
            for (int s = 0; ok && s < live; ++s) {
              if (j > 0) {
                second(s, k0 - 1, j > 1);
                if (ok && s == live - 1) tile_commit(leader, bar(bars.kv_empty[(k0 - 1) % SLOTS]));
              }
              if (!ok) break;
              tile_fence_after();
              const uint64_t queries = q_d + s * (S::kTile >> 4), keys = ring_d + (k0 % SLOTS) * (S::kTile >> 4);
#pragma unroll
              for (int k = 0; k < DP / 16; ++k) {
                constexpr int panel = S::kPanel >> 4;
                tile_mma(leader, tmem + S::kScores * s, queries + (k >> 2) * panel + (k & 3) * 2, keys + (k >> 2) * panel + (k & 3) * 2, score_what, k > 0);
              }
              tile_commit(leader, bar(bars.s_full[s]));
            }
            if (!ok) break;
            tile_commit(leader, bar(bars.kv_empty[k0 % SLOTS]));
            if (j == a.tiles - 1) tile_commit(leader, bar(bars.q_empty));
          }
          slots += 2 * a.tiles;
          for (int s = 0; ok && s < live; ++s) {
            second(s, slots - 1, a.tiles > 1);
            if (ok) tile_commit(leader, bar(bars.o_full[s]));
          }
          if (ok) tile_commit(leader, bar(bars.kv_empty[(slots - 1) % SLOTS]));
        }
        advance(share, a);
      }
      // every product that was issued has ended before the memory is given back
      tile_commit(leader, bar(bars.drained));
      mbar_wait(bar(bars.drained), 0);
    }
    if (TMA && w == 13 && maps.queries) {  // the queries, as soon as the last stretch's scores have been computed
      uint32_t q_loads = 0;
      while (share.left > 0) {
        const Part a = part_of(share);
        if (a.tiles > 0) {
          if (q_loads > 0 && !wait_all(bars.q_empty, q_loads - 1)) break;
          ++q_loads;
          const int halves = a.rows > 128 ? 2 : 1, tokens = 128 / p.group, b = share.it.b;
          if (lane == 0) {
            mbar_arrive_expect_tx(bar(bars.q_full), halves * S::kTile);
            for (int h = 0; h < halves; ++h)
              for (int c = 0; c < DP / 64; ++c)
                tile_copy(q_at + h * S::kTile + c * S::kPanel, &maps.q, 64 * c, share.it.head * p.group, (2 * share.it.tile + h) * tokens, b, bar(bars.q_full));
          }
        }
        advance(share, a);
      }
      if (dead && q_loads > 0) mbar_wait(bar(bars.q_full), (q_loads - 1) & 1);  // given up: the copies on their way still have to come
    }
    __syncwarp();
  }
done:
  copy_wait<0>();
  if (tid == 0) p.shares[blockIdx.x] = begun;
  tile_fence_before();
  __syncthreads();
  tile_fence_after();
  if (w == 12) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
  allow_next();
}

// The maps of a cache whose pages hold whole boxes of 8 to 128 entries (a power of two, so that a tile of 128 is some of
// them); false where there are none, for strides that no map takes or other pages: 16-byte copies bring those.
template <int DT>
bool tile_maps(const AttendPlan& p, TileMaps* maps) {
  maps->rows = 1;
  while (maps->rows < 128 && p.m.page_size % (2 * maps->rows) == 0) maps->rows *= 2;
  const auto encode = tensor_map_encoder();
  if (maps->rows < 8 || !encode || p.m.pages < 1) return false;
  // an array [n2, n1, n0, dim] with those strides (0 where a dimension is 1), in boxes [1, b1, b0, 64]
  const auto encoded = [&](CUtensorMap* map, const void* at, int64_t n0, int64_t s0, int64_t n1, int64_t s1, int64_t n2, int64_t s2, int b0, int b1) {
    const cuuint64_t dims[4] = {(cuuint64_t)p.dim, (cuuint64_t)n0, (cuuint64_t)n1, (cuuint64_t)n2};
    const int64_t steps[3] = {s0, s1, s2};
    cuuint64_t strides[3];
    for (int d = 0; d < 3; ++d) {
      if (steps[d] == 0 && dims[d + 1] > 1) return false;
      if (steps[d] >= (int64_t)1 << 39) return false;
      strides[d] = steps[d] == 0 ? 16 : (cuuint64_t)steps[d] * 2;
    }
    const cuuint32_t box[4] = {64, (cuuint32_t)b0, (cuuint32_t)b1, 1}, ones[4] = {1, 1, 1, 1};
    return encode(map, DT == BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4, const_cast<void*>(at), dims, strides, box,
                  ones, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  };
  for (int side = 0; side < 2; ++side) {
    const int64_t* const s = side ? p.v_stride : p.k_stride;  // page, place, head
    if (!encoded(side ? &maps->v : &maps->k, side ? p.v : p.k, p.m.page_size, s[1], p.kv, s[2], p.m.pages, s[0], maps->rows, 1)) return false;
  }
  bool fits = 128 % p.group == 0 && (uintptr_t)p.q % 16 == 0;
  for (int d = 0; d < 3; ++d) fits = fits && p.q_stride[d] % 8 == 0;
  maps->queries = fits && encoded(&maps->q, p.q, p.heads, p.q_stride[2], p.m.seq, p.q_stride[1], p.m.batch, p.q_stride[0], p.group, 128 / p.group);
  return true;
}

template <int DT, bool F8, int DP, bool TMA>
cudaError_t run_attend_tile(AttendPlan& p, const TileMaps& maps, void* ws, cudaStream_t s) {
  using S = TileShape<DP>;
  const int blocks = device_sm_count();
  attend_layout(&p, ws, blocks, S::kRows, DP);
  bool same = true, q_vectors = (uintptr_t)p.q % 16 == 0, out_vectors = (uintptr_t)p.out % 16 == 0;
  for (int d = 0; d < 2; ++d) same = same && p.k_stride[d] == p.v_stride[d];
  for (int d = 0; d < 3; ++d) {
    q_vectors = q_vectors && p.q_stride[d] % 8 == 0;
    out_vectors = out_vectors && p.out_stride[d] % 8 == 0;
  }
  const auto kernel = attend_tile_kernel<DT, F8, DP, TMA>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
  if (e != cudaSuccess) return e;
  e = launch_after(kernel, dim3((unsigned)blocks), dim3(S::kThreads), S::kSmem, s, 1, p, maps, same, q_vectors, out_vectors);
  return e == cudaSuccess ? launch_attend_join(p, S::kRows, DP, blocks, s) : e;
}

template <int DT, bool F8>
cudaError_t run_attend_tile_type(AttendPlan& p, void* ws, cudaStream_t s) {
  TileMaps maps = {};
  if constexpr (!F8) {
    if (tile_maps<DT>(p, &maps))
      return p.dim <= 64 ? run_attend_tile<DT, F8, 64, true>(p, maps, ws, s) : run_attend_tile<DT, F8, 128, true>(p, maps, ws, s);
  }
  return p.dim <= 64 ? run_attend_tile<DT, F8, 64, false>(p, maps, ws, s) : run_attend_tile<DT, F8, 128, false>(p, maps, ws, s);
}

}  // namespace hlo
