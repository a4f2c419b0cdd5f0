// How the attention's work is shared among blocks, and what all its kernels have in common: which entries a row sees, and
// where its results go.
//
// The new tokens of a sequence and the `group` query heads that read one key head make count * group rows; M of them are a
// tile. A tile's work is the entries it sees, counted in units of N. All tiles' units follow one another (by sequence,
// key head, tile), and every block takes an equal stretch of them: sequences of unequal lengths, few heads or a
// single long sequence all keep every SM streaming. A stretch that is a whole tile's work is finished by its block;
// the others leave their rows' maxima, sums and unnormalised outputs in the workspace (at most two a block: slot 1 for the
// tile that the block begins and does not finish, slot 0 for one that it continues), and attend_join_kernel adds
// them up in the blocks' order.
#pragma once
#include "cache_plans.h"
#include "rows.cuh"

namespace hlo {

struct AttendItem {
  int b, head, tile;       // sequence, key head, tile of its rows
  int length, count, total;  // entries before the new tokens, new tokens, and all (those the cache has room for)
  int tiles;
};

template <int M, int N>
__device__ __forceinline__ int attend_units(const AttendPlan& p, const AttendItem& it, int tile) {
  int keys = it.total;
  if (!p.mask) keys = min(keys, it.length + min(it.count, (int)(((int64_t)(tile + 1) * M - 1) / p.group) + 1));
  return max(1, (keys + N - 1) / N);  // rows that see nothing are written all the same
}

template <int M>
__device__ __forceinline__ void attend_sequence(const AttendPlan& p, AttendItem& it) {
  it.length = cache_length(p.m, it.b);
  it.count = cache_count(p.m, it.b);
  it.total = (int)min((int64_t)it.length + it.count, (int64_t)p.m.capacity);
  it.tiles = (it.count * p.group + M - 1) / M;
}

template <int M, int N>
__device__ __forceinline__ int64_t attend_units_of(const AttendPlan& p, int b) {
  AttendItem it;
  it.b = b;
  attend_sequence<M>(p, it);
  int64_t u = 0;
  if (p.mask) u = (int64_t)it.tiles * attend_units<M, N>(p, it, 0);
  else
    for (int t = 0; t < it.tiles; ++t) u += attend_units<M, N>(p, it, t);
  return u * p.kv;
}

// A block's stretch: `left` units, the first of them unit `unit` of tile `it`.
struct AttendShare {
  AttendItem it;
  int64_t at, left, per;  // at: the first unit's number among all; per: units a block
  int unit;
};

struct AttendScan {
  int64_t warp[32];
  int64_t at;
  int b;
};

// Called by all THREADS threads of a block; every one returns the same.
template <int M, int N, int THREADS>
__device__ __forceinline__ AttendShare attend_share(const AttendPlan& p, AttendScan& s) {
  constexpr int W = THREADS / 32;
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  int64_t mine = 0, first = 0;
  for (int b = tid; b < p.m.batch; b += THREADS) {
    const int64_t u = attend_units_of<M, N>(p, b);
    if (b == tid) first = u;
    mine += u;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
  if (lane == 0) s.warp[w] = mine;
  __syncthreads();
  int64_t all = 0;
  for (int i = 0; i < W; ++i) all += s.warp[i];
  __syncthreads();
  AttendShare r;
  r.per = max((int64_t)1, (all + gridDim.x - 1) / gridDim.x);
  r.at = blockIdx.x * r.per;
  r.left = max((int64_t)0, min(r.per, all - r.at));
  r.unit = 0;
  if (r.left == 0) return r;
  if (tid == 0) s.b = 0, s.at = 0;
  int64_t carry = 0;
  for (int base = 0; base < p.m.batch; base += THREADS) {
    const int b = base + tid;
    const int64_t u = base == 0 ? first : b < p.m.batch ? attend_units_of<M, N>(p, b) : 0;
    int64_t upto = u;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const int64_t x = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += x;
    }
    if (lane == 31) s.warp[w] = upto;
    __syncthreads();
    int64_t before = carry;
    for (int i = 0; i < w; ++i) before += s.warp[i];
    upto += before;
    for (int i = 0; i < W; ++i) carry += s.warp[i];
    if (upto - u <= r.at && r.at < upto) {
      s.b = b;
      s.at = r.at - (upto - u);
    }
    __syncthreads();
    if (carry > r.at) break;  // the same for all threads
  }
  r.it.b = s.b;
  attend_sequence<M>(p, r.it);
  int64_t off = s.at;
  if (p.mask) {
    const int u = attend_units<M, N>(p, r.it, 0);
    const int64_t t = off / u;
    r.unit = (int)(off - t * u);
    r.it.head = (int)(t / max(1, r.it.tiles));
    r.it.tile = (int)(t - (int64_t)r.it.head * r.it.tiles);
  } else {
    const int64_t one = max((int64_t)1, attend_units_of<M, N>(p, r.it.b) / p.kv);
    r.it.head = (int)(off / one);
    off -= r.it.head * one;
    r.it.tile = 0;
    for (;;) {
      const int u = attend_units<M, N>(p, r.it, r.it.tile);
      if (off < u) break;
      off -= u;
      ++r.it.tile;
    }
    r.unit = (int)off;
  }
  return r;
}

// To the next tile. Only called while units are left; false where there is none all the same (lengths that somebody wrote
// meanwhile).
template <int M>
__device__ __forceinline__ bool attend_next(const AttendPlan& p, AttendItem& it) {
  if (++it.tile < it.tiles) return true;
  it.tile = 0;
  if (++it.head < p.kv) return true;
  it.head = 0;
  while (++it.b < p.m.batch) {
    attend_sequence<M>(p, it);
    if (it.tiles > 0) return true;
  }
  return false;
}

// Whether new token t of the sequence sees entry i < total.
__device__ __forceinline__ bool attend_sees(const AttendPlan& p, const AttendItem& it, int t, int i) {
  const int u = i - it.length;
  if (u < 0) return true;
  if (!p.mask) return u <= t;
  return (p.mask[it.b * p.mask_stride[0] + t * p.mask_stride[1] + (u >> 5)] >> (u & 31)) & 1;
}

// The slot of a stretch that is not a whole tile's work, and the note for the join where the tile begins in it.
__device__ __forceinline__ int attend_slot(bool begins) { return 2 * (int)blockIdx.x + (begins ? 1 : 0); }

// Natural logarithm of a row's sum, from the maximum m and sum l in units of a factor 2.
__device__ __forceinline__ float attend_lse(float m, float l) {
  return l > 0.0f ? fmaf(m, 0.693147180559945309f, logf(l)) : l == 0.0f ? __int_as_float(0xFF800000) : l;
}

// Where row r of a tile's rows (token r / group of the sequence, head r % group of the key head's group) goes.
struct AttendRow {
  int token, head;
};
__device__ __forceinline__ AttendRow attend_row(const AttendPlan& p, const AttendItem& it, int64_t row) {
  const int t = (int)(row / p.group);
  return {t, it.head * p.group + (int)(row - (int64_t)t * p.group)};
}

cudaError_t launch_attend_join(const AttendPlan& p, int m, int cols, int blocks, cudaStream_t s);

// Bytes of the workspace of `blocks` blocks whose tiles have m rows of `cols` columns; places its parts.
inline size_t attend_layout(AttendPlan* p, void* ws, int blocks, int m, int cols) {
  const auto up = [](size_t n) { return (n + 255) / 256 * 256; };
  const size_t a = up(sizeof(int4) * blocks), b = up(sizeof(float2) * 2 * blocks * m), c = sizeof(float) * 2 * (size_t)blocks * m * cols;
  if (p) {
    char* const w = static_cast<char*>(ws);
    p->shares = reinterpret_cast<int4*>(w);
    p->stats = reinterpret_cast<float2*>(w + a);
    p->sums = reinterpret_cast<float*>(w + a + b);
  }
  return a + b + c;
}

}  // namespace hlo
