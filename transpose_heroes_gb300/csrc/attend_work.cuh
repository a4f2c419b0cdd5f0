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

// Units of work of a tile: of the entries up to the last one that its last token may see.
template <int M, int N>
__device__ __forceinline__ int attend_units(const AttendPlan& p, const AttendItem& it, int tile) {
  if (p.mask) return max(1, (int)(((uint32_t)it.total + N - 1) / N));  // rows that see nothing are written all the same
  const uint32_t tokens = min((uint32_t)it.count, ((uint32_t)(tile + 1) * M - 1) / (uint32_t)p.group + 1);
  return (int)(((uint32_t)it.length + tokens + N - 1) / N);
}

template <int M>
__device__ __forceinline__ void attend_sequence(const AttendPlan& p, AttendItem& it) {
  it.length = cache_length(p.m, it.b);
  it.count = cache_count(p.m, it.b);
  it.total = (int)min((int64_t)it.length + it.count, (int64_t)p.m.capacity);
  it.tiles = (int)(((uint32_t)it.count * (uint32_t)p.group + M - 1) / M);
}

// Units of the first n tiles of a key head. Without a mask tile t sees length + (t + 1) M / group entries: where the group is a
// power of two this is a sum of floor((a + i) / r), or of an arithmetic series, and no loop over a long prompt's tiles.
template <int M, int N>
__device__ __forceinline__ int64_t attend_units_upto(const AttendPlan& p, const AttendItem& it, int n) {
  if (p.mask) return (int64_t)n * attend_units<M, N>(p, it, 0);
  const int each = M / p.group;  // tokens of a tile
  int64_t u = 0;
  if (each * p.group != M || (each & (each - 1)) != 0) {
    for (int t = 0; t < n; ++t) u += attend_units<M, N>(p, it, t);
    return u;
  }
  const int full = min(n, it.count / each);
  if (n > full) u = (int64_t)(n - full) * (((uint32_t)it.length + (uint32_t)it.count + N - 1) / N);
  const uint32_t up = (uint32_t)it.length + N - 1;
  if (each > N) return u + (int64_t)full * (up / N) + (int64_t)(each / N) * full * (full + 1) / 2;
  const uint32_t r = N / each, c = up / each;
  const auto floors = [r](uint32_t y) {  // the sum of floor(j / r) over j < y
    const uint64_t q = y / r, rest = y % r;
    return r * (q * (q - (q > 0)) / 2) + rest * q;
  };
  return u + (int64_t)(floors(c + full + 1) - floors(c + 1));
}

template <int M, int N>
__device__ __forceinline__ int64_t attend_units_of(const AttendPlan& p, int b) {
  AttendItem it;
  it.b = b;
  attend_sequence<M>(p, it);
  if (it.tiles == 1) return (int64_t)attend_units<M, N>(p, it, 0) * p.kv;
  return attend_units_upto<M, N>(p, it, it.tiles) * p.kv;
}

// a / b for a >= 0, b > 0; nearly always of 32 bits, which is several times shorter.
static __device__ __noinline__ int64_t attend_divide_long(int64_t a, int64_t b) { return a / b; }
__device__ __forceinline__ int64_t attend_divide(int64_t a, int64_t b) {
  return ((uint64_t)(a | b) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : attend_divide_long(a, b);
}

// A block's stretch: `left` units, the first of them unit `unit` of tile `it`; per: units a block.
struct AttendShare {
  AttendItem it;
  int left, per, unit;
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
  const int64_t per = max((int64_t)1, attend_divide(all + gridDim.x - 1, gridDim.x)), start = blockIdx.x * per;
  r.per = (int)per;
  r.left = (int)max((int64_t)0, min(per, all - start));
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
    if (upto - u <= start && start < upto) {
      s.b = b;
      s.at = start - (upto - u);
    }
    __syncthreads();
    if (carry > start) break;  // the same for all threads
  }
  r.it.b = s.b;
  attend_sequence<M>(p, r.it);
  int64_t off = s.at;
  r.it.tile = 0;
  if (r.it.tiles <= 1) {
    const int u = attend_units<M, N>(p, r.it, 0);
    r.it.head = (int)attend_divide(off, u);
    r.unit = (int)(off - (int64_t)r.it.head * u);
    return r;
  }
  const int64_t one = max((int64_t)1, attend_units_upto<M, N>(p, r.it, r.it.tiles));
  r.it.head = (int)attend_divide(off, one);
  off -= r.it.head * one;
  // the last tile that begins at or before `off`, and what lies before it
  int lo = 0, hi = r.it.tiles;
  int64_t before = 0;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    const int64_t upto = attend_units_upto<M, N>(p, r.it, mid);
    if (upto <= off) lo = mid, before = upto;
    else hi = mid;
  }
  r.it.tile = lo;
  r.unit = (int)(off - before);
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

// Entries that every row of the tile sees: the first ones, up to here.
template <int M>
__device__ __forceinline__ int attend_open(const AttendPlan& p, const AttendItem& it) {
  return p.mask ? it.length : min(it.total, it.length + (int)((uint32_t)it.tile * M / (uint32_t)p.group) + 1);
}

// The note for the join of a tile that begins in this block and ends in another, and a stretch's slot where it is not a whole
// tile's work. The block that notes it ends where its share does.
__device__ __forceinline__ int4 attend_note(const AttendShare& s, int units, int take, int rows) {
  return make_int4(s.it.b, s.it.head | rows << 16, s.it.tile, (int)blockIdx.x + (units - take + s.per - 1) / s.per);
}
__device__ __forceinline__ int attend_slot(bool begins) { return 2 * (int)blockIdx.x + (begins ? 1 : 0); }

// Natural logarithm of a row's sum, from the maximum m and sum l in units of a factor 2.
__device__ __forceinline__ float attend_lse(float m, float l) {
  return l > 0.0f ? fmaf(m, 0.693147180559945309f, logf(l)) : l == 0.0f ? __int_as_float(0xFF800000) : l;
}

// Where row r of a tile's rows (token r / group of the sequence, head r % group of the key head's group) goes.
struct AttendRow {
  int token, head;
};
__device__ __forceinline__ AttendRow attend_row(const AttendPlan& p, const AttendItem& it, int row) {
  const int t = (int)((uint32_t)row / (uint32_t)p.group);
  return {t, it.head * p.group + row - t * p.group};
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
