// The acceptance of a drafted branch (hlo_tree_accept): the walk down the tree by the greedy tokens, and the move of the
// accepted entries of every layer to the places behind the sequence's old end.
#include <algorithm>

#include "cache_plans.h"
#include "rows.cuh"

namespace hlo {

struct Move {
  int from_page, from_place, to_page, to_place;
};

// Block (x, y) walks sequence x's tree for itself (a few hundred cycles, less than a second launch) and moves the y-th
// share of its columns: accesses of W bytes at one place of one head's entry, in K or V of one layer. All nodes
// look at once for the parent that would choose them (the lowest child wins), so that the walk is a chase through shared
// memory. A thread moves its column's entries in the path's order, eight loads before their eight stores: entry i goes to
// a place that no later entry comes from (path[j] >= j > i), so nothing is overwritten before it is read.
// Bound: the latency of a chain of dependent loads (parent, pick, page, entry): 16 nodes and 16 layers' 3 entries 3.3 us in a
// captured graph; 64 sequences, 34 MB moved, 9.9 us, half of the copy rate.
template <typename W>
__global__ void __launch_bounds__(256) accept_kernel(const __grid_constant__ AcceptPlan p, int columns, int per_block) {
  extern __shared__ int nodes[];  // [seq] the child that each node chooses, [seq] the path, then the moves
  __shared__ int walked;
  const int n = p.m.seq, b = blockIdx.x, tid = threadIdx.x;
  int *const child = nodes, *const path = nodes + n;
  Move* const moves = reinterpret_cast<Move*>(nodes + 2 * n + (2 * n) % 4);
  for (int c = tid; c < n; c += 256) child[c] = INT_MAX;
  follow();
  __syncthreads();
  const int count = cache_count(p.m, b);
  const int32_t* const tokens = p.tokens + b * p.tokens_stride[0];
  const int32_t* const parents = p.parents + b * p.parents_stride[0];
  const int32_t* const picks = p.picks + b * p.picks_stride[0];
  for (int c = tid + 1; c < count; c += 256) {
    const int up = parents[c * p.parents_stride[1]];
    if (up < 0 || up >= c) continue;
    const int pick = picks[up * p.picks_stride[1]];
    if (pick >= 0 && pick == tokens[c * p.tokens_stride[1]]) atomicMin(child + up, c);
  }
  __syncthreads();
  if (tid == 0) {
    int k = 0;
    if (count > 0)
      for (int c = 0; c != INT_MAX; c = child[c]) path[k++] = c;  // children come after their parents: at most n steps
    walked = k;
  }
  __syncthreads();
  const int k = walked;
  if (blockIdx.y == 0) {
    for (int i = tid; i < n; i += 256) p.path[b * p.path_stride[0] + i * p.path_stride[1]] = i < k ? path[i] : -1;
    if (tid == 0) {
      p.accepted[b] = k;
      p.next[b] = k > 0 ? picks[path[k - 1] * p.picks_stride[1]] : -1;
    }
  }
  if (!p.cache[0]) return;
  const int32_t* const row = p.m.table + b * p.m.table_stride;
  const int length = cache_length(p.m, b);
  for (int i = tid; i < k; i += 256) {
    Move v = {-1, 0, -1, 0};
    const int64_t from = (int64_t)length + path[i];
    if (path[i] > i && from < p.m.capacity) {
      cache_place(p.m, row, (int)from, &v.from_page, &v.from_place);
      cache_place(p.m, row, length + i, &v.to_page, &v.to_place);
    }
    if (v.to_page < 0) v.from_page = -1;
    moves[i] = v;
  }
  __syncthreads();
  const int pieces = (int)(p.row_bytes / sizeof(W));
  const int end = min(columns, (int)(blockIdx.y + 1) * per_block);
  for (int j = blockIdx.y * per_block + tid; j < end; j += 256) {
    int rest = j / pieces;
    const int piece = j - rest * pieces;
    const int head = rest % p.kv;
    rest /= p.kv;
    const int side = rest & 1, layer = rest >> 1;
    const int64_t* const s = p.cache_stride[side];  // in bytes
    char* const base = static_cast<char*>(p.cache[side]) + layer * s[0] + head * s[3] + (int64_t)piece * sizeof(W);
    for (int i0 = 1; i0 < k; i0 += 8) {
      W got[8];
#pragma unroll
      for (int u = 0; u < 8; ++u)
        if (i0 + u < k && moves[i0 + u].from_page >= 0)
          got[u] = *reinterpret_cast<const W*>(base + moves[i0 + u].from_page * s[1] + moves[i0 + u].from_place * s[2]);
#pragma unroll
      for (int u = 0; u < 8; ++u)
        if (i0 + u < k && moves[i0 + u].from_page >= 0)
          *reinterpret_cast<W*>(base + moves[i0 + u].to_page * s[1] + moves[i0 + u].to_place * s[2]) = got[u];
    }
  }
}

template <typename W>
cudaError_t run_accept(const AcceptPlan& p, cudaStream_t s) {
  const int64_t columns = p.cache[0] ? (int64_t)p.layers * 2 * p.kv * (p.row_bytes / (int64_t)sizeof(W)) : 0;
  if (columns > INT32_MAX / 2) return cudaErrorInvalidValue;
  // a column a thread, unless the blocks' repeated walks would outweigh it: eight blocks an SM are enough
  const int64_t want = std::max<int64_t>(1, (columns + 255) / 256);
  const int64_t most = std::max<int64_t>(1, (int64_t)device_sm_count() * 8 / p.m.batch);
  const int gy = (int)std::min<int64_t>({want, most, 65535});
  const int per = (int)(((columns + gy - 1) / gy + 255) / 256 * 256);
  const size_t smem = (size_t)p.m.seq * (2 * sizeof(int) + sizeof(Move)) + 16;
  if (smem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(accept_kernel<W>, cudaFuncAttributeMaxDynamicSharedMemorySize, 100 * 1024);
    if (e != cudaSuccess) return e;
  }
  return launch_after(accept_kernel<W>, dim3((unsigned)p.m.batch, (unsigned)gy), dim3(256), smem, s, 1, p, (int)columns, per);
}

cudaError_t launch_accept(const AcceptPlan& p, cudaStream_t s) {
  switch (p.width) {
    case 16: return run_accept<uint4>(p, s);
    case 8: return run_accept<uint2>(p, s);
    case 4: return run_accept<uint32_t>(p, s);
    case 2: return run_accept<uint16_t>(p, s);
    default: return run_accept<uint8_t>(p, s);
  }
}

}  // namespace hlo
