// Plans of the paged cache's operators (k_cache_append.cu, k_attend*.cu, k_tree_accept.cu): plain data passed to the
// kernels by value, and their launchers.
#pragma once
#include "layer_plans.h"

namespace hlo {

// Which pages belong to which sequence.
struct CacheMap {
  const int32_t* table;
  int64_t table_stride;    // of a sequence's row
  const int32_t* lengths;
  const int32_t* counts;   // or NULL: seq new tokens each
  int64_t pages;
  int page_size, page_shift;  // page_shift: log2(page_size), or -1
  int max_pages, capacity;    // capacity = max_pages * page_size < 2^31
  int batch, seq;
};

struct AppendPlan {
  CacheMap m;
  const void* in[3];       // q (or NULL), k, v
  int64_t in_stride[3][3]; // batch, token, head
  void* q_out;
  int64_t q_stride[3];
  void* cache[2];          // k, v
  int64_t cache_stride[2][3];  // page, place, head
  int heads, kv, dim, pairs;
  int dt, f8, interleaved;
  const int32_t* pos;      // or NULL: the entry's number
  int64_t pos_stride[2];
  const uint64_t* turns;
  float scale;
  float code_scale[2], code_inv[2];  // f8: a code stands for code * code_scale; code_inv = RN(1 / code_scale)
};
cudaError_t launch_append(const AppendPlan& p, cudaStream_t s);

struct AttendPlan {
  CacheMap m;
  const void *q, *k, *v;
  void* out;
  float* lse;              // or NULL; [batch, seq, heads]
  int64_t q_stride[3], out_stride[3];  // batch, token, head
  int64_t k_stride[3], v_stride[3];    // page, place, head
  const uint32_t* mask;    // or NULL: causal
  int64_t mask_stride[2];  // batch, token
  int heads, kv, group, dim;
  int dt, f8;              // of q and out; whether the cache holds f8
  float score_scale;       // scale * k_scale * log2(e): scores in units of a factor 2
  float value_scale;       // v_scale
  // a tile's rows are (token, head of the group) pairs, the group's heads of a token side by side; see attend_work.cuh
  int4* shares;            // workspace: of each block
  float2* stats;           // 2 a block: each row's maximum and sum
  float* sums;             // 2 a block: each row's unnormalised output
};
cudaError_t launch_attend(AttendPlan p, void* workspace, cudaStream_t s);
// f32 queries; entries on 16-byte boundaries.
cudaError_t launch_attend_f32(AttendPlan& p, void* workspace, cudaStream_t s);
cudaError_t launch_attend_f32_f8(AttendPlan& p, void* workspace, cudaStream_t s);
// Few rows a key head, by the types of the queries and of the cache; entries on 16-byte boundaries.
cudaError_t launch_attend_rows_bf16(AttendPlan& p, void* workspace, cudaStream_t s);
cudaError_t launch_attend_rows_bf16_f8(AttendPlan& p, void* workspace, cudaStream_t s);
cudaError_t launch_attend_rows_f16(AttendPlan& p, void* workspace, cudaStream_t s);
cudaError_t launch_attend_rows_f16_f8(AttendPlan& p, void* workspace, cudaStream_t s);
// Many rows a key head; heads of at most 128 elements.
cudaError_t launch_attend_tile_bf16(AttendPlan& p, void* workspace, cudaStream_t s);
cudaError_t launch_attend_tile_bf16_f8(AttendPlan& p, void* workspace, cudaStream_t s);
cudaError_t launch_attend_tile_f16(AttendPlan& p, void* workspace, cudaStream_t s);
cudaError_t launch_attend_tile_f16_f8(AttendPlan& p, void* workspace, cudaStream_t s);
size_t attend_workspace(int64_t batch, int64_t seq, int64_t heads, int64_t kv, int64_t dim);

struct AcceptPlan {
  CacheMap m;              // seq and counts also without a cache
  const int32_t *tokens, *parents, *picks;
  int64_t tokens_stride[2], parents_stride[2], picks_stride[2];
  int32_t* path;
  int64_t path_stride[2];
  int32_t *accepted, *next;
  void* cache[2];          // NULL: no cache
  int64_t cache_stride[2][4];  // layer, page, place, head
  int layers, kv;
  int64_t row_bytes;       // of a head's entry
  int width;               // bytes of an access: divides row_bytes, the strides and the addresses
};
cudaError_t launch_accept(const AcceptPlan& p, cudaStream_t s);

#ifdef __CUDACC__
// The sequence's lengths as they are used.
__device__ __forceinline__ int cache_length(const CacheMap& m, int b) { return min(max(m.lengths[b], 0), m.capacity); }
__device__ __forceinline__ int cache_count(const CacheMap& m, int b) { return m.counts ? min(max(m.counts[b], 0), m.seq) : m.seq; }

// Page and place of entry `slot` (0 <= slot < 2^31) of a sequence whose table row is `row`. The page as the table has it, or -1
// behind the table's end: cache_page() tells whether it is there, and a load that nothing looks at yet is not waited for.
__device__ __forceinline__ int cache_look(const CacheMap& m, const int32_t* row, int slot, int* place) {
  const int at = m.page_shift >= 0 ? slot >> m.page_shift : (int)((uint32_t)slot / (uint32_t)m.page_size);
  *place = slot - at * m.page_size;
  return at < m.max_pages ? row[at] : -1;
}
__device__ __forceinline__ int cache_page(const CacheMap& m, int page) { return (uint32_t)page < (uint32_t)m.pages ? page : -1; }
__device__ __forceinline__ void cache_place(const CacheMap& m, const int32_t* row, int slot, int* page, int* place) {
  *page = cache_page(m, cache_look(m, row, slot, place));
}
#endif

}  // namespace hlo
