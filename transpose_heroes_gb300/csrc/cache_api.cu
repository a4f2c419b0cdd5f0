// C-ABI entry points of the paged cache (hlo_cache_append, hlo_cache_attention, hlo_tree_accept and their host
// helpers): checks, plan and launch. No device memory is allocated here.
#include <cmath>
#include <cstring>

#include "cache_plans.h"
#include "hlo_api.h"
#include "view_checks.h"

using namespace hlo;

namespace {

// The cache's views: `layers` tells whether a dimension of layers may come first. A cache that a call writes has to have
// distinct elements.
hlo_status check_cache(const hlo_cache* c, const char* who, bool layers, bool written) {
  char what[64];
  const auto name = [&](const char* part) {
    snprintf(what, sizeof what, "%s %s", who, part);
    return what;
  };
  TRY(check_view(&c->k, c->k_ptr, name("k_cache"), written));
  TRY(check_view(&c->v, c->v_ptr, name("v_cache"), written));
  if (c->k.rank != 4 && !(layers && c->k.rank == 5))
    return api_fail(HLO_ERR_INVALID_ARG, "%s k_cache: rank %d, expected [%spages, page_size, kv, dim]", who, c->k.rank,
                    layers ? "layers, " : "");
  TRY(same_dims(c->k, c->v, name("v_cache")));
  if (c->k.dtype != c->v.dtype)
    return api_fail(HLO_ERR_INVALID_ARG, "%s v_cache: type %d differs from k_cache's %d", who, c->v.dtype, c->k.dtype);
  if (!is_float(c->k.dtype) && c->k.dtype != HLO_F8E4M3FN)
    return api_fail(HLO_ERR_UNSUPPORTED, "%s k_cache: element type %d not supported", who, c->k.dtype);
  const double scales[2] = {c->k_scale, c->v_scale};
  for (double s : scales) {
    if (!((float)s > 0.0f) || !std::isfinite((float)s))
      return api_fail(HLO_ERR_INVALID_ARG, "%s: k_scale and v_scale must be finite and > 0", who);
    if (c->k.dtype != HLO_F8E4M3FN && s != 1.0)
      return api_fail(HLO_ERR_INVALID_ARG, "%s: k_scale and v_scale belong to an f8E4M3FN cache", who);
  }
  const int lead = c->k.rank - 4;
  if (c->k.dims[lead + 1] < 1) return api_fail(HLO_ERR_INVALID_ARG, "%s k_cache: pages of no entries", who);
  if (c->k.dims[lead] > INT32_MAX || c->k.dims[lead + 1] > INT32_MAX || c->k.dims[lead + 2] > 32767)
    return api_fail(HLO_ERR_UNSUPPORTED, "%s k_cache: %lld pages of %lld entries of %lld heads", who, (long long)c->k.dims[lead],
                    (long long)c->k.dims[lead + 1], (long long)c->k.dims[lead + 2]);
  TRY(check_view(&c->table, c->table_ptr, name("table"), false));
  if (c->table.dtype != HLO_S32) return api_fail(HLO_ERR_INVALID_ARG, "%s table: element type must be s32", who);
  if (c->table.rank != 2) return api_fail(HLO_ERR_INVALID_ARG, "%s table: rank %d, expected [batch, max_pages]", who, c->table.rank);
  if ((long double)c->table.dims[1] * (long double)c->k.dims[lead + 1] > (long double)INT32_MAX)
    return api_fail(HLO_ERR_UNSUPPORTED, "%s table: %lld pages of %lld entries reach 2^31", who, (long long)c->table.dims[1],
                    (long long)c->k.dims[lead + 1]);
  if (c->table.dims[0] > 0 && !c->lengths) return api_fail(HLO_ERR_INVALID_ARG, "%s: lengths is NULL", who);
  if ((uintptr_t)c->lengths % 4 != 0) return api_fail(HLO_ERR_INVALID_ARG, "%s: lengths is not 4-byte aligned", who);
  if (written) {
    const Operand k = {&c->k, c->k_ptr, "the k_cache"}, v[1] = {{&c->v, c->v_ptr, "the v_cache"}};
    TRY(check_overlap(k, nullptr, 0, v, 1));
  }
  return HLO_OK;
}

// An output against everything that a call reads of its cache.
hlo_status check_against_cache(const Operand& o, const hlo_cache* c, bool with_entries) {
  if (numel(*o.v) == 0) return HLO_OK;
  if (with_entries) {
    const Operand kv[2] = {{&c->k, c->k_ptr, "the k_cache"}, {&c->v, c->v_ptr, "the v_cache"}};
    TRY(check_overlap(o, nullptr, 0, kv, 2));
  }
  const Operand t[1] = {{&c->table, c->table_ptr, "the table"}};
  TRY(check_overlap(o, nullptr, 0, t, 1));
  return check_side(o, c->lengths, c->table.dims[0] * 4, "the lengths");
}

void map_of(const hlo_cache* c, const int32_t* counts, int64_t batch, int64_t seq, CacheMap* m) {
  std::memset(m, 0, sizeof *m);
  m->counts = counts;
  m->batch = (int)batch;
  m->seq = (int)seq;
  if (!c) return;
  const int lead = c->k.rank - 4;
  m->table = c->table_ptr;
  m->table_stride = batch > 1 ? c->table.strides[0] : 0;
  m->lengths = c->lengths;
  m->pages = c->k.dims[lead];
  m->page_size = (int)c->k.dims[lead + 1];
  m->page_shift = -1;
  for (int k = 0; k < 31; ++k)
    if (m->page_size == 1 << k) m->page_shift = k;
  m->max_pages = (int)c->table.dims[1];
  m->capacity = m->max_pages * m->page_size;
}

// Strides of the dimensions from `first` on; those of size 1 as 0, so that they do not matter to alignment.
void strides_of(const hlo_view& v, int first, int n, int64_t* out) {
  for (int d = 0; d < n; ++d) out[d] = v.dims[first + d] > 1 ? v.strides[first + d] : 0;
}

hlo_status check_count(int64_t batch, int64_t seq, int64_t heads, const int32_t* counts, const char* who) {
  if (batch > INT32_MAX / 8 || seq > INT32_MAX / 8 || (long double)batch * (long double)seq > (long double)(INT32_MAX / 8) ||
      (long double)seq * (long double)heads > (long double)(INT32_MAX / 8))
    return api_fail(HLO_ERR_UNSUPPORTED, "%s: %lld sequences of %lld new tokens of %lld heads", who, (long long)batch, (long long)seq,
                    (long long)heads);
  if ((uintptr_t)counts % 4 != 0) return api_fail(HLO_ERR_INVALID_ARG, "%s: counts is not 4-byte aligned", who);
  return HLO_OK;
}

hlo_status check_tokens(const hlo_view* v, const void* ptr, int64_t batch, int64_t seq, const char* what, bool output) {
  TRY(check_view(v, ptr, what, output));
  if (v->dtype != HLO_S32) return api_fail(HLO_ERR_INVALID_ARG, "%s: element type must be s32", what);
  if (v->rank != 2 || v->dims[0] != batch || v->dims[1] != seq)
    return api_fail(HLO_ERR_INVALID_ARG, "%s: shape must be [%lld, %lld]", what, (long long)batch, (long long)seq);
  return HLO_OK;
}

}  // namespace

extern "C" {

hlo_status hlo_cache_append(const hlo_cache* cache, const hlo_view* k, const void* k_ptr, const hlo_view* v, const void* v_ptr,
                            const hlo_view* q, const void* q_ptr, const hlo_view* q_out, void* q_out_ptr,
                            const int32_t* counts, const hlo_view* positions, const int32_t* positions_ptr,
                            const uint64_t* turns, int32_t n_pairs, int32_t interleaved, double scale, void* stream) {
  if (!cache) return api_fail(HLO_ERR_INVALID_ARG, "cache_append: the cache is NULL");
  TRY(check_cache(cache, "cache_append", false, true));
  TRY(check_view(k, k_ptr, "cache_append k", false));
  if (!is_float(k->dtype)) return api_fail(HLO_ERR_UNSUPPORTED, "cache_append k: element type %d not supported", k->dtype);
  if (k->rank != 4) return api_fail(HLO_ERR_INVALID_ARG, "cache_append k: rank %d, expected [batch, seq, kv, dim]", k->rank);
  TRY(check_view(v, v_ptr, "cache_append v", false));
  TRY(same_dims(*k, *v, "cache_append v"));
  if ((q == nullptr) != (q_out == nullptr)) return api_fail(HLO_ERR_INVALID_ARG, "cache_append: q and q_out go together");
  if (q) {
    TRY(check_view(q, q_ptr, "cache_append q", false));
    TRY(check_view(q_out, q_out_ptr, "cache_append q_out", true));
    TRY(same_dims(*q, *q_out, "cache_append q_out"));
    if (q->rank != 4 || q->dims[0] != k->dims[0] || q->dims[1] != k->dims[1] || q->dims[3] != k->dims[3])
      return api_fail(HLO_ERR_INVALID_ARG, "cache_append q: shape must be k's but for the heads");
  }
  if (v->dtype != k->dtype || (q && (q->dtype != k->dtype || q_out->dtype != k->dtype)))
    return api_fail(HLO_ERR_INVALID_ARG, "cache_append: q, k and v must have one element type");
  if (cache->k.dtype != k->dtype && cache->k.dtype != HLO_F8E4M3FN)
    return api_fail(HLO_ERR_INVALID_ARG, "cache_append: the cache's type %d is neither k's nor f8E4M3FN", cache->k.dtype);
  const int64_t batch = k->dims[0], seq = k->dims[1], kv = k->dims[2], dim = k->dims[3], heads = q ? q->dims[2] : 0;
  if (cache->k.dims[2] != kv || cache->k.dims[3] != dim)
    return api_fail(HLO_ERR_INVALID_ARG, "cache_append: k has %lld heads of %lld, the cache %lld of %lld", (long long)kv,
                    (long long)dim, (long long)cache->k.dims[2], (long long)cache->k.dims[3]);
  if (cache->table.dims[0] != batch)
    return api_fail(HLO_ERR_INVALID_ARG, "cache_append table: %lld sequences, k has %lld", (long long)cache->table.dims[0], (long long)batch);
  if (dim > 512) return api_fail(HLO_ERR_UNSUPPORTED, "cache_append k: heads of %lld elements (512 at most)", (long long)dim);
  if (heads > 32767) return api_fail(HLO_ERR_UNSUPPORTED, "cache_append q: %lld heads", (long long)heads);
  TRY(check_count(batch, seq, heads + 2 * kv, counts, "cache_append"));
  if (positions) TRY(check_tokens(positions, positions_ptr, batch, seq, "cache_append positions", false));
  if (n_pairs < 0 || 2 * (int64_t)n_pairs > dim)
    return api_fail(HLO_ERR_INVALID_ARG, "cache_append: %d pairs in heads of %lld elements", n_pairs, (long long)dim);
  if (n_pairs > 0 && !turns) return api_fail(HLO_ERR_INVALID_ARG, "cache_append: turns is NULL");
  if ((uintptr_t)turns % 8 != 0) return api_fail(HLO_ERR_INVALID_ARG, "cache_append: turns is not 8-byte aligned");
  if (!std::isfinite(scale)) return api_fail(HLO_ERR_INVALID_ARG, "cache_append: scale is not finite");
  const Operand outs[3] = {{&cache->k, cache->k_ptr, "cache_append k_cache"},
                           {&cache->v, cache->v_ptr, "cache_append v_cache"},
                           {q_out, q_out_ptr, "cache_append q_out"}};
  const Operand ins[4] = {{q, q_ptr, "q"}, {k, k_ptr, "k"}, {v, v_ptr, "v"}, {positions, positions_ptr, "the positions"}};
  for (int i = 0; i < 3; ++i) {
    if (!outs[i].v) continue;
    // queries may turn in place
    TRY(check_overlap(outs[i], ins, i == 2 ? 1 : 0, ins + (i == 2 ? 1 : 0), i == 2 ? 3 : 4));
    TRY(check_against_cache(outs[i], cache, i == 2));
    TRY(check_side(outs[i], counts, batch * 4, "counts"));
    TRY(check_side(outs[i], turns, (int64_t)n_pairs * 8, "turns"));
  }
  AppendPlan p;
  std::memset(&p, 0, sizeof p);
  map_of(cache, counts, batch, seq, &p.m);
  const hlo_view* const views[3] = {q, k, v};
  const void* const ptrs[3] = {q_ptr, k_ptr, v_ptr};
  for (int a = 0; a < 3; ++a) {
    if (!views[a] || numel(*views[a]) == 0) continue;
    p.in[a] = ptrs[a];
    strides_of(*views[a], 0, 3, p.in_stride[a]);
  }
  if (p.in[0]) {
    p.q_out = q_out_ptr;
    strides_of(*q_out, 0, 3, p.q_stride);
  }
  p.cache[0] = cache->k_ptr;
  p.cache[1] = cache->v_ptr;
  strides_of(cache->k, 0, 3, p.cache_stride[0]);
  strides_of(cache->v, 0, 3, p.cache_stride[1]);
  p.heads = p.in[0] ? (int)heads : 0;
  p.kv = p.in[1] ? (int)kv : 0;
  p.dim = (int)dim;
  p.pairs = n_pairs;
  p.dt = k->dtype;
  p.f8 = cache->k.dtype == HLO_F8E4M3FN;
  p.interleaved = interleaved ? 1 : 0;
  p.pos = positions ? positions_ptr : nullptr;
  if (positions) strides_of(*positions, 0, 2, p.pos_stride);
  p.turns = turns;
  p.scale = (float)scale;
  const double scales[2] = {cache->k_scale, cache->v_scale};
  for (int i = 0; i < 2; ++i) {
    p.code_scale[i] = (float)scales[i];
    p.code_inv[i] = 1.0f / p.code_scale[i];
  }
  if (!p.in[0] && !p.in[1]) return api_ok();
  INJECT("hlo_cache_append");
  return api_cuda_status(launch_append(p, as_stream(stream)), "cache_append launch");
}

size_t hlo_cache_attention_workspace_size(int64_t batch, int64_t seq, int64_t heads, int64_t kv, int64_t dim) {
  if (batch <= 0 || seq <= 0 || heads <= 0 || kv <= 0 || dim <= 0 || dim > 256) return 0;
  return attend_workspace(batch, seq, heads, kv, dim);
}

hlo_status hlo_cache_attention(const hlo_cache* cache, const hlo_view* q, const void* q_ptr, const int32_t* counts,
                               const hlo_view* mask, const int32_t* mask_ptr, double scale, const hlo_view* out, void* out_ptr,
                               float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  if (!cache) return api_fail(HLO_ERR_INVALID_ARG, "cache_attention: the cache is NULL");
  TRY(check_cache(cache, "cache_attention", false, false));
  TRY(check_view(q, q_ptr, "cache_attention q", false));
  if (!is_float(q->dtype)) return api_fail(HLO_ERR_UNSUPPORTED, "cache_attention q: element type %d not supported", q->dtype);
  if (q->rank != 4) return api_fail(HLO_ERR_INVALID_ARG, "cache_attention q: rank %d, expected [batch, seq, heads, dim]", q->rank);
  TRY(check_view(out, out_ptr, "cache_attention out", true));
  TRY(same_dims(*q, *out, "cache_attention out"));
  if (out->dtype != q->dtype)
    return api_fail(HLO_ERR_INVALID_ARG, "cache_attention out: type %d differs from q's %d", out->dtype, q->dtype);
  if (cache->k.dtype != q->dtype && cache->k.dtype != HLO_F8E4M3FN)
    return api_fail(HLO_ERR_INVALID_ARG, "cache_attention: the cache's type %d is neither q's nor f8E4M3FN", cache->k.dtype);
  const int64_t batch = q->dims[0], seq = q->dims[1], heads = q->dims[2], dim = q->dims[3], kv = cache->k.dims[2];
  if (cache->k.dims[3] != dim)
    return api_fail(HLO_ERR_INVALID_ARG, "cache_attention: q's heads have %lld elements, the cache's %lld", (long long)dim,
                    (long long)cache->k.dims[3]);
  if (dim < 1 || dim > 256) return api_fail(HLO_ERR_UNSUPPORTED, "cache_attention q: heads of %lld elements (1 to 256)", (long long)dim);
  if (heads > 0 && (kv < 1 || heads % kv != 0))
    return api_fail(HLO_ERR_INVALID_ARG, "cache_attention: %lld query heads are no multiple of %lld key heads", (long long)heads,
                    (long long)kv);
  if (cache->table.dims[0] != batch)
    return api_fail(HLO_ERR_INVALID_ARG, "cache_attention table: %lld sequences, q has %lld", (long long)cache->table.dims[0],
                    (long long)batch);
  TRY(check_count(batch, seq, heads, counts, "cache_attention"));
  if (mask) {
    TRY(check_view(mask, mask_ptr, "cache_attention mask", false));
    if (mask->dtype != HLO_S32) return api_fail(HLO_ERR_INVALID_ARG, "cache_attention mask: element type must be s32");
    if (mask->rank != 3 || mask->dims[0] != batch || mask->dims[1] != seq || mask->dims[2] != (seq + 31) / 32)
      return api_fail(HLO_ERR_INVALID_ARG, "cache_attention mask: shape must be [%lld, %lld, %lld]", (long long)batch, (long long)seq,
                      (long long)((seq + 31) / 32));
  }
  if (!((float)scale > 0.0f) || !std::isfinite((float)scale))
    return api_fail(HLO_ERR_INVALID_ARG, "cache_attention: scale must be finite and > 0");
  const float score = (float)(scale * cache->k_scale * 1.4426950408889634);
  if (!(score > 0.0f) || !std::isfinite(score)) return api_fail(HLO_ERR_UNSUPPORTED, "cache_attention: scale * k_scale leaves f32");
  if ((uintptr_t)lse % 4 != 0) return api_fail(HLO_ERR_INVALID_ARG, "cache_attention: lse is not 4-byte aligned");
  const int64_t need = numel(*q) == 0 ? 0 : (int64_t)hlo_cache_attention_workspace_size(batch, seq, heads, kv, dim);
  if (need > 0) {
    if (!workspace || (int64_t)workspace_bytes < need)
      return api_fail(HLO_ERR_WORKSPACE, "cache_attention: workspace of %zu bytes, %lld needed (hlo_cache_attention_workspace_size)",
                      workspace ? workspace_bytes : (size_t)0, (long long)need);
    if ((uintptr_t)workspace % 16 != 0) return api_fail(HLO_ERR_INVALID_ARG, "cache_attention: workspace is not 16-byte aligned");
  }
  const Operand o = {out, out_ptr, "cache_attention out"};
  const Operand ins[2] = {{q, q_ptr, "cache_attention q"}, {mask, mask_ptr, "the mask"}};
  TRY(check_overlap(o, ins, 1, ins + 1, 1));
  TRY(check_against_cache(o, cache, true));
  TRY(check_side(o, counts, batch * 4, "counts"));
  // what else the call writes: the statistics and the workspace, against all that it reads or writes
  const struct {
    const void* p;
    int64_t bytes;
    const char* what;
  } side[2] = {{lse, batch * seq * heads * 4, "lse"}, {workspace, need, "the workspace"}};
  const Operand all[6] = {o, ins[0], ins[1], {&cache->k, cache->k_ptr, "the k_cache"}, {&cache->v, cache->v_ptr, "the v_cache"},
                          {&cache->table, cache->table_ptr, "the table"}};
  for (const auto& s : side) {
    for (const Operand& a : all)
      if (a.v) TRY(check_side(a, s.p, s.bytes, s.what));
    if (ranges_overlap(s.p, s.bytes, counts, batch * 4) || ranges_overlap(s.p, s.bytes, cache->lengths, batch * 4))
      return api_fail(HLO_ERR_INVALID_ARG, "cache_attention: %s overlaps counts or lengths", s.what);
  }
  if (ranges_overlap(side[0].p, side[0].bytes, side[1].p, side[1].bytes))
    return api_fail(HLO_ERR_INVALID_ARG, "cache_attention: lse overlaps the workspace");
  if (numel(*q) == 0) return api_ok();
  AttendPlan p;
  std::memset(&p, 0, sizeof p);
  map_of(cache, counts, batch, seq, &p.m);
  p.q = q_ptr;
  p.k = cache->k_ptr;
  p.v = cache->v_ptr;
  p.out = out_ptr;
  p.lse = lse;
  strides_of(*q, 0, 3, p.q_stride);
  strides_of(*out, 0, 3, p.out_stride);
  strides_of(cache->k, 0, 3, p.k_stride);
  strides_of(cache->v, 0, 3, p.v_stride);
  if (mask) {
    p.mask = reinterpret_cast<const uint32_t*>(mask_ptr);
    strides_of(*mask, 0, 2, p.mask_stride);
  }
  p.heads = (int)heads;
  p.kv = (int)kv;
  p.group = (int)(heads / kv);
  p.dim = (int)dim;
  p.dt = q->dtype;
  p.f8 = cache->k.dtype == HLO_F8E4M3FN;
  p.score_scale = score;
  p.value_scale = (float)cache->v_scale;
  INJECT("hlo_cache_attention");
  return api_cuda_status(launch_attend(p, workspace, as_stream(stream)), "cache_attention launch");
}

hlo_status hlo_tree_mask(const int32_t* parents, int32_t n, uint32_t* mask, int32_t* depths) {
  if (n < 0) return api_fail(HLO_ERR_INVALID_ARG, "tree_mask: n is negative");
  if (n > 0 && (!parents || !mask)) return api_fail(HLO_ERR_INVALID_ARG, "tree_mask: NULL pointer");
  const int64_t words = ((int64_t)n + 31) / 32;
  for (int32_t c = 0; c < n; ++c)
    if (parents[c] < -1 || parents[c] >= c)
      return api_fail(HLO_ERR_INVALID_ARG, "tree_mask: the parent of node %d is %d, outside -1..%d", c, parents[c], c - 1);
  for (int32_t c = 0; c < n; ++c) {
    uint32_t* const row = mask + c * words;
    const int32_t up = parents[c];
    if (up < 0) std::memset(row, 0, words * sizeof *row);
    else std::memcpy(row, mask + up * words, words * sizeof *row);
    row[c >> 5] |= 1u << (c & 31);
    if (depths) depths[c] = up < 0 ? 0 : depths[up] + 1;
  }
  return api_ok();
}

hlo_status hlo_tree_accept(const hlo_view* tokens, const int32_t* tokens_ptr, const hlo_view* parents, const int32_t* parents_ptr,
                           const hlo_view* picks, const int32_t* picks_ptr, const int32_t* counts, const hlo_cache* cache,
                           const hlo_view* path, int32_t* path_ptr, int32_t* accepted, int32_t* next, void* stream) {
  TRY(check_view(tokens, tokens_ptr, "tree_accept tokens", false));
  if (tokens->rank != 2) return api_fail(HLO_ERR_INVALID_ARG, "tree_accept tokens: rank %d, expected [batch, seq]", tokens->rank);
  const int64_t batch = tokens->dims[0], seq = tokens->dims[1];
  TRY(check_tokens(tokens, tokens_ptr, batch, seq, "tree_accept tokens", false));
  TRY(check_tokens(parents, parents_ptr, batch, seq, "tree_accept parents", false));
  TRY(check_tokens(picks, picks_ptr, batch, seq, "tree_accept picks", false));
  TRY(check_tokens(path, path_ptr, batch, seq, "tree_accept path", true));
  TRY(check_count(batch, seq, 1, counts, "tree_accept"));
  if (seq > 4096) return api_fail(HLO_ERR_UNSUPPORTED, "tree_accept: trees of %lld nodes (4096 at most)", (long long)seq);
  if (batch > 0 && (!accepted || !next)) return api_fail(HLO_ERR_INVALID_ARG, "tree_accept: accepted or next is NULL");
  if (((uintptr_t)accepted | (uintptr_t)next) % 4 != 0)
    return api_fail(HLO_ERR_INVALID_ARG, "tree_accept: accepted and next must be 4-byte aligned");
  if (cache) {
    TRY(check_cache(cache, "tree_accept", true, true));
    if (cache->table.dims[0] != batch)
      return api_fail(HLO_ERR_INVALID_ARG, "tree_accept table: %lld sequences, tokens has %lld", (long long)cache->table.dims[0],
                      (long long)batch);
  }
  const Operand ins[3] = {{tokens, tokens_ptr, "tokens"}, {parents, parents_ptr, "parents"}, {picks, picks_ptr, "picks"}};
  const Operand outs[3] = {{path, path_ptr, "tree_accept path"},
                           {cache ? &cache->k : nullptr, cache ? cache->k_ptr : nullptr, "tree_accept k_cache"},
                           {cache ? &cache->v : nullptr, cache ? cache->v_ptr : nullptr, "tree_accept v_cache"}};
  for (int i = 0; i < 3; ++i) {
    if (!outs[i].v) continue;
    TRY(check_overlap(outs[i], nullptr, 0, ins, 3));
    TRY(check_side(outs[i], counts, batch * 4, "counts"));
    TRY(check_side(outs[i], accepted, batch * 4, "accepted"));
    TRY(check_side(outs[i], next, batch * 4, "next"));
    if (cache) TRY(check_against_cache(outs[i], cache, i == 0));
  }
  int32_t* const vectors[2] = {accepted, next};
  for (int32_t* q : vectors) {
    for (const Operand& i : ins) TRY(check_side(i, q, batch * 4, "accepted or next"));
    if (cache) {
      const Operand t = {&cache->table, cache->table_ptr, "tree_accept table"};
      TRY(check_side(t, q, batch * 4, "accepted or next"));
    }
    if (ranges_overlap(q, batch * 4, counts, batch * 4) || (cache && ranges_overlap(q, batch * 4, cache->lengths, batch * 4)))
      return api_fail(HLO_ERR_INVALID_ARG, "tree_accept: accepted or next overlaps counts or lengths");
  }
  if (ranges_overlap(accepted, batch * 4, next, batch * 4))
    return api_fail(HLO_ERR_INVALID_ARG, "tree_accept: accepted overlaps next");
  AcceptPlan p;
  std::memset(&p, 0, sizeof p);
  map_of(cache, counts, batch, seq, &p.m);
  p.tokens = tokens_ptr;
  p.parents = parents_ptr;
  p.picks = picks_ptr;
  p.path = path_ptr;
  p.accepted = accepted;
  p.next = next;
  strides_of(*tokens, 0, 2, p.tokens_stride);
  strides_of(*parents, 0, 2, p.parents_stride);
  strides_of(*picks, 0, 2, p.picks_stride);
  strides_of(*path, 0, 2, p.path_stride);
  p.width = 1;
  if (cache && numel(cache->k) > 0) {
    const int lead = cache->k.rank - 4, eb = view_dt_bytes(cache->k.dtype);
    p.layers = lead ? (int)std::min<int64_t>(cache->k.dims[0], INT32_MAX) : 1;
    p.kv = (int)cache->k.dims[lead + 2];
    p.row_bytes = cache->k.dims[lead + 3] * eb;
    p.cache[0] = cache->k_ptr;
    p.cache[1] = cache->v_ptr;
    const hlo_view* const views[2] = {&cache->k, &cache->v};
    uintptr_t bits = (uintptr_t)p.row_bytes;
    for (int i = 0; i < 2; ++i) {
      strides_of(*views[i], 0, 3 + lead, p.cache_stride[i] + 1 - lead);
      for (int d = 0; d < 4; ++d) {
        p.cache_stride[i][d] *= eb;
        bits |= (uintptr_t)p.cache_stride[i][d];
      }
      bits |= (uintptr_t)p.cache[i];
    }
    while (p.width < 16 && bits % (2 * p.width) == 0) p.width *= 2;
    if ((long double)p.layers * 2 * p.kv * (p.row_bytes / p.width) > (long double)(INT32_MAX / 2))
      return api_fail(HLO_ERR_UNSUPPORTED, "tree_accept: %d layers of %d heads of %lld bytes", p.layers, p.kv, (long long)p.row_bytes);
  }
  if (batch == 0) return api_ok();
  INJECT("hlo_tree_accept");
  return api_cuda_status(launch_accept(p, as_stream(stream)), "tree_accept launch");
}

}  // extern "C"
