// Checks of the views that the layer entry points take (layer_api.cu, cache_api.cu): dimensions, strides and alignment,
// and whether operands share memory.
#pragma once
#include <algorithm>
#include <cstdint>

#include "hlo_api.h"
#include "layer_plans.h"

namespace hlo {

inline bool is_float(int dt) { return dt == F32 || dt == BF16 || dt == F16; }

// Elements from the first to one past the last that a view spans (0 if it is empty).
inline int64_t span(const hlo_view& v, int first = 0) {
  int64_t s = 1;
  for (int d = first; d < v.rank; ++d) {
    if (v.dims[d] == 0) return 0;
    if (v.dims[d] > 1) s += (v.dims[d] - 1) * v.strides[d];
  }
  return s;
}

inline int64_t numel(const hlo_view& v) {
  int64_t n = 1;
  for (int d = 0; d < v.rank; ++d) n *= v.dims[d];
  return n;
}

inline const char* end_of(const hlo_view* v, const void* ptr) {
  return v ? static_cast<const char*>(ptr) + span(*v) * view_dt_bytes(v->dtype) : nullptr;
}

inline hlo_status check_view(const hlo_view* v, const void* ptr, const char* what, bool output) {
  if (!v) return api_fail(HLO_ERR_INVALID_ARG, "%s: view is NULL", what);
  if (v->rank < 1 || v->rank > HLO_MAX_RANK)
    return api_fail(HLO_ERR_INVALID_ARG, "%s: rank %d outside 1..%d", what, v->rank, HLO_MAX_RANK);
  if (view_dt_bytes(v->dtype) == 0) return api_fail(HLO_ERR_INVALID_ARG, "%s: unknown element type %d", what, v->dtype);
  long double count = 1, extent = 1;
  bool empty = false;
  for (int d = 0; d < v->rank; ++d) {
    if (v->dims[d] < 0) return api_fail(HLO_ERR_INVALID_ARG, "%s: dimension %d has negative size", what, d);
    if (v->strides[d] < 0) return api_fail(HLO_ERR_INVALID_ARG, "%s: dimension %d has a negative stride", what, d);
    empty = empty || v->dims[d] == 0;
    count *= (long double)v->dims[d];
    if (v->dims[d] > 1) extent += (long double)(v->dims[d] - 1) * (long double)v->strides[d];
  }
  if (!empty && (count * 4 > 4.0e18L || extent * 4 > 4.0e18L)) return api_fail(HLO_ERR_INVALID_ARG, "%s: array too large", what);
  if (v->dims[v->rank - 1] > 1 && v->strides[v->rank - 1] != 1)
    return api_fail(HLO_ERR_UNSUPPORTED, "%s: the last dimension's stride must be 1, not %lld", what,
                    (long long)v->strides[v->rank - 1]);
  if (empty) return HLO_OK;
  if (!ptr) return api_fail(HLO_ERR_INVALID_ARG, "%s: NULL pointer", what);
  if ((uintptr_t)ptr % view_dt_bytes(v->dtype) != 0)
    return api_fail(HLO_ERR_INVALID_ARG, "%s: pointer is not aligned to its element type", what);
  if (output) {  // distinct elements: each stride clears the span of the smaller ones
    int order[HLO_MAX_RANK], k = 0;
    for (int d = 0; d < v->rank; ++d)
      if (v->dims[d] > 1) order[k++] = d;
    std::sort(order, order + k, [&](int a, int b) { return v->strides[a] < v->strides[b]; });
    int64_t inner = 1;
    for (int i = 0; i < k; ++i) {
      if (v->strides[order[i]] < inner)
        return api_fail(HLO_ERR_INVALID_ARG, "%s: output elements overlap (stride %lld of dimension %d)", what,
                        (long long)v->strides[order[i]], order[i]);
      inner += (v->dims[order[i]] - 1) * v->strides[order[i]];
    }
  }
  return HLO_OK;
}

inline hlo_status same_dims(const hlo_view& a, const hlo_view& b, const char* what) {
  if (a.rank != b.rank) return api_fail(HLO_ERR_INVALID_ARG, "%s: rank %d, expected %d", what, b.rank, a.rank);
  for (int d = 0; d < a.rank; ++d)
    if (a.dims[d] != b.dims[d])
      return api_fail(HLO_ERR_INVALID_ARG, "%s: dimension %d is %lld, expected %lld", what, d, (long long)b.dims[d],
                      (long long)a.dims[d]);
  return HLO_OK;
}

inline bool ranges_overlap(const void* a, int64_t abytes, const void* b, int64_t bbytes) {
  if (!a || !b || abytes <= 0 || bbytes <= 0) return false;
  const uintptr_t a0 = (uintptr_t)a, b0 = (uintptr_t)b;
  return a0 < b0 + (uintptr_t)bbytes && b0 < a0 + (uintptr_t)abytes;
}

// A view as a byte box: sizes and byte strides of its dimensions of more than one element, largest
// stride first, neighbours merged; the innermost entry is the element itself.
struct Box {
  int n = 0;
  int64_t size[HLO_MAX_RANK], stride[HLO_MAX_RANK];
  int64_t inner = 1;  // bytes of the contiguous run

  explicit Box(const hlo_view& v) {
    const int eb = view_dt_bytes(v.dtype);
    inner = eb;
    int order[HLO_MAX_RANK], k = 0;
    for (int d = 0; d < v.rank; ++d)
      if (v.dims[d] > 1 && v.strides[d] > 0) order[k++] = d;
    std::sort(order, order + k, [&](int a, int b) { return v.strides[a] > v.strides[b]; });
    for (int i = 0; i < k; ++i) {
      const int64_t sz = v.dims[order[i]], st = v.strides[order[i]] * eb;
      if (n > 0 && stride[n - 1] == st * sz) {
        size[n - 1] *= sz;
        stride[n - 1] = st;
      } else {
        size[n] = sz;
        stride[n++] = st;
      }
    }
    if (n > 0 && stride[n - 1] == inner) inner *= size[--n];
  }
  int64_t bytes(int from) const {
    int64_t s = inner;
    for (int i = from; i < n; ++i) s += (size[i] - 1) * stride[i];
    return s;
  }
};

// Whether box a (at byte 0, from dimension i) and box b (at byte `at`, from dimension j) provably share
// no byte: their ranges are apart, or they step alike and within one step their windows are apart.
inline bool apart(const Box& a, int i, const Box& b, int j, int64_t at) {
  if (at < 0) return apart(b, j, a, i, -at);
  if (at >= a.bytes(i)) return true;
  if (i >= a.n || j >= b.n || a.stride[i] != b.stride[j]) return false;
  const int64_t step = a.stride[i], wa = a.bytes(i + 1), wb = b.bytes(j + 1), r = at % step;
  if (r >= wa && r + wb <= step) return true;
  // the windows fall into the same step of each period, or b's hangs over into the next one
  if (wa <= step && r + wb <= step) return apart(a, i + 1, b, j + 1, r);
  return false;
}

struct Operand {
  const hlo_view* v;
  const void* p;
  const char* what;
};

inline bool same_place(const hlo_view& a, const void* pa, const hlo_view& b, const void* pb) {
  if (pa != pb || a.dtype != b.dtype || a.rank != b.rank) return false;
  for (int d = 0; d < a.rank; ++d)
    if (a.dims[d] != b.dims[d] || (a.dims[d] > 1 && a.strides[d] != b.strides[d])) return false;
  return true;
}

// Checks one output against the inputs it may replace in place (`ins`) and the other outputs.
inline hlo_status check_overlap(const Operand& o, const Operand* ins, int n_ins, const Operand* outs, int n_outs) {
  if (numel(*o.v) == 0) return HLO_OK;
  for (int k = 0; k < n_ins + n_outs; ++k) {
    const Operand& q = k < n_ins ? ins[k] : outs[k - n_ins];
    if (&q == &o || !q.v || !q.p || numel(*q.v) == 0) continue;
    if (k < n_ins && same_place(*o.v, o.p, *q.v, q.p)) continue;
    const Box a(*o.v), b(*q.v);
    if (!apart(a, 0, b, 0, (int64_t)((intptr_t)q.p - (intptr_t)o.p)))
      return api_fail(HLO_ERR_INVALID_ARG, "%s overlaps %s", o.what, q.what);
  }
  return HLO_OK;
}

// ... and against a dense side buffer.
inline hlo_status check_side(const Operand& o, const void* p, int64_t bytes, const char* what) {
  if (ranges_overlap(o.p, span(*o.v) * view_dt_bytes(o.v->dtype), p, bytes))
    return api_fail(HLO_ERR_INVALID_ARG, "%s overlaps %s", o.what, what);
  return HLO_OK;
}

inline cudaStream_t as_stream(void* s) { return reinterpret_cast<cudaStream_t>(s); }

}  // namespace hlo

#define TRY(call)                     \
  do {                                \
    const hlo_status st_ = (call);    \
    if (st_ != HLO_OK) return st_;    \
  } while (0)
#define INJECT(site) \
  if (api_injected(site)) return api_fail(HLO_ERR_CUDA, "%s: injected fault (HLOFUSION_FAULT)", site)
