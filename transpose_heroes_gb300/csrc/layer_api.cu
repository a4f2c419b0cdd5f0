// C-ABI entry points of the fusions between a decoder's matrix products (hlo_rms_norm and its gradient,
// hlo_dropout, hlo_rotary, hlo_logits_process): checks of the views, merging of outer dimensions, plan and
// launch. No device memory is allocated here.
#include <algorithm>
#include <cmath>
#include <cstring>

#include "hlo_api.h"
#include "layer_plans.h"
#include "philox.cuh"

using namespace hlo;

namespace {

bool is_float(int dt) { return dt == F32 || dt == BF16 || dt == F16; }

// Elements from the first to one past the last that a view spans (0 if it is empty).
int64_t span(const hlo_view& v, int first = 0) {
  int64_t s = 1;
  for (int d = first; d < v.rank; ++d) {
    if (v.dims[d] == 0) return 0;
    if (v.dims[d] > 1) s += (v.dims[d] - 1) * v.strides[d];
  }
  return s;
}

int64_t numel(const hlo_view& v) {
  int64_t n = 1;
  for (int d = 0; d < v.rank; ++d) n *= v.dims[d];
  return n;
}

const char* end_of(const hlo_view* v, const void* ptr) {
  return v ? static_cast<const char*>(ptr) + span(*v) * view_dt_bytes(v->dtype) : nullptr;
}

hlo_status check_view(const hlo_view* v, const void* ptr, const char* what, bool output) {
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

hlo_status same_dims(const hlo_view& a, const hlo_view& b, const char* what) {
  if (a.rank != b.rank) return api_fail(HLO_ERR_INVALID_ARG, "%s: rank %d, expected %d", what, b.rank, a.rank);
  for (int d = 0; d < a.rank; ++d)
    if (a.dims[d] != b.dims[d])
      return api_fail(HLO_ERR_INVALID_ARG, "%s: dimension %d is %lld, expected %lld", what, d, (long long)b.dims[d],
                      (long long)a.dims[d]);
  return HLO_OK;
}

bool ranges_overlap(const void* a, int64_t abytes, const void* b, int64_t bbytes) {
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
bool apart(const Box& a, int i, const Box& b, int j, int64_t at) {
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

bool same_place(const hlo_view& a, const void* pa, const hlo_view& b, const void* pb) {
  if (pa != pb || a.dtype != b.dtype || a.rank != b.rank) return false;
  for (int d = 0; d < a.rank; ++d)
    if (a.dims[d] != b.dims[d] || (a.dims[d] > 1 && a.strides[d] != b.strides[d])) return false;
  return true;
}

// Checks one output against the inputs it may replace in place (`ins`) and the other outputs.
hlo_status check_overlap(const Operand& o, const Operand* ins, int n_ins, const Operand* outs, int n_outs) {
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
hlo_status check_side(const Operand& o, const void* p, int64_t bytes, const char* what) {
  if (ranges_overlap(o.p, span(*o.v) * view_dt_bytes(o.v->dtype), p, bytes))
    return api_fail(HLO_ERR_INVALID_ARG, "%s overlaps %s", o.what, what);
  return HLO_OK;
}

// Merges the outer dimensions 0..last-1 of the views (absent ones NULL) into Rows.
template <int NV>
Rows<NV> merge_rows(const hlo_view* const (&views)[NV], int last) {
  Rows<NV> m;
  std::memset(&m, 0, sizeof m);
  const hlo_view& x = *views[0];
  for (int d = 0; d < last; ++d) {
    if (x.dims[d] == 1) continue;
    bool merge = m.n > 0;
    for (int v = 0; v < NV; ++v)
      if (views[v]) merge = merge && m.stride[v][m.n - 1] == views[v]->strides[d] * x.dims[d];
    const int at = merge ? m.n - 1 : m.n;
    m.size[at] = (merge ? m.size[at] : 1) * x.dims[d];
    for (int v = 0; v < NV; ++v) m.stride[v][at] = views[v] ? views[v]->strides[d] : 0;
    m.n = at + 1;
  }
  return m;
}

// `count`: the elements that are numbered.
hlo_status check_dropout(const hlo_dropout_params* d, int64_t count, DropPlan* out) {
  std::memset(out, 0, sizeof *out);
  if (!d) return HLO_OK;
  if (!(d->p >= 0.0 && d->p <= 1.0)) return api_fail(HLO_ERR_INVALID_ARG, "dropout: p = %g outside 0..1", d->p);
  if ((uintptr_t)d->state % 8 != 0) return api_fail(HLO_ERR_INVALID_ARG, "dropout: state is not 8-byte aligned");
  out->mode = d->state || count > (int64_t)1 << 34 ? DROP_DEVICE : DROP_HOST;
  const double threshold = std::floor(d->p * 4294967296.0 + 0.5);
  out->all = threshold >= 4294967296.0;
  out->threshold = out->all ? 0xFFFFFFFFu : (uint32_t)threshold;
  out->scale = d->p < 1.0 ? (float)(1.0 / (1.0 - d->p)) : 0.0f;
  out->seed = d->seed;
  out->offset = d->offset;
  out->state = d->state;
  philox_constants(out, d->seed, d->offset);
  return HLO_OK;
}

hlo_status check_weight(const void* w, int dtype, int x_dtype) {
  if (!w) return HLO_OK;
  if (dtype != x_dtype && dtype != HLO_F32)
    return api_fail(HLO_ERR_INVALID_ARG, "rms_norm: weight type %d is neither the input's nor f32", dtype);
  if ((uintptr_t)w % dt_bytes(dtype) != 0)
    return api_fail(HLO_ERR_INVALID_ARG, "rms_norm: weight is not aligned to its element type");
  return HLO_OK;
}

cudaStream_t as_stream(void* s) { return reinterpret_cast<cudaStream_t>(s); }

#define TRY(call)                     \
  do {                                \
    const hlo_status st_ = (call);    \
    if (st_ != HLO_OK) return st_;    \
  } while (0)
#define INJECT(site) \
  if (api_injected(site)) return api_fail(HLO_ERR_CUDA, "%s: injected fault (HLOFUSION_FAULT)", site)

}  // namespace

extern "C" {

hlo_status hlo_rms_norm(const hlo_view* x, const void* x_ptr, const hlo_view* residual, const void* residual_ptr,
                        const hlo_dropout_params* dropout, const void* weight_ptr, int32_t weight_dtype,
                        double weight_offset, double eps, const hlo_view* sum, void* sum_ptr, const hlo_view* out,
                        void* out_ptr, float* scales, const hlo_quant* out_q, float* rstd, void* stream) {
  TRY(check_view(x, x_ptr, "rms_norm x", false));
  if (!is_float(x->dtype)) return api_fail(HLO_ERR_UNSUPPORTED, "rms_norm x: element type %d not supported", x->dtype);
  const int64_t n = x->dims[x->rank - 1];
  if (n < 1) return api_fail(HLO_ERR_INVALID_ARG, "rms_norm x: the last dimension is empty");
  TRY(check_view(out, out_ptr, "rms_norm out", true));
  TRY(same_dims(*x, *out, "rms_norm out"));
  if (residual) {
    TRY(check_view(residual, residual_ptr, "rms_norm residual", false));
    TRY(same_dims(*x, *residual, "rms_norm residual"));
    if (residual->dtype != x->dtype)
      return api_fail(HLO_ERR_INVALID_ARG, "rms_norm residual: type %d differs from x's %d", residual->dtype, x->dtype);
  }
  if (sum) {
    TRY(check_view(sum, sum_ptr, "rms_norm sum", true));
    TRY(same_dims(*x, *sum, "rms_norm sum"));
    if (sum->dtype != x->dtype)
      return api_fail(HLO_ERR_INVALID_ARG, "rms_norm sum: type %d differs from x's %d", sum->dtype, x->dtype);
  }
  TRY(check_weight(weight_ptr, weight_dtype, x->dtype));
  if (!(eps >= 0.0) || !std::isfinite(eps)) return api_fail(HLO_ERR_INVALID_ARG, "rms_norm: eps must be finite and >= 0");
  NormPlan p;
  std::memset(&p, 0, sizeof p);
  TRY(check_dropout(dropout, numel(*x), &p.drop));
  const int od = out->dtype;
  if (scales) {
    if (od != HLO_S8 && od != HLO_F8E4M3FN)
      return api_fail(HLO_ERR_INVALID_ARG, "rms_norm: scales belong to an s8 or f8E4M3FN output, not type %d", od);
    if (out_q) return api_fail(HLO_ERR_INVALID_ARG, "rms_norm: scales and out_q exclude each other");
    p.quant = NQ_ROW;
  } else if (out_q) {
    if (od != HLO_S8) return api_fail(HLO_ERR_INVALID_ARG, "rms_norm: out_q belongs to an s8 output, not type %d", od);
    hlo_array a;
    std::memset(&a, 0, sizeof a);
    a.rank = out->rank;
    a.dtype = out->dtype;
    std::memcpy(a.dims, out->dims, sizeof a.dims);
    TRY(api_check_quant(out_q, a, "rms_norm out", &p.q));
    if (p.q.axis >= 0) return api_fail(HLO_ERR_UNSUPPORTED, "rms_norm out: static parameters must be per-tensor");
    p.quant = NQ_STATIC;
  } else if (od != x->dtype && od != HLO_F32) {
    return api_fail(HLO_ERR_INVALID_ARG, "rms_norm out: type %d needs to be x's, f32, or 8 bits with scales or out_q", od);
  }
  const int64_t rows = numel(*x) / n;
  const Operand ins[2] = {{x, x_ptr, "rms_norm x"}, {residual, residual_ptr, "rms_norm residual"}};
  const Operand outs[2] = {{out, out_ptr, "rms_norm out"}, {sum, sum_ptr, "rms_norm sum"}};
  for (const Operand& o : outs) {
    if (!o.v) continue;
    TRY(check_overlap(o, ins, 2, outs, 2));
    if (weight_ptr) TRY(check_side(o, weight_ptr, n * dt_bytes(weight_dtype), "the weight"));
    TRY(check_side(o, scales, rows * 4, "scales"));
    TRY(check_side(o, rstd, rows * 4, "rstd"));
    if (dropout) TRY(check_side(o, dropout->state, 16, "the generator's state"));
  }
  if (((uintptr_t)scales | (uintptr_t)rstd) % 4 != 0)
    return api_fail(HLO_ERR_INVALID_ARG, "rms_norm: scales and rstd must be 4-byte aligned");
  float* const side[2] = {scales, rstd};
  for (float* f : side) {
    if (!f) continue;
    for (const Operand& i : ins)
      if (i.v) TRY(check_side(i, f, rows * 4, "scales or rstd"));
    if (weight_ptr && ranges_overlap(f, rows * 4, weight_ptr, n * dt_bytes(weight_dtype)))
      return api_fail(HLO_ERR_INVALID_ARG, "rms_norm: scales or rstd overlaps the weight");
    if (dropout && ranges_overlap(f, rows * 4, dropout->state, 16))
      return api_fail(HLO_ERR_INVALID_ARG, "rms_norm: scales or rstd overlaps the generator's state");
  }
  if (ranges_overlap(scales, rows * 4, rstd, rows * 4)) return api_fail(HLO_ERR_INVALID_ARG, "rms_norm: scales overlaps rstd");
  if (rows == 0) return api_ok();
  p.x = x_ptr;
  p.res = residual ? residual_ptr : nullptr;
  p.w = weight_ptr;
  p.sum = sum ? sum_ptr : nullptr;
  p.out = out_ptr;
  p.scales = scales;
  p.rstd = rstd;
  p.rows = rows;
  p.n = n;
  p.dt = x->dtype;
  p.out_dt = od;
  p.w_dt = weight_dtype;
  p.w_offset = (float)weight_offset;
  p.eps = (float)eps;
  const hlo_view* const views[4] = {x, residual, sum, out};
  p.map = merge_rows<4>(views, x->rank - 1);
  INJECT("hlo_rms_norm");
  return api_cuda_status(launch_norm(p, as_stream(stream)), "rms_norm launch");
}

size_t hlo_rms_norm_workspace_size(int64_t rows, int64_t n) {
  if (rows <= 0 || n <= 0) return 0;
  return (size_t)(norm_grad_partials(rows, n) * n * 4);
}

hlo_status hlo_rms_norm_backward(const hlo_view* dy, const void* dy_ptr, const hlo_view* h, const void* h_ptr,
                                 const float* rstd, const void* weight_ptr, int32_t weight_dtype, double weight_offset,
                                 const hlo_view* dsum, const void* dsum_ptr, const hlo_dropout_params* dropout,
                                 const hlo_view* dh, void* dh_ptr, const hlo_view* dx, void* dx_ptr, float* dweight,
                                 void* workspace, size_t workspace_bytes, void* stream) {
  TRY(check_view(h, h_ptr, "rms_norm_backward h", false));
  if (!is_float(h->dtype))
    return api_fail(HLO_ERR_UNSUPPORTED, "rms_norm_backward h: element type %d not supported", h->dtype);
  const int64_t n = h->dims[h->rank - 1];
  if (n < 1) return api_fail(HLO_ERR_INVALID_ARG, "rms_norm_backward h: the last dimension is empty");
  const Operand all[5] = {{dy, dy_ptr, "rms_norm_backward dy"},
                          {h, h_ptr, "rms_norm_backward h"},
                          {dsum, dsum_ptr, "rms_norm_backward dsum"},
                          {dh, dh_ptr, "rms_norm_backward dh"},
                          {dx, dx_ptr, "rms_norm_backward dx"}};
  NormGradPlan p;
  std::memset(&p, 0, sizeof p);
  TRY(check_dropout(dropout, numel(*h), &p.drop));
  if ((dx != nullptr) != (dropout != nullptr))
    return api_fail(HLO_ERR_INVALID_ARG, "rms_norm_backward: dx goes with dropout (without it dx equals dh)");
  for (int k = 0; k < 5; ++k) {
    if (!all[k].v && (k == 2 || k == 4)) continue;
    TRY(check_view(all[k].v, all[k].p, all[k].what, k >= 3));
    TRY(same_dims(*h, *all[k].v, all[k].what));
    if (all[k].v->dtype != h->dtype)
      return api_fail(HLO_ERR_INVALID_ARG, "%s: type %d differs from h's %d", all[k].what, all[k].v->dtype, h->dtype);
  }
  TRY(check_weight(weight_ptr, weight_dtype, h->dtype));
  const int64_t rows = numel(*h) / n;
  if (rows > 0 && !rstd) return api_fail(HLO_ERR_INVALID_ARG, "rms_norm_backward: rstd is NULL");
  if (((uintptr_t)rstd | (uintptr_t)dweight) % 4 != 0)
    return api_fail(HLO_ERR_INVALID_ARG, "rms_norm_backward: rstd and dweight must be 4-byte aligned");
  const int64_t need = dweight ? (int64_t)hlo_rms_norm_workspace_size(rows, n) : 0;
  if (need > 0) {
    if (!workspace || (int64_t)workspace_bytes < need)
      return api_fail(HLO_ERR_WORKSPACE, "rms_norm_backward: workspace of %zu bytes, %lld needed (hlo_rms_norm_workspace_size)",
                      workspace ? workspace_bytes : (size_t)0, (long long)need);
    if ((uintptr_t)workspace % 16 != 0)
      return api_fail(HLO_ERR_INVALID_ARG, "rms_norm_backward: workspace is not 16-byte aligned");
  }
  for (int k = 3; k < 5; ++k) {
    if (!all[k].v) continue;
    TRY(check_overlap(all[k], all, 3, all + 3, 2));
    if (weight_ptr) TRY(check_side(all[k], weight_ptr, n * dt_bytes(weight_dtype), "the weight"));
    TRY(check_side(all[k], rstd, rows * 4, "rstd"));
    if (dropout) TRY(check_side(all[k], dropout->state, 16, "the generator's state"));
  }
  for (int k = 0; k < 5; ++k) {
    if (!all[k].v) continue;
    TRY(check_side(all[k], dweight, n * 4, "dweight"));
    TRY(check_side(all[k], workspace, need, "the workspace"));
  }
  if (ranges_overlap(dweight, n * 4, workspace, need) || ranges_overlap(dweight, n * 4, rstd, rows * 4) ||
      ranges_overlap(workspace, need, rstd, rows * 4) ||
      (weight_ptr && (ranges_overlap(dweight, n * 4, weight_ptr, n * dt_bytes(weight_dtype)) ||
                      ranges_overlap(workspace, need, weight_ptr, n * dt_bytes(weight_dtype)))))
    return api_fail(HLO_ERR_INVALID_ARG, "rms_norm_backward: dweight or the workspace overlaps another buffer");
  if (dropout && (ranges_overlap(dweight, n * 4, dropout->state, 16) || ranges_overlap(workspace, need, dropout->state, 16)))
    return api_fail(HLO_ERR_INVALID_ARG, "rms_norm_backward: dweight or the workspace overlaps the generator's state");
  INJECT("hlo_rms_norm_backward");
  if (rows == 0) {  // a sum over no rows
    if (!dweight) return api_ok();
    return api_cuda_status(launch_fill(dweight, F32, n, 0.0f, as_stream(stream)), "rms_norm_backward launch");
  }
  p.dy = dy_ptr;
  p.h = h_ptr;
  p.dsum = dsum ? dsum_ptr : nullptr;
  p.rstd = rstd;
  p.w = weight_ptr;
  p.dh = dh_ptr;
  p.dx = dx ? dx_ptr : nullptr;
  p.dw = dweight;
  p.ws = static_cast<float*>(workspace);
  p.rows = rows;
  p.n = n;
  p.dt = h->dtype;
  p.w_dt = weight_dtype;
  p.w_offset = (float)weight_offset;
  const hlo_view* const views[5] = {dy, h, dsum, dh, dx};
  p.map = merge_rows<5>(views, h->rank - 1);
  return api_cuda_status(launch_norm_grad(p, as_stream(stream)), "rms_norm_backward launch");
}

hlo_status hlo_dropout(const hlo_view* x, const void* x_ptr, const hlo_view* residual, const void* residual_ptr,
                       const hlo_dropout_params* dropout, const hlo_view* out, void* out_ptr, void* stream) {
  TRY(check_view(x, x_ptr, "dropout x", false));
  if (!is_float(x->dtype)) return api_fail(HLO_ERR_UNSUPPORTED, "dropout x: element type %d not supported", x->dtype);
  TRY(check_view(out, out_ptr, "dropout out", true));
  TRY(same_dims(*x, *out, "dropout out"));
  if (residual) {
    TRY(check_view(residual, residual_ptr, "dropout residual", false));
    TRY(same_dims(*x, *residual, "dropout residual"));
  }
  if (out->dtype != x->dtype || (residual && residual->dtype != x->dtype))
    return api_fail(HLO_ERR_INVALID_ARG, "dropout: x, residual and out must have one element type");
  DropoutPlan p;
  std::memset(&p, 0, sizeof p);
  if (!dropout) return api_fail(HLO_ERR_INVALID_ARG, "dropout: parameters are NULL");
  TRY(check_dropout(dropout, numel(*x), &p.drop));
  const Operand ins[2] = {{x, x_ptr, "dropout x"}, {residual, residual_ptr, "dropout residual"}};
  const Operand o = {out, out_ptr, "dropout out"};
  TRY(check_overlap(o, ins, 2, nullptr, 0));
  TRY(check_side(o, dropout->state, 16, "the generator's state"));
  if (numel(*x) == 0) return api_ok();
  p.x = x_ptr;
  p.res = residual ? residual_ptr : nullptr;
  p.out = out_ptr;
  p.dt = x->dtype;
  const hlo_view* const views[3] = {x, residual, out};
  p.map = merge_rows<3>(views, x->rank - 1);
  p.end[0] = end_of(x, x_ptr);
  p.end[1] = end_of(residual, residual_ptr);
  p.n = x->dims[x->rank - 1];
  p.rows = numel(*x) / p.n;
  // rows that follow one another in every view are one long row
  const int j = p.map.n - 1;
  if (j >= 0) {
    bool dense = true;
    for (int v = 0; v < 3; ++v)
      if (views[v]) dense = dense && p.map.stride[v][j] == p.n;
    if (dense) {
      p.n *= p.map.size[j];
      p.rows /= p.map.size[j];
      p.map.n = j;
    }
  }
  INJECT("hlo_dropout");
  return api_cuda_status(launch_dropout(p, as_stream(stream)), "dropout launch");
}

hlo_status hlo_rotary_turns(int32_t n_pairs, double base, int32_t scaling, double factor, double original_length,
                            double low, double high, uint64_t* turns) {
  if (n_pairs < 0) return api_fail(HLO_ERR_INVALID_ARG, "rotary_turns: n_pairs is negative");
  if (n_pairs > 0 && !turns) return api_fail(HLO_ERR_INVALID_ARG, "rotary_turns: NULL pointer");
  if (!(base >= 1.0) || !std::isfinite(base)) return api_fail(HLO_ERR_INVALID_ARG, "rotary_turns: base must be finite and >= 1");
  if (scaling < HLO_ROTARY_PLAIN || scaling > HLO_ROTARY_BY_PARTS)
    return api_fail(HLO_ERR_INVALID_ARG, "rotary_turns: unknown scaling %d", scaling);
  if (scaling != HLO_ROTARY_PLAIN && (!(factor >= 1.0) || !std::isfinite(factor)))
    return api_fail(HLO_ERR_INVALID_ARG, "rotary_turns: factor must be finite and >= 1");
  if (scaling == HLO_ROTARY_BASE && n_pairs == 1)
    return api_fail(HLO_ERR_INVALID_ARG, "rotary_turns: changing the base needs two pairs or more");
  if (scaling == HLO_ROTARY_BY_PARTS && !(original_length > 0.0 && std::isfinite(original_length) && low < high &&
                                          std::isfinite(low) && std::isfinite(high)))
    return api_fail(HLO_ERR_INVALID_ARG, "rotary_turns: by parts needs original_length > 0 and low < high");
  const double tau = 6.283185307179586476925286766559, rot = 2.0 * n_pairs;
  const double b = scaling == HLO_ROTARY_BASE ? base * std::pow(factor, rot / (rot - 2.0)) : base;
  for (int32_t i = 0; i < n_pairs; ++i) {
    double th = std::pow(b, -2.0 * i / rot);
    if (scaling == HLO_ROTARY_LINEAR) th /= factor;
    if (scaling == HLO_ROTARY_BY_PARTS) {
      const double w = original_length * th / tau;
      const double g = std::min(1.0, std::max(0.0, (w - low) / (high - low)));
      th *= g + (1.0 - g) / factor;
    }
    turns[i] = (uint64_t)std::ldexp(th / tau, 64);  // th <= 1: below 0.16 * 2^64
  }
  return api_ok();
}

hlo_status hlo_rotary(const hlo_view* x, const void* x_ptr, const hlo_view* x_out, void* x_out_ptr, const hlo_view* y,
                      const void* y_ptr, const hlo_view* y_out, void* y_out_ptr, const hlo_view* positions,
                      const int32_t* positions_ptr, const uint64_t* turns, int32_t n_pairs, int32_t interleaved,
                      int32_t inverse, double scale, void* stream) {
  TRY(check_view(x, x_ptr, "rotary x", false));
  if (!is_float(x->dtype)) return api_fail(HLO_ERR_UNSUPPORTED, "rotary x: element type %d not supported", x->dtype);
  if (x->rank != 3 && x->rank != 4)
    return api_fail(HLO_ERR_INVALID_ARG, "rotary x: rank %d, expected [batch,] seq, heads, dim", x->rank);
  if ((y == nullptr) != (y_out == nullptr)) return api_fail(HLO_ERR_INVALID_ARG, "rotary: y and y_out go together");
  TRY(check_view(x_out, x_out_ptr, "rotary x_out", true));
  TRY(same_dims(*x, *x_out, "rotary x_out"));
  const int lead = x->rank - 2;  // batch and seq, or seq
  if (y) {
    TRY(check_view(y, y_ptr, "rotary y", false));
    TRY(check_view(y_out, y_out_ptr, "rotary y_out", true));
    TRY(same_dims(*y, *y_out, "rotary y_out"));
    if (y->rank != x->rank) return api_fail(HLO_ERR_INVALID_ARG, "rotary y: rank differs from x's");
    for (int d = 0; d < x->rank; ++d)
      if (d != lead && y->dims[d] != x->dims[d])
        return api_fail(HLO_ERR_INVALID_ARG, "rotary y: dimension %d is %lld, x has %lld", d, (long long)y->dims[d],
                        (long long)x->dims[d]);
  }
  if (x_out->dtype != x->dtype || (y && (y->dtype != x->dtype || y_out->dtype != x->dtype)))
    return api_fail(HLO_ERR_INVALID_ARG, "rotary: the arrays must have one element type");
  TRY(check_view(positions, positions_ptr, "rotary positions", false));
  if (positions->dtype != HLO_S32) return api_fail(HLO_ERR_INVALID_ARG, "rotary positions: element type must be s32");
  if (positions->rank != lead) return api_fail(HLO_ERR_INVALID_ARG, "rotary positions: rank %d, expected %d", positions->rank, lead);
  for (int d = 0; d < lead; ++d)
    if (positions->dims[d] != x->dims[d])
      return api_fail(HLO_ERR_INVALID_ARG, "rotary positions: dimension %d is %lld, x has %lld", d,
                      (long long)positions->dims[d], (long long)x->dims[d]);
  const int64_t dim = x->dims[x->rank - 1];
  if (dim > (1 << 20)) return api_fail(HLO_ERR_UNSUPPORTED, "rotary x: heads of %lld elements", (long long)dim);
  if (n_pairs < 0 || 2 * (int64_t)n_pairs > dim)
    return api_fail(HLO_ERR_INVALID_ARG, "rotary: %d pairs in heads of %lld elements", n_pairs, (long long)dim);
  if (n_pairs > 0 && !turns) return api_fail(HLO_ERR_INVALID_ARG, "rotary: turns is NULL");
  if ((uintptr_t)turns % 8 != 0) return api_fail(HLO_ERR_INVALID_ARG, "rotary: turns is not 8-byte aligned");
  if (!std::isfinite(scale)) return api_fail(HLO_ERR_INVALID_ARG, "rotary: scale is not finite");
  const Operand own[2] = {{x, x_ptr, "rotary x"}, {y, y_ptr, "rotary y"}};
  const Operand outs[2] = {{x_out, x_out_ptr, "rotary x_out"}, {y_out, y_out_ptr, "rotary y_out"}};
  for (int k = 0; k < 2; ++k) {
    if (!outs[k].v) continue;
    // an array may be rotated in place, but not onto the other one's input
    TRY(check_overlap(outs[k], own + k, 1, outs, 2));
    const Operand other[1] = {own[1 - k]};
    TRY(check_overlap(outs[k], nullptr, 0, other, 1));
    TRY(check_side(outs[k], positions_ptr, span(*positions) * 4, "the positions"));
    TRY(check_side(outs[k], turns, (int64_t)n_pairs * 8, "turns"));
  }
  RotaryPlan p;
  std::memset(&p, 0, sizeof p);
  p.batch = lead == 2 ? x->dims[0] : 1;
  p.seq = x->dims[lead - 1];
  p.dim = (int)dim;
  p.pairs = n_pairs;
  p.dt = x->dtype;
  p.interleaved = interleaved ? 1 : 0;
  p.pos = positions_ptr;
  p.pos_stride[0] = lead == 2 ? positions->strides[0] : 0;
  p.pos_stride[1] = positions->strides[lead - 1];
  p.turns = turns;
  p.scale = (float)scale;
  p.sin_scale = inverse ? -p.scale : p.scale;
  const hlo_view* const vi[2] = {x, y};
  const hlo_view* const vo[2] = {x_out, y_out};
  const void* const pi[2] = {x_ptr, y_ptr};
  void* const po[2] = {x_out_ptr, y_out_ptr};
  for (int k = 0; k < 2; ++k) {
    if (!vi[k] || numel(*vi[k]) == 0) continue;
    RotaryArray& a = p.a[p.arrays++];
    a.in = pi[k];
    a.out = po[k];
    a.heads = vi[k]->dims[lead];
    for (int s = 0; s < 3; ++s) {
      const int d = lead - 2 + s;  // batch, seq, head
      a.in_stride[s] = d >= 0 ? vi[k]->strides[d] : 0;
      a.out_stride[s] = d >= 0 ? vo[k]->strides[d] : 0;
    }
  }
  if (p.arrays == 0) return api_ok();
  INJECT("hlo_rotary");
  return api_cuda_status(launch_rotary(p, as_stream(stream)), "rotary launch");
}

hlo_status hlo_logits_process(const hlo_view* logits, const void* logits_ptr, const hlo_view* bias, const float* bias_ptr,
                              const hlo_view* history, const int32_t* history_ptr, const int32_t* lengths,
                              const int32_t* prompt_lengths, const float* repetition, const float* frequency,
                              const float* presence, const hlo_view* mask, const int32_t* mask_ptr, const hlo_view* out,
                              void* out_ptr, int32_t* token, void* stream) {
  TRY(check_view(logits, logits_ptr, "logits", false));
  if (!is_float(logits->dtype)) return api_fail(HLO_ERR_UNSUPPORTED, "logits: element type %d not supported", logits->dtype);
  if (logits->rank != 2) return api_fail(HLO_ERR_INVALID_ARG, "logits: rank %d, expected [batch, vocab]", logits->rank);
  const int64_t b = logits->dims[0], v = logits->dims[1];
  if (v > INT32_MAX || b > INT32_MAX / 8)
    return api_fail(HLO_ERR_UNSUPPORTED, "logits: %lld rows of %lld tokens", (long long)b, (long long)v);
  if (!out && !token) return api_fail(HLO_ERR_INVALID_ARG, "logits: neither out nor token is wanted");
  LogitsPlan p;
  std::memset(&p, 0, sizeof p);
  const int64_t words = (v + 31) / 32;
  struct Side {
    const hlo_view* v;
    const void* p;
    int dtype;
    int64_t cols;
    const char* what;
  } const sides[3] = {{bias, bias_ptr, HLO_F32, v, "logits bias"},
                      {history, history_ptr, HLO_S32, -1, "logits history"},
                      {mask, mask_ptr, HLO_S32, words, "logits mask"}};
  for (const Side& s : sides) {
    if (!s.v) continue;
    TRY(check_view(s.v, s.p, s.what, false));
    if (s.v->dtype != s.dtype) return api_fail(HLO_ERR_INVALID_ARG, "%s: element type must be %s", s.what, s.dtype == HLO_F32 ? "f32" : "s32");
    if (s.v->rank != 2 || s.v->dims[0] != b || (s.cols >= 0 && s.v->dims[1] != s.cols))
      return api_fail(HLO_ERR_INVALID_ARG, "%s: shape must be [%lld, %lld]", s.what, (long long)b,
                      (long long)(s.cols >= 0 ? s.cols : s.v->rank == 2 ? s.v->dims[1] : 0));
  }
  if (history && history->dims[1] > INT32_MAX) return api_fail(HLO_ERR_UNSUPPORTED, "logits history: %lld entries", (long long)history->dims[1]);
  const void* const vectors[6] = {lengths, prompt_lengths, repetition, frequency, presence, token};
  for (const void* q : vectors)
    if ((uintptr_t)q % 4 != 0) return api_fail(HLO_ERR_INVALID_ARG, "logits: a per-row vector is not 4-byte aligned");
  if (!history && (lengths || prompt_lengths || repetition || frequency || presence))
    return api_fail(HLO_ERR_INVALID_ARG, "logits: lengths and penalties need a history");
  if (out) {
    TRY(check_view(out, out_ptr, "logits out", true));
    TRY(same_dims(*logits, *out, "logits out"));
    if (out->dtype != logits->dtype && out->dtype != HLO_F32)
      return api_fail(HLO_ERR_INVALID_ARG, "logits out: type %d is neither the logits' nor f32", out->dtype);
    const Operand o = {out, out_ptr, "logits out"};
    const Operand in[1] = {{logits, logits_ptr, "logits"}};
    const Operand rest[3] = {{bias, bias_ptr, "the bias"}, {history, history_ptr, "the history"}, {mask, mask_ptr, "the mask"}};
    TRY(check_overlap(o, in, 1, rest, 3));
    for (const void* q : vectors) TRY(check_side(o, q, b * 4, "a per-row vector"));
  }
  if (token) {
    const Operand ins[4] = {{logits, logits_ptr, "logits"}, {bias, bias_ptr, "the bias"}, {history, history_ptr, "the history"},
                            {mask, mask_ptr, "the mask"}};
    for (const Operand& i : ins)
      if (i.v) TRY(check_side(i, token, b * 4, "token"));
    for (int k = 0; k < 5; ++k)
      if (ranges_overlap(token, b * 4, vectors[k], b * 4)) return api_fail(HLO_ERR_INVALID_ARG, "logits: token overlaps a per-row vector");
  }
  if (b == 0 || (v == 0 && !token)) return api_ok();
  p.x = logits_ptr;
  p.x_end = end_of(logits, logits_ptr);
  p.out = out ? out_ptr : nullptr;
  p.token = token;
  p.batch = b;
  p.vocab = v;
  p.x_stride = b > 1 ? logits->strides[0] : 0;
  p.out_stride = out && b > 1 ? out->strides[0] : 0;
  p.dt = logits->dtype;
  p.out_dt = out ? out->dtype : logits->dtype;
  p.bias = bias ? bias_ptr : nullptr;
  p.bias_stride = bias && b > 1 ? bias->strides[0] : 0;
  if (history && history->dims[1] > 0) {
    p.history = history_ptr;
    p.history_stride = b > 1 ? history->strides[0] : 0;
    p.max_length = history->dims[1];
    p.lengths = lengths;
    p.prompts = prompt_lengths;
    p.repetition = repetition;
    p.frequency = frequency;
    p.presence = presence;
  }
  p.mask = mask ? reinterpret_cast<const uint32_t*>(mask_ptr) : nullptr;
  p.mask_stride = mask && b > 1 ? mask->strides[0] : 0;
  INJECT("hlo_logits_process");
  return api_cuda_status(launch_logits(p, as_stream(stream)), "logits launch");
}

}  // extern "C"
