// Plans of the fusions between a decoder's matrix products (k_norm.cu, k_dropout.cu, k_rotary.cu,
// k_logits.cu): plain data passed to the kernels by value, and their launchers.
#pragma once
#include "hlo_internal.h"

namespace hlo {

constexpr int F8 = 5;  // HLO_F8E4M3FN: an output type of hlo_rms_norm only

inline __host__ __device__ int view_dt_bytes(int dt) { return dt == F8 ? 1 : dt_bytes(dt); }

// The outer dimensions that up to NV views share, merged where every view allows it (major first):
// row k of view v starts at offset sum_j ((k / inner_j) % size_j) * stride[v][j] elements. A stride is 0 in
// views that are absent.
template <int NV>
struct Rows {
  int n;
  int64_t size[kMaxRank];
  int64_t stride[NV][kMaxRank];
};

template <int NV>
__host__ __device__ inline void row_offsets(const Rows<NV>& m, int64_t k, int64_t (&off)[NV]) {
  for (int v = 0; v < NV; ++v) off[v] = 0;
  for (int j = m.n - 1; j > 0; --j) {
    const int64_t q = k / m.size[j], i = k - q * m.size[j];
    for (int v = 0; v < NV; ++v) off[v] += i * m.stride[v][j];
    k = q;
  }
  if (m.n > 0)
    for (int v = 0; v < NV; ++v) off[v] += k * m.stride[v][0];
}

// The generator's key and counter words (philox.cuh) and the keep rule: keep iff word >= threshold, or
// nothing at all (`all`: round(p 2^32) = 2^32). DROP_HOST: seed and offset are known on the host and every
// element's index is below 2^34, so a counter's high words are the same for all elements; what the first three
// rounds make of them, and the rounds' keys, are then constants. DROP_DEVICE: anything else.
enum DropMode : int { DROP_NONE = 0, DROP_HOST = 1, DROP_DEVICE = 2 };
struct DropPlan {
  int mode, all;
  uint32_t threshold;
  float scale;              // f32(1 / (1 - p))
  const uint64_t* state;    // DROP_DEVICE: seed and offset on the device, or NULL
  uint64_t seed, offset;    // DROP_DEVICE: the offset is added to the device's, if there is one
  uint32_t key[20];         // DROP_HOST: round r uses key[2 r], key[2 r + 1]
  uint32_t x1, y2, x2, y3;  // DROP_HOST: constants of the first rounds (philox_constants)
};

enum NormQuant : int { NQ_NONE = 0, NQ_ROW = 1, NQ_STATIC = 2 };

struct NormPlan {
  const void* x;
  const void* res;
  const void* w;
  void* sum;
  void* out;
  float* scales;
  float* rstd;
  int64_t rows, n;
  int dt, out_dt, w_dt;
  float w_offset, eps;
  int quant;          // NormQuant
  QuantParams q;      // NQ_STATIC
  DropPlan drop;
  Rows<4> map;        // x, residual, sum, out
};
cudaError_t launch_norm(const NormPlan& p, cudaStream_t s);

struct NormGradPlan {
  const void* dy;
  const void* h;
  const void* dsum;
  const float* rstd;
  const void* w;
  void* dh;
  void* dx;
  float* dw;
  float* ws;          // partials of dweight, [norm_grad_partials(rows, n)][n]
  int64_t rows, n;
  int dt, w_dt;
  float w_offset;
  DropPlan drop;
  Rows<5> map;        // dy, h, dsum, dh, dx
};
// Row groups whose shares of dweight are summed apart (each one row of n f32 in the workspace).
int64_t norm_grad_partials(int64_t rows, int64_t n);
cudaError_t launch_norm_grad(const NormGradPlan& p, cudaStream_t s);

struct DropoutPlan {
  const void* x;
  const void* res;
  void* out;
  int64_t rows, n;
  int dt;
  DropPlan drop;
  Rows<3> map;        // x, residual, out
  const char* end[2]; // of x and residual
};
cudaError_t launch_dropout(const DropoutPlan& p, cudaStream_t s);

struct RotaryArray {
  const void* in;
  void* out;
  int64_t heads;
  int64_t in_stride[3], out_stride[3];  // batch, seq, head
};
struct RotaryPlan {
  RotaryArray a[2];
  int arrays;
  int64_t batch, seq;
  int dim, pairs;
  int dt, interleaved;
  const int32_t* pos;
  int64_t pos_stride[2];
  const uint64_t* turns;
  float scale, sin_scale;  // sin_scale = -scale for the inverse
};
cudaError_t launch_rotary(const RotaryPlan& p, cudaStream_t s);

struct LogitsPlan {
  const void* x;
  const char* x_end;
  void* out;
  int32_t* token;
  int64_t batch, vocab;
  int64_t x_stride, out_stride;
  int dt, out_dt;
  const float* bias;
  int64_t bias_stride;
  const int32_t* history;
  int64_t history_stride, max_length;
  const int32_t* lengths;
  const int32_t* prompts;
  const float* repetition;
  const float* frequency;
  const float* presence;
  const uint32_t* mask;
  int64_t mask_stride;
};
cudaError_t launch_logits(const LogitsPlan& p, cudaStream_t s);

}  // namespace hlo
