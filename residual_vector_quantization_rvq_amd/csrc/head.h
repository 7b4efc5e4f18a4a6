// head.h -- arguments and launchers of the head of a model: the layer norm, the
// 8-bit product and its quantiser, log probabilities and the distillation loss.
#pragma once

#include "learn.h"

namespace rvq {

struct LayerNormArgs {
  const void *x, *residual;     // residual may be null
  const void *weight, *bias;    // either may be null: ones, zeros
  bool w_bf16;                  // weight and bias
  void *sum, *y;                // sum may be null
  int y_type;                   // rvq_dtype
  float *scale, *mean, *rstd;   // scale: 8-bit output only; mean and rstd may be null
  int64_t n;
  int d;
  float eps;
};
hipError_t launch_layer_norm(const LayerNormArgs &a, bool x_bf16, hipStream_t s);

struct LayerNormGradArgs {
  const void *dy, *h, *dsum;    // dsum may be null
  const float *mean, *rstd;
  const void *weight;           // null: ones
  bool w_bf16;
  void *dx;
  float *dweight, *dbias;       // either may be null
  float *part;                  // [layer_norm_grad_parts(n, d, bf16)][2][d]: dweight's parts, dbias'
  int64_t n;
  int d;
};
int64_t layer_norm_grad_parts(int64_t n, int d, bool bf16);
hipError_t launch_layer_norm_grad(const LayerNormGradArgs &a, bool bf16, hipStream_t s);

// 8-bit operands: one scale for kScaleBlock elements along the contracted axis.
constexpr int kScaleBlock = 128;
struct QuantArgs {
  const void *x;                // [rows][cols]
  int64_t rows, cols;
  uint8_t *q;                   // [rows][cols], or [cols][rows] transposed, with row stride q_stride
  int64_t q_stride;
  float *scale;                 // by the rows of q: [rows][ceil(cols / 128)], or 128 x 128 blocks
  bool block_rows;              // 128 x 128 blocks
  bool transpose;
};
hipError_t launch_quantize_f8(const QuantArgs &a, bool x_bf16, hipStream_t s);

// A scale's place: scale[(row >> shift) * row_stride + block * block_stride]
struct ScaleView {
  const float *p;
  int64_t row_stride;
  int shift, block_stride;
};
struct MatmulArgs {
  const uint8_t *a, *b;         // [m][k], [n][k] e4m3 with row strides
  int64_t a_stride, b_stride;
  ScaleView sa, sb;
  int64_t m, n, k;
  void *out;                    // [m][n]
  bool out_bf16;
};
hipError_t launch_matmul_f8(const MatmulArgs &a, hipStream_t s);

// ---- rows of logits ----
constexpr int kMaxTop = 64;
struct LogprobArgs {
  const void *x;                // [n][V]
  int64_t n;
  int V;
  const int32_t *ids;           // [n]; null: no token's log probability is asked for
  float inv_t;                  // 1 / temperature
  float *logprob, *entropy;     // entropy may be null
  float *stats;                 // [n][2]: the largest logit, log of sum exp((x - largest) / T)
  float *top_logprob;           // [n][top]
  int32_t *top_ids;
  int top;
  uint32_t *bad;                // may be null
  float *part;                  // workspace of a split row
};
struct LogprobPlan {
  int slices;                   // workgroups per row
  int64_t slice;                // columns of each, a multiple of 8
};
LogprobPlan logprob_plan(int64_t n, int V, int top, bool bf16);
size_t logprob_part_floats(int64_t n, const LogprobPlan &p, int top);
hipError_t launch_logprobs(const LogprobArgs &a, bool x_bf16, hipStream_t s);

struct LogprobGradArgs {
  const void *x;
  int64_t n;
  int V;
  const int32_t *ids;
  float inv_t;
  const float *stats, *entropy; // entropy: with dentropy
  const float *dlogprob, *dentropy;  // either may be null
  void *dx;                     // [n][V], may be x
};
hipError_t launch_logprobs_grad(const LogprobGradArgs &a, bool x_bf16, hipStream_t s);

constexpr int kMaxTeacher = 256;
struct DistillArgs {
  const void *x;                // [n][V]
  int64_t n;
  int V;
  const int32_t *ids;           // [n][k]
  const float *teacher;         // [n][k]
  int k;
  bool tail;
  float inv_t;
  float *loss, *stats;          // [n], [n][4]: the largest logit, log S, and of tokens outside the teacher's
  uint32_t *bad;                // may be null
  const float *dloss;           // gradient
  void *dx;                     // gradient: [n][V], may be x
};
hipError_t launch_distill(const DistillArgs &a, bool x_bf16, hipStream_t s);
hipError_t launch_distill_grad(const DistillArgs &a, bool x_bf16, hipStream_t s);

}  // namespace rvq
