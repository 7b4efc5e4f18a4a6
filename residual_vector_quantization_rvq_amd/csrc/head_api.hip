// head_api.hip -- the part of the C ABI (include/rvq.h) for the head of a model:
// the layer norm, the 8-bit product and its quantiser, log probabilities and the
// distillation loss.  Host side only: arguments are checked before any HIP call,
// workspaces are laid out, launches go to the caller's stream.
#include <cmath>

#include "head.h"

using namespace rvq;

namespace {

constexpr int64_t kMaxRows = (int64_t)1 << 25;
constexpr int kMaxWidth = 1 << 20;
constexpr int kMaxVocab = 1 << 24;
constexpr int64_t kMaxSide = (int64_t)1 << 30, kMaxArea = (int64_t)1 << 40;
// of a product: its workgroups stay under 2^32 work-items
constexpr int64_t kMaxMatmulRows = (int64_t)1 << 27, kMaxMatmulArea = (int64_t)1 << 36;

rvq_status need(const void *p, const char *name, size_t align) {
  if (!p) return fail(RVQ_ERR_INVALID_ARGUMENT, "%s must not be NULL", name);
  if (!at_multiple(p, align))
    return fail(RVQ_ERR_INVALID_ARGUMENT, "%s must be %zu-byte aligned", name, align);
  return RVQ_OK;
}
rvq_status may(const void *p, const char *name, size_t align) {
  return p ? need(p, name, align) : RVQ_OK;
}

#define RVQ_TRY(expr)              \
  do {                             \
    rvq_status _st = (expr);       \
    if (_st != RVQ_OK) return _st; \
  } while (0)

rvq_status launched(hipError_t e, const char *what) {
  return e == hipSuccess ? RVQ_OK : fail(RVQ_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
}

rvq_status check_rows(int64_t n, int32_t d, const char *width, int most) {
  if (n < 0) return fail(RVQ_ERR_INVALID_ARGUMENT, "n must be >= 0 (got %lld)", (long long)n);
  if (d < 1) return fail(RVQ_ERR_INVALID_ARGUMENT, "%s must be >= 1 (got %d)", width, d);
  if (n > kMaxRows)
    return fail(RVQ_ERR_UNSUPPORTED, "n above %lld rows per call (got %lld)", (long long)kMaxRows, (long long)n);
  if (d > most) return fail(RVQ_ERR_UNSUPPORTED, "%s above %d (got %d)", width, most, d);
  return RVQ_OK;
}
rvq_status check_dtype(rvq_dtype t, const char *name) {
  return float_or_bf16(t) ? RVQ_OK : fail(RVQ_ERR_INVALID_ARGUMENT, "unknown %s %d", name, (int)t);
}
rvq_status check_temperature(float t) {
  if (!(t >= 1e-4f && t <= 1e4f))
    return fail(RVQ_ERR_INVALID_ARGUMENT, "temperature must be within 1e-4 .. 1e4 (got %g)", (double)t);
  return RVQ_OK;
}

rvq_status view_of(const float *scale, rvq_scale_layout layout, int64_t k, const char *name, ScaleView *v) {
  const int64_t blocks = ceil_div(k, kScaleBlock);
  if (layout == RVQ_SCALE_ROW)
    *v = {scale, 1, 0, 0};
  else if (layout == RVQ_SCALE_ROW_128)
    *v = {scale, blocks, 0, 1};
  else if (layout == RVQ_SCALE_128_128)
    *v = {scale, blocks, 7, 1};
  else
    return fail(RVQ_ERR_INVALID_ARGUMENT, "unknown %s %d", name, (int)layout);
  return RVQ_OK;
}

// the gradients' output: the logits' own memory, or clear of it
rvq_status check_in_place(const void *x, const void *dx, int64_t bytes) {
  const char *p = (const char *)x, *q = (const char *)dx;
  if (p != q && p < q + bytes && q < p + bytes)
    return fail(RVQ_ERR_INVALID_ARGUMENT, "dlogits must be logits itself or not overlap it");
  return RVQ_OK;
}

}  // namespace

extern "C" {

rvq_status rvq_layer_norm(const void *x, const void *residual, rvq_dtype x_dtype, int64_t n,
                          int32_t d, const void *weight, const void *bias, rvq_dtype weight_dtype,
                          float eps, void *sum_out, void *y, rvq_dtype y_dtype, float *y_scale,
                          float *mean, float *rstd, hipStream_t stream) {
  RVQ_TRY(check_rows(n, d, "d", kMaxWidth));
  RVQ_TRY(check_dtype(x_dtype, "x_dtype"));
  if (!float_or_bf16(y_dtype) && y_dtype != RVQ_F8E4M3)
    return fail(RVQ_ERR_INVALID_ARGUMENT, "unknown y_dtype %d", (int)y_dtype);
  if (!(eps > 0.f) || !std::isfinite(eps))
    return fail(RVQ_ERR_INVALID_ARGUMENT, "eps must be positive and finite (got %g)", (double)eps);
  if (weight || bias) RVQ_TRY(check_dtype(weight_dtype, "weight_dtype"));
  RVQ_TRY(may(weight, "weight", dtype_bytes(weight_dtype)));
  RVQ_TRY(may(bias, "bias", dtype_bytes(weight_dtype)));
  if (n == 0) return RVQ_OK;
  const size_t xs = dtype_bytes(x_dtype);
  RVQ_TRY(need(x, "x", xs));
  RVQ_TRY(may(residual, "residual", xs));
  RVQ_TRY(may(sum_out, "sum_out", xs));
  RVQ_TRY(need(y, "y", dtype_bytes(y_dtype)));
  if (sum_out == y)
    return fail(RVQ_ERR_INVALID_ARGUMENT, "sum_out and y must not be the same memory");
  if (y_dtype == RVQ_F8E4M3) RVQ_TRY(need(y_scale, "y_scale", 4));
  RVQ_TRY(may(mean, "mean", 4));
  RVQ_TRY(may(rstd, "rstd", 4));
  const LayerNormArgs a = {x, residual, weight, bias, weight_dtype == RVQ_BF16, sum_out, y, (int)y_dtype,
                           y_scale, mean, rstd, n, d, eps};
  return launched(launch_layer_norm(a, x_dtype == RVQ_BF16, stream), "layer norm launch");
}

rvq_status rvq_layer_norm_backward_workspace_size(int64_t n, int32_t d, size_t *bytes) {
  RVQ_TRY(check_rows(n, d, "d", kMaxWidth));
  if (!bytes) return fail(RVQ_ERR_INVALID_ARGUMENT, "bytes must not be NULL");
  const int64_t p32 = layer_norm_grad_parts(n, d, false), p16 = layer_norm_grad_parts(n, d, true);
  *bytes = al256((size_t)(p32 > p16 ? p32 : p16) * 2 * (size_t)d * sizeof(float));
  return RVQ_OK;
}

rvq_status rvq_layer_norm_backward(const void *dy, const void *h, rvq_dtype dtype, int64_t n,
                                   int32_t d, const float *mean, const float *rstd,
                                   const void *weight, rvq_dtype weight_dtype, const void *dsum,
                                   void *dx, float *dweight, float *dbias, void *workspace,
                                   size_t workspace_bytes, hipStream_t stream) {
  RVQ_TRY(check_rows(n, d, "d", kMaxWidth));
  RVQ_TRY(check_dtype(dtype, "dtype"));
  if (weight) {
    RVQ_TRY(check_dtype(weight_dtype, "weight_dtype"));
    RVQ_TRY(need(weight, "weight", dtype_bytes(weight_dtype)));
  }
  const size_t xs = dtype_bytes(dtype);
  if (n > 0) {
    RVQ_TRY(need(dy, "dy", xs));
    RVQ_TRY(need(h, "h", xs));
    RVQ_TRY(need(mean, "mean", 4));
    RVQ_TRY(need(rstd, "rstd", 4));
    RVQ_TRY(may(dsum, "dsum", xs));
    RVQ_TRY(need(dx, "dx", xs));
  }
  if (dweight || dbias) {
    RVQ_TRY(may(dweight, "dweight", 4));
    RVQ_TRY(may(dbias, "dbias", 4));
    size_t want = 0;
    RVQ_TRY(rvq_layer_norm_backward_workspace_size(n, d, &want));
    RVQ_TRY(need(workspace, "workspace", 256));
    if (workspace_bytes < want)
      return fail(RVQ_ERR_WORKSPACE_TOO_SMALL, "norm gradient workspace needs %zu bytes (got %zu)", want,
                  workspace_bytes);
  } else if (n == 0) {
    return RVQ_OK;
  }
  const LayerNormGradArgs a = {dy, h, dsum, mean, rstd, weight, weight_dtype == RVQ_BF16, dx, dweight, dbias,
                               (float *)workspace, n, d};
  return launched(launch_layer_norm_grad(a, dtype == RVQ_BF16, stream), "layer norm gradient launch");
}

rvq_status rvq_quantize_f8(const void *x, rvq_dtype x_dtype, int64_t rows, int64_t cols,
                           rvq_scale_layout layout, int32_t transpose, void *q, int64_t q_stride,
                           float *scale, hipStream_t stream) {
  if (rows < 0 || cols < 0)
    return fail(RVQ_ERR_INVALID_ARGUMENT, "rows and cols must be >= 0 (got %lld, %lld)", (long long)rows,
                (long long)cols);
  if (rows > kMaxSide || cols > kMaxSide || rows * cols > kMaxArea)
    return fail(RVQ_ERR_UNSUPPORTED, "rows or cols above 2^30, or rows cols above 2^40 (got %lld, %lld)",
                (long long)rows, (long long)cols);
  RVQ_TRY(check_dtype(x_dtype, "x_dtype"));
  if (layout != RVQ_SCALE_ROW_128 && layout != RVQ_SCALE_128_128)
    return fail(RVQ_ERR_INVALID_ARGUMENT, "layout must be RVQ_SCALE_ROW_128 or RVQ_SCALE_128_128 (got %d)",
                (int)layout);
  if (rows == 0 || cols == 0) return RVQ_OK;
  RVQ_TRY(need(x, "x", dtype_bytes(x_dtype)));
  RVQ_TRY(need(q, "q", 1));
  RVQ_TRY(need(scale, "scale", 4));
  if (q_stride < (transpose ? rows : cols))
    return fail(RVQ_ERR_INVALID_ARGUMENT, "q_stride must be at least a row of q (got %lld)", (long long)q_stride);
  const QuantArgs a = {x, rows, cols, (uint8_t *)q, q_stride, scale, layout == RVQ_SCALE_128_128, transpose != 0};
  return launched(launch_quantize_f8(a, x_dtype == RVQ_BF16, stream), "quantiser launch");
}

rvq_status rvq_matmul_f8(const void *a, int64_t a_stride, const float *a_scale,
                         rvq_scale_layout a_layout, const void *b, int64_t b_stride,
                         const float *b_scale, rvq_scale_layout b_layout, int64_t m, int64_t n,
                         int64_t k, void *out, rvq_dtype out_dtype, hipStream_t stream) {
  if (m < 0 || n < 0 || k < 0)
    return fail(RVQ_ERR_INVALID_ARGUMENT, "m, n and k must be >= 0 (got %lld, %lld, %lld)", (long long)m, (long long)n,
                (long long)k);
  if (m > kMaxMatmulRows || n > kMaxMatmulRows || k > kMaxSide || m * n > kMaxMatmulArea)
    return fail(RVQ_ERR_UNSUPPORTED, "m or n above 2^27, k above 2^30, or m n above 2^36 (got %lld, %lld, %lld)",
                (long long)m, (long long)n, (long long)k);
  RVQ_TRY(check_dtype(out_dtype, "out_dtype"));
  MatmulArgs r;
  RVQ_TRY(view_of(a_scale, a_layout, k, "a_layout", &r.sa));
  RVQ_TRY(view_of(b_scale, b_layout, k, "b_layout", &r.sb));
  if (m == 0 || n == 0) return RVQ_OK;
  RVQ_TRY(need(out, "out", dtype_bytes(out_dtype)));
  if (k > 0) {
    RVQ_TRY(need(a, "a", 1));
    RVQ_TRY(need(b, "b", 1));
    RVQ_TRY(need(a_scale, "a_scale", 4));
    RVQ_TRY(need(b_scale, "b_scale", 4));
    if (a_stride < k || b_stride < k)
      return fail(RVQ_ERR_INVALID_ARGUMENT, "a_stride and b_stride must be at least k (got %lld, %lld)",
                  (long long)a_stride, (long long)b_stride);
  }
  r.a = (const uint8_t *)a;
  r.b = (const uint8_t *)b;
  r.a_stride = a_stride;
  r.b_stride = b_stride;
  r.m = m;
  r.n = n;
  r.k = k;
  r.out = out;
  r.out_bf16 = out_dtype == RVQ_BF16;
  return launched(launch_matmul_f8(r, stream), "8-bit product launch");
}

rvq_status rvq_token_logprobs_workspace_size(int64_t n, int32_t V, int32_t top, size_t *bytes) {
  RVQ_TRY(check_rows(n, V, "V", kMaxVocab));
  if (top < 0 || top > kMaxTop)
    return fail(RVQ_ERR_INVALID_ARGUMENT, "top must be within 0 .. %d (got %d)", kMaxTop, top);
  if (!bytes) return fail(RVQ_ERR_INVALID_ARGUMENT, "bytes must not be NULL");
  size_t floats = 0;
  if (n > 0)
    for (const bool bf16 : {false, true}) {
      const size_t f = logprob_part_floats(n, logprob_plan(n, V, top, bf16), top);
      if (f > floats) floats = f;
    }
  *bytes = al256(floats * sizeof(float));
  return RVQ_OK;
}

rvq_status rvq_token_logprobs(const void *logits, rvq_dtype dtype, int64_t n, int32_t V,
                              const int32_t *ids, float temperature, float *logprob,
                              float *entropy, float *stats, int32_t top, float *top_logprob,
                              int32_t *top_ids, uint32_t *bad_ids, void *workspace,
                              size_t workspace_bytes, hipStream_t stream) {
  size_t want = 0;
  RVQ_TRY(rvq_token_logprobs_workspace_size(n, V, top, &want));
  RVQ_TRY(check_dtype(dtype, "dtype"));
  RVQ_TRY(check_temperature(temperature));
  if (n == 0) return RVQ_OK;
  RVQ_TRY(need(logits, "logits", dtype_bytes(dtype)));
  RVQ_TRY(may(ids, "ids", 4));
  if (ids) RVQ_TRY(need(logprob, "logprob", 4));
  RVQ_TRY(may(entropy, "entropy", 4));
  RVQ_TRY(need(stats, "stats", 4));
  if (top > 0) {
    RVQ_TRY(need(top_logprob, "top_logprob", 4));
    RVQ_TRY(need(top_ids, "top_ids", 4));
  }
  RVQ_TRY(may(bad_ids, "bad_ids", 4));
  if (want > 0) {
    RVQ_TRY(need(workspace, "workspace", 256));
    if (workspace_bytes < want)
      return fail(RVQ_ERR_WORKSPACE_TOO_SMALL, "log probability workspace needs %zu bytes (got %zu)", want,
                  workspace_bytes);
  }
  const LogprobArgs a = {logits, n, V, ids, 1.f / temperature, logprob, entropy, stats, top_logprob, top_ids, top,
                         bad_ids, (float *)workspace};
  return launched(launch_logprobs(a, dtype == RVQ_BF16, stream), "log probability launch");
}

rvq_status rvq_token_logprobs_backward(const void *logits, rvq_dtype dtype, int64_t n, int32_t V,
                                       const int32_t *ids, float temperature, const float *stats,
                                       const float *dlogprob, const float *entropy,
                                       const float *dentropy, void *dlogits, hipStream_t stream) {
  RVQ_TRY(check_rows(n, V, "V", kMaxVocab));
  RVQ_TRY(check_dtype(dtype, "dtype"));
  RVQ_TRY(check_temperature(temperature));
  if (n == 0) return RVQ_OK;
  RVQ_TRY(need(logits, "logits", dtype_bytes(dtype)));
  RVQ_TRY(need(stats, "stats", 4));
  RVQ_TRY(need(dlogits, "dlogits", dtype_bytes(dtype)));
  RVQ_TRY(check_in_place(logits, dlogits, n * V * (int64_t)dtype_bytes(dtype)));
  if (!dlogprob && !dentropy)
    return fail(RVQ_ERR_INVALID_ARGUMENT, "dlogprob and dentropy must not both be NULL");
  if (dlogprob) {
    RVQ_TRY(need(dlogprob, "dlogprob", 4));
    RVQ_TRY(need(ids, "ids", 4));
  }
  if (dentropy) {
    RVQ_TRY(need(dentropy, "dentropy", 4));
    RVQ_TRY(need(entropy, "entropy", 4));
  }
  const LogprobGradArgs a = {logits, n, V, ids, 1.f / temperature, stats, entropy, dlogprob, dentropy, dlogits};
  return launched(launch_logprobs_grad(a, dtype == RVQ_BF16, stream), "log probability gradient launch");
}

static rvq_status check_distill(const void *logits, rvq_dtype dtype, int64_t n, int32_t V, const int32_t *teacher_ids,
                                const float *teacher, int32_t k, float temperature, const float *stats) {
  RVQ_TRY(check_rows(n, V, "V", kMaxVocab));
  RVQ_TRY(check_dtype(dtype, "dtype"));
  RVQ_TRY(check_temperature(temperature));
  if (k < 1) return fail(RVQ_ERR_INVALID_ARGUMENT, "k must be >= 1 (got %d)", k);
  if (k > kMaxTeacher) return fail(RVQ_ERR_UNSUPPORTED, "k above %d (got %d)", kMaxTeacher, k);
  if (n == 0) return RVQ_OK;
  RVQ_TRY(need(logits, "logits", dtype_bytes(dtype)));
  RVQ_TRY(need(teacher_ids, "teacher_ids", 4));
  RVQ_TRY(need(teacher, "teacher", 4));
  return need(stats, "stats", 4);
}

rvq_status rvq_distill_loss(const void *logits, rvq_dtype dtype, int64_t n, int32_t V,
                            const int32_t *teacher_ids, const float *teacher, int32_t k,
                            int32_t tail, float temperature, float *loss, float *stats,
                            uint32_t *bad_ids, hipStream_t stream) {
  RVQ_TRY(check_distill(logits, dtype, n, V, teacher_ids, teacher, k, temperature, stats));
  if (n == 0) return RVQ_OK;
  RVQ_TRY(need(loss, "loss", 4));
  RVQ_TRY(may(bad_ids, "bad_ids", 4));
  const DistillArgs a = {logits, n, V, teacher_ids, teacher, k, tail != 0, 1.f / temperature, loss, stats, bad_ids,
                         nullptr, nullptr};
  return launched(launch_distill(a, dtype == RVQ_BF16, stream), "distillation launch");
}

rvq_status rvq_distill_loss_backward(const void *logits, rvq_dtype dtype, int64_t n, int32_t V,
                                     const int32_t *teacher_ids, const float *teacher, int32_t k,
                                     int32_t tail, float temperature, const float *stats,
                                     const float *dloss, void *dlogits, hipStream_t stream) {
  RVQ_TRY(check_distill(logits, dtype, n, V, teacher_ids, teacher, k, temperature, stats));
  if (n == 0) return RVQ_OK;
  RVQ_TRY(need(dloss, "dloss", 4));
  RVQ_TRY(need(dlogits, "dlogits", dtype_bytes(dtype)));
  RVQ_TRY(check_in_place(logits, dlogits, n * V * (int64_t)dtype_bytes(dtype)));
  const DistillArgs a = {logits, n, V, teacher_ids, teacher, k, tail != 0, 1.f / temperature, nullptr,
                         (float *)stats, nullptr, dloss, dlogits};
  return launched(launch_distill_grad(a, dtype == RVQ_BF16, stream), "distillation gradient launch");
}

}  // extern "C"
