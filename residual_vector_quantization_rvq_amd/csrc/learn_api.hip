// learn_api.hip -- the part of the C ABI (include/rvq.h) that trains the
// token embedding: the RMS norm and its gradient, the embedding's gradient
// and the AdamW step.  Host side only: arguments are checked before any HIP
// call, workspaces are laid out, launches go to the caller's stream.
#include <cmath>

#include "learn.h"

namespace rvq {
uint32_t adam_key(uint32_t seed, uint32_t step);
}
using namespace rvq;

namespace {

constexpr int64_t kMaxRows = (int64_t)1 << 25;
constexpr int kMaxWidth = 1 << 20;
constexpr int kMaxLevels = 64;
constexpr int64_t kMaxTableRows = (int64_t)1 << 28;  // 512 rows a workgroup of 1024: under 2^32 work-items
constexpr int64_t kMaxList = (int64_t)1 << 30;       // list positions are 32-bit, also a batch beyond the end
constexpr int64_t kMaxNumel = (int64_t)1 << 34;      // a tensor's workgroups stay under 2^24

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

rvq_status check_rows(int64_t n, int32_t d) {
  if (n < 0) return fail(RVQ_ERR_INVALID_ARGUMENT, "n must be >= 0 (got %lld)", (long long)n);
  if (d < 1) return fail(RVQ_ERR_INVALID_ARGUMENT, "d must be >= 1 (got %d)", d);
  if (n > kMaxRows)
    return fail(RVQ_ERR_UNSUPPORTED, "n above %lld rows per call (got %lld)", (long long)kMaxRows,
                (long long)n);
  if (d > kMaxWidth) return fail(RVQ_ERR_UNSUPPORTED, "d above %d (got %d)", kMaxWidth, d);
  return RVQ_OK;
}

rvq_status check_weight(const void *weight, rvq_dtype w_dtype) {
  if (!weight) return RVQ_OK;
  if (!float_or_bf16(w_dtype))
    return fail(RVQ_ERR_INVALID_ARGUMENT, "unknown weight_dtype %d", (int)w_dtype);
  return need(weight, "weight", dtype_bytes(w_dtype));
}

rvq_status check_tables(int64_t T, int32_t L, int32_t K, int64_t V, int32_t D) {
  if (T < 0) return fail(RVQ_ERR_INVALID_ARGUMENT, "T must be >= 0 (got %lld)", (long long)T);
  if (L < 1 || K < 1 || D < 1 || V < 0)
    return fail(RVQ_ERR_INVALID_ARGUMENT, "need L, K, D >= 1 and V >= 0 (got %d, %d, %d, %lld)",
                L, K, D, (long long)V);
  if (L > kMaxLevels)
    return fail(RVQ_ERR_UNSUPPORTED, "embedding supports L <= %d (got %d)", kMaxLevels, L);
  if (D > kMaxWidth) return fail(RVQ_ERR_UNSUPPORTED, "D above %d (got %d)", kMaxWidth, D);
  if (T > kMaxRows || T * (L + 1) > kMaxList)
    return fail(RVQ_ERR_UNSUPPORTED, "T above %lld tokens, or T (L + 1) above 2^30 (got %lld, %d)",
                (long long)kMaxRows, (long long)T, L);
  if (V > kMaxTableRows || (int64_t)L * K + V > kMaxTableRows)
    return fail(RVQ_ERR_UNSUPPORTED, "L K + V above %lld rows", (long long)kMaxTableRows);
  return RVQ_OK;
}

}  // namespace

extern "C" {

rvq_status rvq_rms_norm(const void *x, const void *residual, rvq_dtype x_dtype, int64_t n,
                        int32_t d, const void *weight, rvq_dtype weight_dtype, float eps,
                        void *sum_out, void *y, rvq_dtype y_dtype, float *y_scale, float *rstd,
                        hipStream_t stream) {
  RVQ_TRY(check_rows(n, d));
  if (!float_or_bf16(x_dtype))
    return fail(RVQ_ERR_INVALID_ARGUMENT, "unknown x_dtype %d", (int)x_dtype);
  if (!float_or_bf16(y_dtype) && y_dtype != RVQ_F8E4M3)
    return fail(RVQ_ERR_INVALID_ARGUMENT, "unknown y_dtype %d", (int)y_dtype);
  if (!(eps > 0.f) || !std::isfinite(eps))
    return fail(RVQ_ERR_INVALID_ARGUMENT, "eps must be positive and finite (got %g)", (double)eps);
  RVQ_TRY(check_weight(weight, weight_dtype));
  if (n == 0) return RVQ_OK;
  const size_t xs = dtype_bytes(x_dtype);
  RVQ_TRY(need(x, "x", xs));
  RVQ_TRY(may(residual, "residual", xs));
  RVQ_TRY(may(sum_out, "sum_out", xs));
  RVQ_TRY(need(y, "y", dtype_bytes(y_dtype)));
  if (sum_out == y)
    return fail(RVQ_ERR_INVALID_ARGUMENT, "sum_out and y must not be the same memory");
  if (y_dtype == RVQ_F8E4M3) RVQ_TRY(need(y_scale, "y_scale", 4));
  RVQ_TRY(may(rstd, "rstd", 4));
  NormArgs a = {x, residual, weight, weight_dtype == RVQ_BF16, sum_out, y, (int)y_dtype,
                y_scale, rstd, n, d, eps};
  return launched(launch_rms_norm(a, x_dtype == RVQ_BF16, stream), "RMS norm launch");
}

rvq_status rvq_rms_norm_backward_workspace_size(int64_t n, int32_t d, size_t *bytes) {
  RVQ_TRY(check_rows(n, d));
  if (!bytes) return fail(RVQ_ERR_INVALID_ARGUMENT, "bytes must not be NULL");
  const int64_t p32 = norm_grad_parts(n, d, false), p16 = norm_grad_parts(n, d, true);
  *bytes = al256((size_t)(p32 > p16 ? p32 : p16) * (size_t)d * sizeof(float));
  return RVQ_OK;
}

rvq_status rvq_rms_norm_backward(const void *dy, const void *h, rvq_dtype dtype, int64_t n,
                                 int32_t d, const float *rstd, const void *weight,
                                 rvq_dtype weight_dtype, const void *dsum, void *dx,
                                 float *dweight, void *workspace, size_t workspace_bytes,
                                 hipStream_t stream) {
  RVQ_TRY(check_rows(n, d));
  if (!float_or_bf16(dtype))
    return fail(RVQ_ERR_INVALID_ARGUMENT, "unknown dtype %d", (int)dtype);
  RVQ_TRY(check_weight(weight, weight_dtype));
  const size_t xs = dtype_bytes(dtype);
  if (n > 0) {
    RVQ_TRY(need(dy, "dy", xs));
    RVQ_TRY(need(h, "h", xs));
    RVQ_TRY(need(rstd, "rstd", 4));
    RVQ_TRY(may(dsum, "dsum", xs));
    RVQ_TRY(need(dx, "dx", xs));
  }
  if (dweight) {
    RVQ_TRY(need(dweight, "dweight", 4));
    size_t want = 0;
    RVQ_TRY(rvq_rms_norm_backward_workspace_size(n, d, &want));
    RVQ_TRY(need(workspace, "workspace", 256));
    if (workspace_bytes < want)
      return fail(RVQ_ERR_WORKSPACE_TOO_SMALL, "norm gradient workspace needs %zu bytes (got %zu)",
                  want, workspace_bytes);
  }
  if (n == 0 && !dweight) return RVQ_OK;
  NormGradArgs a = {dy, h, dsum, rstd, weight, weight_dtype == RVQ_BF16, dx, dweight,
                    (float *)workspace, n, d};
  return launched(launch_rms_norm_grad(a, dtype == RVQ_BF16, stream), "RMS norm gradient launch");
}

rvq_status rvq_embed_tokens_backward_workspace_size(int64_t T, int32_t L, int32_t K, int64_t V,
                                                    int32_t D, size_t *bytes) {
  RVQ_TRY(check_tables(T, L, K, V, D));
  if (!bytes) return fail(RVQ_ERR_INVALID_ARGUMENT, "bytes must not be NULL");
  // whichever tables a call asks for
  size_t most = embed_grad_layout(T, L, L, K, V, D).total;
  const size_t levels = embed_grad_layout(T, L, L, K, 0, D).total;
  const size_t text = V > 0 ? embed_grad_layout(T, L, 0, K, V, D).total : 0;
  if (levels > most) most = levels;
  if (text > most) most = text;
  *bytes = most;
  return RVQ_OK;
}

rvq_status rvq_embed_tokens_backward(const void *dout, rvq_dtype dout_dtype, const int32_t *ids,
                                     const uint8_t *is_visual, int64_t T, int32_t L, int32_t K,
                                     int64_t V, int32_t D, void *dlevel, void *dtext,
                                     rvq_dtype grad_dtype, int32_t accumulate, uint32_t *bad_ids,
                                     void *workspace, size_t workspace_bytes, hipStream_t stream) {
  RVQ_TRY(check_tables(T, L, K, V, D));
  if (!float_or_bf16(dout_dtype))
    return fail(RVQ_ERR_INVALID_ARGUMENT, "unknown dout_dtype %d", (int)dout_dtype);
  if (!float_or_bf16(grad_dtype))
    return fail(RVQ_ERR_INVALID_ARGUMENT, "unknown grad_dtype %d", (int)grad_dtype);
  if (!dlevel && !dtext)
    return fail(RVQ_ERR_INVALID_ARGUMENT, "dlevel and dtext must not both be NULL");
  if (T > 0) {
    RVQ_TRY(need(dout, "dout", dtype_bytes(dout_dtype)));
    RVQ_TRY(need(ids, "ids", 4));
  }
  RVQ_TRY(may(dlevel, "dlevel", dtype_bytes(grad_dtype)));
  RVQ_TRY(may(dtext, "dtext", dtype_bytes(grad_dtype)));
  RVQ_TRY(may(bad_ids, "bad_ids", 4));
  size_t want = 0;
  RVQ_TRY(rvq_embed_tokens_backward_workspace_size(T, L, K, V, D, &want));
  RVQ_TRY(need(workspace, "workspace", 256));
  if (workspace_bytes < want)
    return fail(RVQ_ERR_WORKSPACE_TOO_SMALL,
                "embedding gradient workspace needs %zu bytes (got %zu)", want, workspace_bytes);
  const EmbedGradLayout w = embed_grad_layout(T, L, dlevel ? L : 0, K, dtext ? V : 0, D);
  char *ws = (char *)workspace;
  EmbedGradArgs a = {dout, ids, is_visual, T, L, K, D, V, dlevel, dtext, accumulate != 0, bad_ids,
                     (int2 *)(ws + w.place),
                     (int32_t *)(ws + w.token), (int32_t *)(ws + w.row), (float *)(ws + w.part),
                     (int32_t *)(ws + w.keys)};
  return launched(launch_embed_grad(a, dout_dtype == RVQ_BF16, grad_dtype == RVQ_BF16, stream),
                  "embedding gradient launch");
}

rvq_status rvq_adamw_workspace_size(int32_t count, size_t *bytes) {
  if (count < 0) return fail(RVQ_ERR_INVALID_ARGUMENT, "count must be >= 0 (got %d)", count);
  if (!bytes) return fail(RVQ_ERR_INVALID_ARGUMENT, "bytes must not be NULL");
  *bytes = 256 + al256(adam_part_count(count) * sizeof(double));
  return RVQ_OK;
}

rvq_status rvq_adamw_step(const rvq_adamw_tensor *tensors, int32_t count, rvq_dtype param_dtype,
                          rvq_dtype grad_dtype, int32_t state_bits,
                          const rvq_adamw_options *options, float *grad_norm, void *workspace,
                          size_t workspace_bytes, hipStream_t stream) {
  if (count < 0) return fail(RVQ_ERR_INVALID_ARGUMENT, "count must be >= 0 (got %d)", count);
  if (count > 0 && !tensors) return fail(RVQ_ERR_INVALID_ARGUMENT, "tensors must not be NULL");
  if (!options) return fail(RVQ_ERR_INVALID_ARGUMENT, "options must not be NULL");
  if (!float_or_bf16(param_dtype))
    return fail(RVQ_ERR_INVALID_ARGUMENT, "unknown param_dtype %d", (int)param_dtype);
  if (!float_or_bf16(grad_dtype))
    return fail(RVQ_ERR_INVALID_ARGUMENT, "unknown grad_dtype %d", (int)grad_dtype);
  if (state_bits != 8 && state_bits != 32)
    return fail(RVQ_ERR_INVALID_ARGUMENT, "state_bits must be 8 or 32 (got %d)", state_bits);
  const rvq_adamw_options &o = *options;
  if (!(o.lr >= 0.0) || !std::isfinite(o.lr) || !(o.beta1 >= 0.0 && o.beta1 < 1.0) ||
      !(o.beta2 >= 0.0 && o.beta2 < 1.0))
    return fail(RVQ_ERR_INVALID_ARGUMENT, "need a finite lr >= 0 and beta1, beta2 in [0, 1)");
  if (!(o.eps >= 1e-12) || !std::isfinite(o.eps))
    return fail(RVQ_ERR_INVALID_ARGUMENT, "eps must be finite and at least 1e-12 (got %g)", o.eps);
  if (o.step < 1)
    return fail(RVQ_ERR_INVALID_ARGUMENT, "step must be >= 1 (got %lld)", (long long)o.step);
  if (!std::isfinite((float)o.grad_scale) || !std::isfinite(o.max_norm))
    return fail(RVQ_ERR_INVALID_ARGUMENT, "grad_scale and max_norm must be finite, grad_scale in fp32");
  // as the kernels take them, in fp32
  const float lr1 = (float)(o.lr / (1.0 - std::pow(o.beta1, (double)o.step)));
  const float rk2 = (float)(1.0 / std::sqrt(1.0 - std::pow(o.beta2, (double)o.step)));
  if (!std::isfinite(lr1) || !std::isfinite(rk2))
    return fail(RVQ_ERR_INVALID_ARGUMENT, "lr / (1 - beta1^step) must be within fp32");
  const size_t ps = dtype_bytes(param_dtype), ss = state_bits == 8 ? 1 : 4;
  bool any = false;
  for (int32_t i = 0; i < count; ++i) {
    const rvq_adamw_tensor &t = tensors[i];
    if (t.numel < 0)
      return fail(RVQ_ERR_INVALID_ARGUMENT, "tensor %d: numel must be >= 0 (got %lld)", i,
                  (long long)t.numel);
    if (t.numel > kMaxNumel)
      return fail(RVQ_ERR_UNSUPPORTED, "tensor %d: numel above %lld (got %lld)", i,
                  (long long)kMaxNumel, (long long)t.numel);
    if (!std::isfinite(t.weight_decay))
      return fail(RVQ_ERR_INVALID_ARGUMENT, "tensor %d: weight_decay must be finite", i);
    if (t.numel == 0) continue;
    any = true;
    const bool ok = t.param && at_multiple(t.param, ps) && t.grad &&
                    at_multiple(t.grad, dtype_bytes(grad_dtype)) && t.m && at_multiple(t.m, ss) &&
                    t.v && at_multiple(t.v, ss) && at_multiple(t.copy, 2) &&
                    (state_bits == 32 || (t.m_scale && at_multiple(t.m_scale, 4) && t.v_scale &&
                                          at_multiple(t.v_scale, 4)));
    if (!ok)
      return fail(RVQ_ERR_INVALID_ARGUMENT,
                  "tensor %d: param, grad, m, v (and, in 8 bits, m_scale, v_scale) must not be NULL "
                  "and must be aligned to their elements, as copy if it is given", i);
  }
  const bool norm = o.max_norm > 0.0 || grad_norm;
  RVQ_TRY(may(grad_norm, "grad_norm", 4));
  if (norm) {
    size_t want = 0;
    RVQ_TRY(rvq_adamw_workspace_size(count, &want));
    RVQ_TRY(need(workspace, "workspace", 256));
    if (workspace_bytes < want)
      return fail(RVQ_ERR_WORKSPACE_TOO_SMALL, "AdamW workspace needs %zu bytes (got %zu)", want,
                  workspace_bytes);
  }
  if (!any && !grad_norm) return RVQ_OK;
  AdamArgs a;
  a.count = count;
  a.p_bf16 = param_dtype == RVQ_BF16;
  a.g_bf16 = grad_dtype == RVQ_BF16;
  a.eight = state_bits == 8;
  a.b1 = (float)o.beta1;
  a.c1 = (float)(1.0 - o.beta1);
  a.b2 = (float)o.beta2;
  a.c2 = (float)(1.0 - o.beta2);
  a.eps = (float)o.eps;
  a.lr = o.lr;
  a.lr1 = lr1;
  a.rk2 = rk2;
  a.grad_scale = (float)o.grad_scale;
  a.max_norm = (float)o.max_norm;
  if (o.max_norm > 0.0 && a.max_norm == 0.f) a.max_norm = 0x1p-149f;  // 0 would be no clipping
  a.stochastic = o.stochastic != 0;
  a.key = adam_key((uint32_t)o.seed, (uint32_t)o.step);
  a.grad_norm = grad_norm;
  a.clip = norm ? (float *)workspace : nullptr;
  a.part = norm ? (double *)((char *)workspace + 256) : nullptr;
  return launched(launch_adamw(tensors, a, stream), "AdamW launch");
}

}  // extern "C"
