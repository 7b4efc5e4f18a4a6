// learn.h -- device and host helpers shared by the kernels that train the
// token embedding: the RMS norm, the embedding's gradient and the optimizer.
#pragma once

#include "common.h"
#include "rvq.h"

namespace rvq {

// ---- host side ----
rvq_status fail(rvq_status st, const char *fmt, ...) __attribute__((format(printf, 2, 3)));

inline size_t al256(size_t v) { return (v + 255) & ~(size_t)255; }
inline bool at_multiple(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }
inline size_t dtype_bytes(rvq_dtype t) { return t == RVQ_F32 ? 4 : t == RVQ_BF16 ? 2 : 1; }
inline bool float_or_bf16(rvq_dtype t) { return t == RVQ_F32 || t == RVQ_BF16; }

// ---- 8-bit values: e4m3, largest 448, with fp32 scales ----
constexpr float kF8Max = 448.f;
// The smallest scale: a block of zeros (or of values below 2^-91) divides by
// it and not by zero.
constexpr float kScaleMin = 0x1p-100f;

// four fp32 values as e4m3 bytes, rounded to nearest even; |v| <= 448
__device__ __forceinline__ uint32_t pack_f8x4(float a, float b, float c, float d) {
  int w = 0;
  w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, w, false);
  w = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
  return (uint32_t)w;
}
__device__ __forceinline__ uint8_t f32_to_f8(float a) {
  return (uint8_t)(__builtin_amdgcn_cvt_pk_fp8_f32(a, a, 0, false) & 0xff);
}
__device__ __forceinline__ float f8_to_f32(uint8_t b) {
  return __builtin_amdgcn_cvt_f32_fp8((int)b, 0);
}
__device__ __forceinline__ float clamp_f8(float v) { return fminf(fmaxf(v, -kF8Max), kF8Max); }

// ---- element access; bf16 is held as its 16 bits ----
__device__ __forceinline__ float load_f32(const float *p, int64_t i) { return p[i]; }
__device__ __forceinline__ float load_f32(const uint16_t *p, int64_t i) {
  return bf16_bits_to_f32(p[i]);
}
__device__ __forceinline__ void store_f32(float *p, int64_t i, float v) { p[i] = v; }
__device__ __forceinline__ void store_f32(uint16_t *p, int64_t i, float v) {
  p[i] = f32_to_bf16_bits(v);
}
// a pointer of either type, told apart by a flag that is the same for the whole launch
__device__ __forceinline__ float load_either(const void *p, bool bf16, int64_t i) {
  return bf16 ? load_f32((const uint16_t *)p, i) : load_f32((const float *)p, i);
}

__device__ __forceinline__ float wave_max_f32(float v) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v = fmaxf(v, __shfl_xor(v, off, 64));
  return v;
}

// ---- launchers ----
struct NormArgs {
  const void *x, *residual;   // residual may be null
  const void *weight;         // null: ones
  bool w_bf16;
  void *sum, *y;              // sum may be null
  int y_type;                 // rvq_dtype
  float *scale, *rstd;        // scale: 8-bit output only; rstd may be null
  int64_t n;
  int d;
  float eps;
};
hipError_t launch_rms_norm(const NormArgs &a, bool x_bf16, hipStream_t s);

struct NormGradArgs {
  const void *dy, *h, *dsum;  // dsum may be null
  const float *rstd;
  const void *weight;         // null: ones
  bool w_bf16;
  void *dx;
  float *dweight;             // null: not wanted
  float *part;                // [norm_grad_parts(n)][d]
  int64_t n;
  int d;
};
int64_t norm_grad_parts(int64_t n);
hipError_t launch_rms_norm_grad(const NormGradArgs &a, bool bf16, hipStream_t s);

struct EmbedGradArgs {
  const void *dout;
  const int32_t *ids;
  const uint8_t *is_visual;   // null: every token is visual
  int64_t T;
  int L, K, D;
  int64_t V;
  void *dlevel, *dtext;       // either may be null
  bool accumulate;
  uint32_t *bad;
  // workspace
  int32_t *start, *count;     // [rows]: each destination row's piece of the list
  int32_t *token, *row;       // the list: tokens by destination row, in token order; its row
  float *part;                // [2 segments][D]: sums of the pieces of long rows
};
struct EmbedGradLayout {
  size_t start, count, token, row, part, total;
};
EmbedGradLayout embed_grad_layout(int64_t T, int L, int K, int64_t V, int D);
hipError_t launch_embed_grad(const EmbedGradArgs &a, bool x_bf16, bool g_bf16, hipStream_t s);

struct AdamArgs {
  int count;
  bool p_bf16, g_bf16, eight;
  float b1, c1, b2, c2, eps;    // c = 1 - b
  float lr1, rk2;               // lr / (1 - b1^t), 1 / sqrt(1 - b2^t)
  double lr;
  float grad_scale, max_norm;   // max_norm <= 0: no clipping
  bool stochastic;
  uint32_t key;                 // mixed from seed and step
  float *grad_norm;             // may be null
  double *part;                 // workspace: partial sums of squares
  float *clip;                  // workspace: the factor of the gradients (NaN: skip)
};
size_t adam_part_count(int count);
hipError_t launch_adamw(const rvq_adamw_tensor *t, const AdamArgs &a, hipStream_t s);

}  // namespace rvq
