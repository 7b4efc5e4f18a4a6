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
constexpr float kF8Unit = 1.f / 448.f;  // scales: the largest value times this
// The smallest scale: a block of zeros (or of values below 2^-91) divides by
// it and not by zero.
constexpr float kScaleMin = 0x1p-100f;

// four fp32 values as e4m3 bytes, rounded to nearest even; |v| <= 448 or a few
// units of the last place above it, which rounding brings to 448; NaN stays NaN
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
// The nearest fp32 to x / d, inv the nearest to 1 / d: an e4m3 value turns on
// the quotient's last place (x * inv is stored as the neighbour on the grid
// about once in 10^6 values, 6 to 12% away).
__device__ __forceinline__ float nearest_quotient(float x, float d, float inv) {
  const float q = x * inv;
  return __builtin_fmaf(__builtin_fmaf(-q, d, x), inv, q);
}

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

// ---- 16-byte pieces of a row: 4 fp32 or 8 bf16 elements ----
// Rows need not begin at a multiple of 16 bytes (odd widths, slices): the
// hardware takes wide loads and stores at any element's address, so one path
// serves every alignment.  The piece a row ends in is taken by elements.
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef u32x4 u32x4_at2 __attribute__((aligned(2)));
typedef u32x4 u32x4_at4 __attribute__((aligned(4)));
typedef u32x2 u32x2_at1 __attribute__((aligned(1)));
typedef u32x2 u32x2_at2 __attribute__((aligned(2)));
typedef uint32_t u32_at1 __attribute__((aligned(1)));

template <typename T>
constexpr int kPiece = 16 / (int)sizeof(T);

__device__ __forceinline__ void unpack(u32x4 q, float (&v)[4]) {
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = __uint_as_float(q[e]);
}
__device__ __forceinline__ void unpack(u32x4 q, float (&v)[8]) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    v[2 * e] = __uint_as_float(q[e] << 16);
    v[2 * e + 1] = __uint_as_float(q[e] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint32_t pack_bf16x2(float a, float b) {
  return (uint32_t)f32_to_bf16_bits(a) | ((uint32_t)f32_to_bf16_bits(b) << 16);
}
__device__ __forceinline__ u32x4 load16(const float *p) { return *(const u32x4_at4 *)p; }
__device__ __forceinline__ u32x4 load16(const uint16_t *p) { return *(const u32x4_at2 *)p; }

// A piece as it is stored; `left` (which may be negative) of its elements
// exist, the others read as zero.
__device__ __forceinline__ u32x4 load_piece(const float *p, int left) {
  if (left >= 4) return load16(p);
  u32x4 q = {0, 0, 0, 0};
#pragma unroll
  for (int e = 0; e < 3; ++e)
    if (e < left) q[e] = __float_as_uint(p[e]);
  return q;
}
__device__ __forceinline__ u32x4 load_piece(const uint16_t *p, int left) {
  if (left >= 8) return load16(p);
  u32x4 q = {0, 0, 0, 0};
#pragma unroll
  for (int e = 0; e < 7; ++e)
    if (e < left) q[e >> 1] |= (uint32_t)p[e] << (16 * (e & 1));
  return q;
}

// N elements at p; `left` of them exist (the others read as zero)
template <int N>
__device__ __forceinline__ void load_n(const float *p, int left, float (&v)[N]) {
  if (left >= N) {
#pragma unroll
    for (int j = 0; j < N; j += 4) {
      const u32x4 q = load16(p + j);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[j + e] = __uint_as_float(q[e]);
    }
  } else {
#pragma unroll
    for (int e = 0; e < N; ++e) v[e] = e < left ? p[e] : 0.f;
  }
}
template <int N>
__device__ __forceinline__ void load_n(const uint16_t *p, int left, float (&v)[N]) {
  if (left >= N) {
    if constexpr (N == 8) {
      unpack(load16(p), v);
    } else {
      const u32x2 q = *(const u32x2_at2 *)p;
      v[0] = __uint_as_float(q[0] << 16);
      v[1] = __uint_as_float(q[0] & 0xffff0000u);
      v[2] = __uint_as_float(q[1] << 16);
      v[3] = __uint_as_float(q[1] & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int e = 0; e < N; ++e) v[e] = e < left ? bf16_bits_to_f32(p[e]) : 0.f;
  }
}
template <int N>
__device__ __forceinline__ void store_n(float *p, int left, const float (&v)[N]) {
  if (left >= N) {
#pragma unroll
    for (int j = 0; j < N; j += 4) {
      const u32x4 q = {__float_as_uint(v[j]), __float_as_uint(v[j + 1]), __float_as_uint(v[j + 2]),
                       __float_as_uint(v[j + 3])};
      *(u32x4_at4 *)(p + j) = q;
    }
  } else {
#pragma unroll
    for (int e = 0; e < N; ++e)
      if (e < left) p[e] = v[e];
  }
}
template <int N>
__device__ __forceinline__ void store_n(uint16_t *p, int left, const float (&v)[N]) {
  if (left >= N) {
    if constexpr (N == 8) {
      const u32x4 q = {pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                       pack_bf16x2(v[6], v[7])};
      *(u32x4_at2 *)p = q;
    } else {
      const u32x2 q = {pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
      *(u32x2_at2 *)p = q;
    }
  } else {
#pragma unroll
    for (int e = 0; e < N; ++e)
      if (e < left) p[e] = f32_to_bf16_bits(v[e]);
  }
}
// the same, for what is not read again soon: kept out of the caches' way
template <int N>
__device__ __forceinline__ void stream_n(float *p, const float (&v)[N]) {
#pragma unroll
  for (int j = 0; j < N; j += 4) {
    const u32x4 q = {__float_as_uint(v[j]), __float_as_uint(v[j + 1]), __float_as_uint(v[j + 2]),
                     __float_as_uint(v[j + 3])};
    __builtin_nontemporal_store(q, (u32x4_at4 *)(p + j));
  }
}
template <int N>
__device__ __forceinline__ void stream_n(uint16_t *p, const float (&v)[N]) {
  if constexpr (N == 8) {
    const u32x4 q = {pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                     pack_bf16x2(v[6], v[7])};
    __builtin_nontemporal_store(q, (u32x4_at2 *)p);
  } else {
    const u32x2 q = {pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
    __builtin_nontemporal_store(q, (u32x2_at2 *)p);
  }
}
// e4m3 bytes, of values as for pack_f8x4
template <int N>
__device__ __forceinline__ void store_f8_n(uint8_t *p, int left, const float (&v)[N]) {
  if (left >= N) {
    if constexpr (N == 8) {
      const u32x2 q = {pack_f8x4(v[0], v[1], v[2], v[3]), pack_f8x4(v[4], v[5], v[6], v[7])};
      *(u32x2_at1 *)p = q;
    } else {
      *(u32_at1 *)p = pack_f8x4(v[0], v[1], v[2], v[3]);
    }
  } else {
#pragma unroll
    for (int e = 0; e < N; ++e)
      if (e < left) p[e] = f32_to_f8(v[e]);
  }
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
  float *part;                // [norm_grad_parts(n, d, bf16)][d]
  int64_t n;
  int d;
};
int64_t norm_grad_parts(int64_t n, int d, bool bf16);
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
  int2 *place;                // [rows]: where a destination row's tokens begin in the list, and how many
  int32_t *token, *row;       // the list: tokens by destination row, in token order; its row
  float *part;                // [2 segments][D]: sums of the pieces of long rows
  int32_t *keys;              // [tables][T]: the IDs by table
};
struct EmbedGradLayout {
  size_t place, token, row, part, keys, total;
};
// L: the level tables that are asked for (all L_ids or none)
EmbedGradLayout embed_grad_layout(int64_t T, int L_ids, int L, int K, int64_t V, int D);
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
