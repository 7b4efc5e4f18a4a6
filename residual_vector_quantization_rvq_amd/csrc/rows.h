// rows.h -- what the kernels that norm or quantise rows share: how a row is spread over
// lanes, sums and largest values over them, the scale of an 8-bit row, and rows
// whose squares leave fp32.
#pragma once

#include "learn.h"

namespace rvq {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxGroups = 1 << 20;  // workgroups of a launch; rows beyond are looped over

// Sum over the W lanes of a row; for W == kThreads through `red`, which is
// free again after the next barrier.
template <int W>
__device__ __forceinline__ float row_sum(float v, float *red) {
#pragma unroll
  for (int off = (W < 64 ? W : 64) / 2; off >= 1; off >>= 1) v += __shfl_xor(v, off, 64);
  if constexpr (W > 64) {
    __syncthreads();
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0.f;
#pragma unroll
    for (int w = 0; w < W / 64; ++w) v += red[w];
  }
  return v;
}
// The largest magnitude of a row, as its bits: whole numbers in the same order,
// with infinity and then NaN above every finite value, so that neither is lost.
__device__ __forceinline__ uint32_t magnitude_bits(float v) { return __float_as_uint(fabsf(v)); }
template <int W>
__device__ __forceinline__ uint32_t row_max(uint32_t v, float *red) {
#pragma unroll
  for (int off = (W < 64 ? W : 64) / 2; off >= 1; off >>= 1) v = max(v, (uint32_t)__shfl_xor((int)v, off, 64));
  if constexpr (W > 64) {
    __syncthreads();
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = __uint_as_float(v);
    __syncthreads();
    v = __float_as_uint(red[0]);
#pragma unroll
    for (int w = 1; w < W / 64; ++w) v = max(v, __float_as_uint(red[w]));
  }
  return v;
}
// An 8-bit row's scale out of that; NaN where a value of the row is not finite,
// which its e4m3 bytes cannot say.
__device__ __forceinline__ float row_scale(uint32_t top) {
  const float t = __uint_as_float(top);
  return t < INFINITY ? fmaxf(t * kF8Unit, kScaleMin) : NAN;
}
// the same with the quotient by 448 itself, nearest (of a block of 128 or 128 x 128 values, too)
__device__ __forceinline__ float row_scale_of(uint32_t top) {
  const float t = __uint_as_float(top);
  return t < INFINITY ? fmaxf(t / 448.f, kScaleMin) : NAN;
}

template <int N>
__device__ __forceinline__ void load_weight(const void *w, bool bf16, int c, int left, float (&v)[N]) {
  if (!w) {
#pragma unroll
    for (int e = 0; e < N; ++e) v[e] = 1.f;
  } else if (bf16) {
    load_n<N>((const uint16_t *)w + c, left, v);
  } else {
    load_n<N>((const float *)w + c, left, v);
  }
}

// A row's mean of squares plus eps that fp32 does not hold, or holds in less
// than full precision: such a row is taken again with its values times
// range_factor(), a power of two.  (r comes out for the values as multiplied;
// times the factor it is the row's.)  2^-80: 2^20 squares of the largest value add
// up to 2^116, and one that can overflow with 2^20 others is 2^-52 or more.  Only
// rows with values beyond 10^16, or an eps below 2^-100, get there.
__device__ __forceinline__ bool out_of_range(float mean) { return !(mean < INFINITY && mean > 0x1p-100f); }
__device__ __forceinline__ float range_factor(float mean) { return mean < 1.f ? 0x1p70f : 0x1p-80f; }

// how a row of `pieces` is shared: W lanes, P pieces each
#define RVQ_NORM_SHAPES(X) \
  X(8, 1) X(16, 1) X(32, 1) X(64, 1) X(64, 2) X(64, 3) X(256, 1) X(256, 2) X(256, 4) X(256, 8)
struct Shape {
  int w, p;
};
Shape shape_of(int64_t pieces) {
#define RVQ_SHAPE(W, P) \
  if (pieces <= W * P) return {W, P};
  RVQ_NORM_SHAPES(RVQ_SHAPE)
#undef RVQ_SHAPE
  return {0, 0};
}

}  // namespace
}  // namespace rvq
