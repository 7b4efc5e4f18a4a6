// lanes.h -- sums and largest values over the lanes of a wave, without LDS.
//
// Each step joins a lane with a partner that holds the other half of what is to be
// joined: neighbours and pairs of four lanes by their permutation, quads and halves of
// sixteen lanes by mirroring (all lanes of a quad hold the same by then), rows of
// sixteen and halves of the wave by the instructions that swap them.  All lanes end with the
// same bits.  Six steps take about 80 cycles, where as many exchanges through LDS take 700:
// a row that one wave sums three times is bound by that.
#pragma once

#include "common.h"

namespace rvq {
namespace {

template <int CTRL>
__device__ __forceinline__ float from_lane(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xf, 0xf, true));
}
constexpr int kNeighbours = 0xB1, kPairs = 0x4E, kHalfMirror = 0x141, kMirror = 0x140;

// f(v, partner's v) over aligned groups of W lanes
template <int W, typename F>
__device__ __forceinline__ float over_lanes(float v, F f) {
  static_assert(W == 8 || W == 16 || W == 32 || W == 64, "groups of lanes");
  v = f(v, from_lane<kNeighbours>(v));
  v = f(v, from_lane<kPairs>(v));
  v = f(v, from_lane<kHalfMirror>(v));
  if constexpr (W >= 16) v = f(v, from_lane<kMirror>(v));
  if constexpr (W >= 32) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = f(__uint_as_float(r[0]), __uint_as_float(r[1]));
  }
  if constexpr (W == 64) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = f(__uint_as_float(r[0]), __uint_as_float(r[1]));
  }
  return v;
}
template <int W>
__device__ __forceinline__ float lane_sum(float v) {
  return over_lanes<W>(v, [](float a, float b) { return a + b; });
}
template <int W>
__device__ __forceinline__ float lane_max(float v) {  // NaN is passed over
  return over_lanes<W>(v, [](float a, float b) { return fmaxf(a, b); });
}
template <int W>
__device__ __forceinline__ uint32_t lane_max_bits(uint32_t v) {
  return __float_as_uint(over_lanes<W>(__uint_as_float(v), [](float a, float b) {
    return __uint_as_float(max(__float_as_uint(a), __float_as_uint(b)));
  }));
}

// the larger of a lane's value and that of the lane 16 (or 32) away
__device__ __forceinline__ uint32_t lane_max_rows(uint32_t v) {
  const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  return max(r[0], r[1]);
}
__device__ __forceinline__ uint32_t lane_max_halves(uint32_t v) {
  const auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  return max(r[0], r[1]);
}

}  // namespace
}  // namespace rvq
