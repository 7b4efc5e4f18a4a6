// quant_f8.hip -- rows of fp32 or bf16 as 8-bit values (e4m3) with one fp32 scale
// for 128 of them, or for 128 x 128: the operands of the 8-bit product.
//
//   scale = max(max|x| / 448, 2^-100) over the block,  q = e4m3(x / scale), nearest even
//
// A transposed output holds x's columns as its rows, with blocks along them: what
// the weight's gradient contracts are the tokens, the rows of both its operands.
// Bound by memory: x is read once (a tile of 128 x 128 stays in registers between
// its largest value and its quotients), and the bytes are written once; a
// transposed tile turns through LDS, so that its rows leave in whole lines.
// 39,731 x 4096 bf16: rows 95 us (5.1 TB/s), transposed 101 (4.8), blocks of 128 x 128 92 (5.3),
// transposed 98 (5.0); 39,731 x 8192 transposed 191.
#include "head.h"
#include "lanes.h"
#include "rows.h"

namespace rvq {

namespace {

constexpr int kB = kScaleBlock;

template <int N>
__device__ __forceinline__ uint32_t top_of(const float (&v)[N]) {
  uint32_t top = 0;
#pragma unroll
  for (int e = 0; e < N; ++e) top = max(top, magnitude_bits(v[e]));
  return top;
}

}  // namespace

// One scale for 128 elements of a row: 16 (bf16) or 32 (fp32) lanes a block.
template <typename T>
__global__ __launch_bounds__(kThreads) void quantize_rows_kernel(QuantArgs a) {
  constexpr int N = kPiece<T>, L = kB / N;
  const int64_t blocks = ceil_div(a.cols, kB), total = a.rows * blocks;
  const int lane = threadIdx.x % L;
  // the bound is the same for a block's lanes, which exchange their values
  for (int64_t i = (int64_t)blockIdx.x * (kThreads / L) + threadIdx.x / L; i < total;
       i += (int64_t)gridDim.x * (kThreads / L)) {
    const int64_t row = i / blocks, kb = i - row * blocks;
    const int64_t c = kb * kB + lane * N;
    const int left = (int)(a.cols - c < N ? a.cols - c : N);
    float v[N];
    unpack(load_piece((const T *)a.x + row * a.cols + (left > 0 ? c : 0), left), v);
    uint32_t top = top_of<N>(v);
#pragma unroll
    for (int off = L / 2; off >= 1; off >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, off, 64));
    const float scale = row_scale_of(top), inv = 1.f / scale;
    if (lane == 0) a.scale[i] = scale;
    if (left <= 0) continue;
#pragma unroll
    for (int e = 0; e < N; ++e) v[e] = nearest_quotient(v[e], scale, inv);
    store_f8_n<N>(a.q + row * a.q_stride + c, left, v);
  }
}

// A tile of 128 x 128 a workgroup: one scale for all of it (BLOCK), or transposed
// one for each column.  A thread holds N columns of kB * N / kThreads rows that
// follow one another, so that a column's bytes of its rows leave as one word.
template <typename T, bool BLOCK, bool TRANS>
__global__ __launch_bounds__(kThreads) void quantize_tile_kernel(QuantArgs a) {
  constexpr int N = kPiece<T>, L = kB / N, G = kThreads / L, R = kB / G;  // G groups of R rows
  constexpr int kWaves = kThreads / 64;
  __shared__ __attribute__((aligned(16))) uint32_t tops[BLOCK ? kWaves : kWaves * kB];
  // a turned row is eight pieces of 16 bytes, piece p of row r at p ^ (r / 8 % 8), so that
  // the lanes of a wave, eight or four rows apart, do not meet in a bank
  __shared__ __attribute__((aligned(16))) uint8_t turned[TRANS ? kB * kB : 16];
  const int64_t tiles_c = ceil_div(a.cols, kB), tiles_r = ceil_div(a.rows, kB);
  const int lane = threadIdx.x % L, g = threadIdx.x / L;
  for (int64_t t = blockIdx.x; t < tiles_r * tiles_c; t += gridDim.x) {
    const int64_t tr = t / tiles_c, tc = t - tr * tiles_c;
    const int64_t c = tc * kB + lane * N;
    const int left = (int)(a.cols - c < N ? a.cols - c : N);
    float v[R][N];
    uint32_t top[N];
#pragma unroll
    for (int e = 0; e < N; ++e) top[e] = 0;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int64_t row = tr * kB + g * R + i;
      const bool in = row < a.rows && left > 0;
      unpack(load_piece((const T *)a.x + (in ? row * a.cols + c : 0), in ? left : 0), v[i]);
    }
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int e = 0; e < N; ++e) top[e] = max(top[e], magnitude_bits(v[i][e]));
    float scale[N], inv[N];
    if constexpr (BLOCK) {
      uint32_t all = top[0];
#pragma unroll
      for (int e = 1; e < N; ++e) all = max(all, top[e]);
#pragma unroll
      for (int off = 32; off >= 1; off >>= 1) all = max(all, (uint32_t)__shfl_xor((int)all, off, 64));
      __syncthreads();  // the tile before has read tops and turned
      if ((threadIdx.x & 63) == 0) tops[threadIdx.x >> 6] = all;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < kThreads / 64; ++w) all = max(all, tops[w]);
#pragma unroll
      for (int e = 0; e < N; ++e) scale[e] = row_scale_of(all);
      if (threadIdx.x == 0) a.scale[TRANS ? tc * tiles_r + tr : t] = scale[0];
    } else {
      // over the groups of this wave, then over the waves
#pragma unroll
      for (int e = 0; e < N; ++e) {
        if constexpr (L == 16) top[e] = lane_max_rows(top[e]);
        top[e] = lane_max_halves(top[e]);
      }
      __syncthreads();  // the tile before has read tops and turned
      if ((threadIdx.x & 63) < L) {
#pragma unroll
        for (int e = 0; e < N; e += 4)
          *(u32x4 *)(tops + (threadIdx.x >> 6) * kB + lane * N + e) = u32x4{top[e], top[e + 1], top[e + 2], top[e + 3]};
      }
      __syncthreads();
#pragma unroll
      for (int w = 0; w < kWaves; ++w)
#pragma unroll
        for (int e = 0; e < N; e += 4) {
          const u32x4 q = *(const u32x4 *)(tops + w * kB + lane * N + e);
#pragma unroll
          for (int f = 0; f < 4; ++f) top[e + f] = max(top[e + f], q[f]);
        }
#pragma unroll
      for (int e = 0; e < N; ++e) {
        scale[e] = row_scale_of(top[e]);
        if (g == 0 && e < left) a.scale[(c + e) * tiles_r + tr] = scale[e];
      }
    }
#pragma unroll
    for (int e = 0; e < N; ++e) inv[e] = 1.f / scale[e];
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int e = 0; e < N; ++e) v[i][e] = nearest_quotient(v[i][e], scale[e], inv[e]);
    if constexpr (!TRANS) {
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const int64_t row = tr * kB + g * R + i;
        if (row < a.rows && left > 0) store_f8_n<N>(a.q + row * a.q_stride + c, left, v[i]);
      }
    } else {
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const int row = lane * N + e, at = row * kB + (((g * R) >> 4 ^ (row >> 3 & 7)) << 4) + (g * R & 15);
        uint32_t word[R / 4];
#pragma unroll
        for (int i = 0; i < R; i += 4) word[i / 4] = pack_f8x4(v[i][e], v[i + 1][e], v[i + 2][e], v[i + 3][e]);
        if constexpr (R == 8)
          *(u32x2 *)(turned + at) = u32x2{word[0], word[1]};
        else
          *(u32x4 *)(turned + at) = u32x4{word[0], word[1], word[2], word[3]};
      }
      __syncthreads();
      // 16 bytes a lane, 8 lanes a turned row
      const int64_t r0 = tr * kB + (threadIdx.x % 8) * 16;
      const int left_r = (int)(a.rows - r0 < 16 ? a.rows - r0 : 16);
      for (int i = threadIdx.x / 8; i < kB; i += kThreads / 8) {
        const int64_t col = tc * kB + i;
        if (col >= a.cols || left_r <= 0) continue;
        const uint8_t *from = turned + i * kB + ((threadIdx.x % 8 ^ (i >> 3 & 7)) << 4);
        uint8_t *to = a.q + col * a.q_stride + r0;
        if (left_r == 16) {
          typedef u32x4 u32x4_at1 __attribute__((aligned(1)));
          *(u32x4_at1 *)to = *(const u32x4 *)from;
        } else {
          for (int e = 0; e < left_r; ++e) to[e] = from[e];
        }
      }
    }
  }
}

template <typename T>
static hipError_t quantize(const QuantArgs &a, hipStream_t s) {
  if (!a.block_rows && !a.transpose) {
    const int64_t groups = ceil_div(a.rows * ceil_div(a.cols, kB), kThreads / (kB / kPiece<T>));
    quantize_rows_kernel<T><<<dim3((unsigned)(groups < kMaxGroups ? groups : kMaxGroups)), kThreads, 0, s>>>(a);
    return hipGetLastError();
  }
  const int64_t tiles = ceil_div(a.rows, kB) * ceil_div(a.cols, kB);
  const dim3 grid((unsigned)(tiles < kMaxGroups ? tiles : kMaxGroups));
  if (a.block_rows && a.transpose)
    quantize_tile_kernel<T, true, true><<<grid, kThreads, 0, s>>>(a);
  else if (a.block_rows)
    quantize_tile_kernel<T, true, false><<<grid, kThreads, 0, s>>>(a);
  else
    quantize_tile_kernel<T, false, true><<<grid, kThreads, 0, s>>>(a);
  return hipGetLastError();
}

hipError_t launch_quantize_f8(const QuantArgs &a, bool x_bf16, hipStream_t s) {
  if (a.rows == 0 || a.cols == 0) return hipSuccess;
  return x_bf16 ? quantize<uint16_t>(a, s) : quantize<float>(a, s);
}

}  // namespace rvq
