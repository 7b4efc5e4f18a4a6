// norm.hip -- root-mean-square norm of rows, with the residual's addition
// and an 8-bit output, and its gradient.
//
//   h = x (+ residual),  r = 1 / sqrt(mean(h^2) + eps),  y = h r w
//
// Everything between the loads and the stores is fp32; h is rounded to the
// rows' type only where it is stored, and the norm uses the unrounded sum.
//
// Bound by memory: a row is read once, held in registers for the sum and for
// the products, and written once.  A row is shared by W lanes of P 16-byte
// pieces each: a part of a wave for narrow rows (several rows a wave), a wave
// up to 192 pieces, else a workgroup.  Rows of more than 2048 pieces (8192
// fp32 or 16384 bf16 elements) are read again for each pass over them.
//
// Measured (bytes read and written): 39,731 x 4096 bf16 with residual 229 us,
// 5.7 TB/s, to 8 bits 207 us, and without residual to 8 bits 112 us, 4.4 TB/s;
// 39,731 x 1152 bf16 80 us, 4.6 TB/s (a workgroup a row was 8% slower); 3001 x
// 1155 fp32 8.0 us: 289 pieces on 512 slots, and two rounds of workgroups; one row
// of 4096 4.0 us, the time of a launch.  Gradient, 39,731 x 4096 bf16 with dsum and
// dweight: 237 + 6 us, 5.3 TB/s.
// Streaming stores gain 4% of the norm and 1% of its gradient, and take the
// rows out of the caches, where the next layer looks for them: not used.
#include "rows.h"

namespace rvq {

// Two pieces a lane: held to the 72 registers of seven waves (with 74 and six,
// 39,731 x 4096 bf16 to 8 bits take 121 us and not 112, 60,000 x 640 bf16 with
// residual 67 and not 62).
template <typename T, int W, int P>
__global__ __launch_bounds__(kThreads, P == 2 ? 7 : 1) void rms_norm_kernel(NormArgs a) {
  constexpr int N = kPiece<T>, R = kThreads / W;
  __shared__ float red[kThreads / 64];
  const int lane = threadIdx.x % W;
  // W == kThreads: the row is the same for the whole workgroup, as the barriers need
  for (int64_t row = (int64_t)blockIdx.x * R + threadIdx.x / W; row < a.n; row += (int64_t)gridDim.x * R) {
    const int64_t at = row * a.d;
    float h[P][N];
    float ss = 0.f;
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int c = (p * W + lane) * N;
      if (c < a.d) {
        load_n<N>((const T *)a.x + at + c, a.d - c, h[p]);
      } else {
#pragma unroll
        for (int e = 0; e < N; ++e) h[p][e] = 0.f;
      }
    }
    if (a.residual) {
#pragma unroll
      for (int p = 0; p < P; ++p) {
        const int c = (p * W + lane) * N;
        if (c >= a.d) continue;
        float v[N];
        load_n<N>((const T *)a.residual + at + c, a.d - c, v);
#pragma unroll
        for (int e = 0; e < N; ++e) h[p][e] += v[e];
      }
    }
    if (a.sum) {  // after this lane's own loads of the piece: sum may be x or residual itself
#pragma unroll
      for (int p = 0; p < P; ++p) {
        const int c = (p * W + lane) * N;
        if (c < a.d) store_n<N>((T *)a.sum + at + c, a.d - c, h[p]);
      }
    }
#pragma unroll
    for (int p = 0; p < P; ++p)
#pragma unroll
      for (int e = 0; e < N; ++e) ss += h[p][e] * h[p][e];
    ss = row_sum<W>(ss, red);
    float mean = ss / (float)a.d + a.eps, factor = 1.f;
    if (out_of_range(mean)) {  // the same for the row's lanes
      factor = range_factor(mean);
      ss = 0.f;
#pragma unroll
      for (int p = 0; p < P; ++p)
#pragma unroll
        for (int e = 0; e < N; ++e) {
          h[p][e] *= factor;
          ss += h[p][e] * h[p][e];
        }
      ss = row_sum<W>(ss, red);
      mean = ss / (float)a.d + a.eps * factor * factor;
    }
    const float r = 1.f / sqrtf(mean);
    if (a.rstd && lane == 0) a.rstd[row] = r * factor;
    const bool f8 = a.y_type == RVQ_F8E4M3;
    uint32_t top = 0;
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int c = (p * W + lane) * N;
      if (c >= a.d) continue;
      float w[N];
      load_weight<N>(a.weight, a.w_bf16, c, a.d - c, w);
#pragma unroll
      for (int e = 0; e < N; ++e) h[p][e] = h[p][e] * r * w[e];
      if (f8) {
#pragma unroll
        for (int e = 0; e < N; ++e) top = max(top, magnitude_bits(h[p][e]));
      } else if (a.y_type == RVQ_BF16) {
        store_n<N>((uint16_t *)a.y + at + c, a.d - c, h[p]);
      } else {
        store_n<N>((float *)a.y + at + c, a.d - c, h[p]);
      }
    }
    if (f8) {
      const float scale = row_scale(row_max<W>(top, red));
      const float inv = 1.f / scale;
      if (lane == 0) a.scale[row] = scale;
#pragma unroll
      for (int p = 0; p < P; ++p) {
        const int c = (p * W + lane) * N;
        if (c >= a.d) continue;
#pragma unroll
        for (int e = 0; e < N; ++e) h[p][e] = nearest_quotient(h[p][e], scale, inv);
        store_f8_n<N>((uint8_t *)a.y + at + c, a.d - c, h[p]);
      }
    }
  }
}

// Rows too wide for registers: one workgroup per row, which is read again for
// each pass over it.  By elements, the simplest form that is right: no workload here
// has rows of more than 8192.  8,000 x 20,480 bf16 with residual: 811 us, 1.6 TB/s
// (gradient 798 us); 10,000 x 16,384, the widest that registers hold, 298 us.
template <typename T>
__global__ __launch_bounds__(kThreads) void rms_norm_wide_kernel(NormArgs a) {
  __shared__ float red[kThreads / 64];
  const T *x = (const T *)a.x, *res = (const T *)a.residual;
  for (int64_t row = blockIdx.x; row < a.n; row += gridDim.x) {
    const int64_t at = row * a.d;
    const auto h_of = [&](int i) {
      float h = load_f32(x, at + i);
      if (res) h += load_f32(res, at + i);
      return h;
    };
    const auto w_of = [&](int i) { return a.weight ? load_either(a.weight, a.w_bf16, i) : 1.f; };
    const auto mean_of = [&](float factor) {
      float ss = 0.f;
      for (int i = threadIdx.x; i < a.d; i += kThreads) {
        const float h = h_of(i) * factor;
        ss += h * h;
      }
      return row_sum<kThreads>(ss, red) / (float)a.d + a.eps * factor * factor;
    };
    float factor = 1.f, mean = mean_of(1.f);
    if (out_of_range(mean)) {
      factor = range_factor(mean);
      mean = mean_of(factor);
    }
    const float r = 1.f / sqrtf(mean);
    if (a.rstd && threadIdx.x == 0) a.rstd[row] = r * factor;
    float scale = 1.f, inv = 1.f;
    if (a.y_type == RVQ_F8E4M3) {
      uint32_t top = 0;
      for (int i = threadIdx.x; i < a.d; i += kThreads) top = max(top, magnitude_bits(h_of(i) * factor * r * w_of(i)));
      scale = row_scale(row_max<kThreads>(top, red));
      inv = 1.f / scale;
      if (threadIdx.x == 0) a.scale[row] = scale;
    }
    for (int i = threadIdx.x; i < a.d; i += kThreads) {
      const float h = h_of(i);
      const float y = h * factor * r * w_of(i);
      if (a.sum) store_f32((T *)a.sum, at + i, h);
      if (a.y_type == RVQ_F8E4M3)
        ((uint8_t *)a.y)[at + i] = f32_to_f8(nearest_quotient(y, scale, inv));
      else if (a.y_type == RVQ_BF16)
        store_f32((uint16_t *)a.y, at + i, y);
      else
        store_f32((float *)a.y, at + i, y);
    }
  }
}

template <typename T>
static hipError_t norm_rows(const NormArgs &a, hipStream_t s) {
  const Shape sh = shape_of(ceil_div(a.d, kPiece<T>));
  const int64_t groups = sh.w ? ceil_div(a.n, kThreads / sh.w) : a.n;
  const dim3 grid((unsigned)(groups < kMaxGroups ? groups : kMaxGroups));
#define RVQ_NORM(W, P)                                           \
  if (sh.w == W && sh.p == P) {                                  \
    rms_norm_kernel<T, W, P><<<grid, kThreads, 0, s>>>(a);       \
    return hipGetLastError();                                    \
  }
  RVQ_NORM_SHAPES(RVQ_NORM)
#undef RVQ_NORM
  rms_norm_wide_kernel<T><<<grid, kThreads, 0, s>>>(a);
  return hipGetLastError();
}

hipError_t launch_rms_norm(const NormArgs &a, bool x_bf16, hipStream_t s) {
  if (a.n == 0) return hipSuccess;
  return x_bf16 ? norm_rows<uint16_t>(a, s) : norm_rows<float>(a, s);
}

// ---- gradient ----
//   dx = r (g - u mean(g u)) + dsum with g = dy w, u = h r;  dw = sum over rows of dy u
// One pass: a workgroup takes rows blockIdx.x, + gridDim.x, ... and keeps its
// part of dw in registers; the parts are added in order by a second launch.
// The number of parts depends on n, d and the type alone, so the result does
// too.

namespace {

constexpr int kMaxParts = 1024;
constexpr int kWideParts = 256;

int rows_per_group(int64_t pieces) {
  const Shape sh = shape_of(pieces);
  return sh.w ? kThreads / sh.w : 1;
}

}  // namespace

int64_t norm_grad_parts(int64_t n, int d, bool bf16) {
  const int64_t pieces = ceil_div(d, bf16 ? kPiece<uint16_t> : kPiece<float>);
  if (n == 0) return 1;
  if (!shape_of(pieces).w) return n < kWideParts ? n : kWideParts;
  // two rows in turn before there are as many workgroups as the device holds
  const int64_t groups = ceil_div(n, 2 * rows_per_group(pieces));
  return groups < kMaxParts ? groups : kMaxParts;
}

// kMaxParts workgroups of four waves are as many as fit at once with 128
// registers, as the shapes up to two pieces of bf16 or four of fp32 have: a second
// round of fewer would cost as much as the first (39,731 x 4096 bf16: 1024
// workgroups 232 us, 1280 300 us).  The wider bf16 shapes and the widest fp32 one
// have more, and pay that round: 142 registers for three pieces of a wave's lanes
// (768 workgroups at once), 173 and over 256 for four and eight of a workgroup's
// (512, 256).  With dsum, with dweight and without: 39,731 x 1152 bf16 94 and 69 us
// (3.9 and 5.4 TB/s), 20,000 x 8192 301 and 277, 10,000 x 16,384 415 and 263.  All of
// a row's loads are issued before its sum; more waves hide the rest (holding the
// next row too was 2% slower).
template <typename T, int W, int P, bool DW>
__global__ __launch_bounds__(kThreads) void rms_norm_grad_kernel(NormGradArgs a) {
  constexpr int N = kPiece<T>, R = kThreads / W;
  __shared__ float red[kThreads / 64];
  const int lane = threadIdx.x % W;
  float acc[P][N];
#pragma unroll
  for (int p = 0; p < P; ++p)
#pragma unroll
    for (int e = 0; e < N; ++e) acc[p][e] = 0.f;
  for (int64_t row = (int64_t)blockIdx.x * R + threadIdx.x / W; row < a.n; row += (int64_t)gridDim.x * R) {
    const int64_t at = row * a.d;
    const float r = a.rstd[row];
    u32x4 q[P][3];
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int c = (p * W + lane) * N;
      q[p][0] = load_piece((const T *)a.dy + at + c, a.d - c);
      q[p][1] = load_piece((const T *)a.h + at + c, a.d - c);
      if (a.dsum) q[p][2] = load_piece((const T *)a.dsum + at + c, a.d - c);
    }
    float g[P][N], u[P][N];
#pragma unroll
    for (int p = 0; p < P; ++p) {
      unpack(q[p][0], g[p]);
      unpack(q[p][1], u[p]);
    }
    float dot = 0.f;
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int c = (p * W + lane) * N;
      if (c >= a.d) continue;
      float w[N];
      load_weight<N>(a.weight, a.w_bf16, c, a.d - c, w);
#pragma unroll
      for (int e = 0; e < N; ++e) {
        u[p][e] *= r;
        if (DW) acc[p][e] += g[p][e] * u[p][e];
        g[p][e] *= w[e];
        dot += g[p][e] * u[p][e];
      }
    }
    const float mean = row_sum<W>(dot, red) / (float)a.d;
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int c = (p * W + lane) * N;
      if (c >= a.d) continue;
      float v[N];
      if (a.dsum) {
        unpack(q[p][2], v);
      } else {
#pragma unroll
        for (int e = 0; e < N; ++e) v[e] = 0.f;
      }
#pragma unroll
      for (int e = 0; e < N; ++e) v[e] += r * (g[p][e] - u[p][e] * mean);
      // dx may be dy or dsum itself: both were loaded by this lane
      store_n<N>((T *)a.dx + at + c, a.d - c, v);
    }
  }
  if constexpr (DW) {
    float *part = a.part + (int64_t)blockIdx.x * a.d;
    if constexpr (R == 1) {
#pragma unroll
      for (int p = 0; p < P; ++p) {
        const int c = (p * W + lane) * N;
        if (c < a.d) store_n<N>(part + c, a.d - c, acc[p]);
      }
    } else {  // the workgroup's rows, in order
      constexpr int C = W * P * N;  // padded width
      __shared__ float sums[R * C];
#pragma unroll
      for (int p = 0; p < P; ++p)
#pragma unroll
        for (int e = 0; e < N; ++e) sums[(threadIdx.x / W) * C + (p * W + lane) * N + e] = acc[p][e];
      __syncthreads();
      for (int c = threadIdx.x; c < a.d; c += kThreads) {
        float s = 0.f;
#pragma unroll
        for (int q = 0; q < R; ++q) s += sums[q * C + c];
        part[c] = s;
      }
    }
  }
}

template <typename T>
__global__ __launch_bounds__(kThreads) void rms_norm_grad_wide_kernel(NormGradArgs a) {
  __shared__ float red[kThreads / 64];
  const T *dy = (const T *)a.dy, *h = (const T *)a.h, *ds = (const T *)a.dsum;
  for (int64_t row = blockIdx.x; row < a.n; row += gridDim.x) {
    const int64_t at = row * a.d;
    const float r = a.rstd[row];
    const auto w_of = [&](int i) { return a.weight ? load_either(a.weight, a.w_bf16, i) : 1.f; };
    float dot = 0.f;
    for (int i = threadIdx.x; i < a.d; i += kThreads)
      dot += load_f32(dy, at + i) * w_of(i) * (load_f32(h, at + i) * r);
    const float mean = row_sum<kThreads>(dot, red) / (float)a.d;
    for (int i = threadIdx.x; i < a.d; i += kThreads) {
      float v = r * (load_f32(dy, at + i) * w_of(i) - load_f32(h, at + i) * r * mean);
      if (ds) v += load_f32(ds, at + i);
      store_f32((T *)a.dx, at + i, v);
    }
  }
}

template <typename T>
__global__ __launch_bounds__(kThreads) void rms_norm_dweight_wide_kernel(NormGradArgs a, int64_t parts) {
  const int c = blockIdx.x * kThreads + threadIdx.x;
  const int64_t part = blockIdx.y;
  if (c >= a.d) return;
  const int64_t r0 = a.n * part / parts, r1 = a.n * (part + 1) / parts;
  float s = 0.f;
  for (int64_t r = r0; r < r1; ++r)
    s += load_f32((const T *)a.dy, r * a.d + c) * (load_f32((const T *)a.h, r * a.d + c) * a.rstd[r]);
  a.part[part * a.d + c] = s;
}

// Columns' sums over the parts: 64 columns a workgroup, a wave for every 1/16
// of the parts.
__global__ __launch_bounds__(1024) void rms_norm_dweight_join_kernel(const float *part, int64_t parts,
                                                                     int d, float *dweight) {
  __shared__ float sums[16][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int c = blockIdx.x * 64 + lane;
  float s = 0.f;
  if (c < d) {
    const int p1 = (int)(parts * (wave + 1) / 16);
#pragma unroll 8
    for (int p = (int)(parts * wave / 16); p < p1; ++p) s += part[(int64_t)p * d + c];
  }
  sums[wave][lane] = s;
  __syncthreads();
  if (wave == 0 && c < d) {
    s = 0.f;
#pragma unroll
    for (int w = 0; w < 16; ++w) s += sums[w][lane];
    dweight[c] = s;
  }
}

template <typename T>
static hipError_t norm_grad_rows(const NormGradArgs &a, hipStream_t s) {
  const int64_t parts = norm_grad_parts(a.n, a.d, sizeof(T) == 2);
  const Shape sh = shape_of(ceil_div(a.d, kPiece<T>));
  if (!sh.w || a.n == 0) {
    if (a.dweight)  // before dx, which may take the place of dy
      rms_norm_dweight_wide_kernel<T>
          <<<dim3((unsigned)ceil_div(a.d, kThreads), (unsigned)parts), kThreads, 0, s>>>(a, parts);
    if (a.n > 0)
      rms_norm_grad_wide_kernel<T>
          <<<dim3((unsigned)(a.n < kMaxGroups ? a.n : kMaxGroups)), kThreads, 0, s>>>(a);
  }
  const dim3 grid((unsigned)parts);
#define RVQ_NORM(W, P)                                                                    \
  if (a.n > 0 && sh.w == W && sh.p == P) {                                                \
    if (a.dweight)                                                                        \
      rms_norm_grad_kernel<T, W, P, true><<<grid, kThreads, 0, s>>>(a);                   \
    else                                                                                  \
      rms_norm_grad_kernel<T, W, P, false><<<grid, kThreads, 0, s>>>(a);                  \
  }
  RVQ_NORM_SHAPES(RVQ_NORM)
#undef RVQ_NORM
  if (a.dweight)
    rms_norm_dweight_join_kernel<<<dim3((unsigned)ceil_div(a.d, 64)), 1024, 0, s>>>(a.part, parts, a.d,
                                                                                    a.dweight);
  return hipGetLastError();
}

hipError_t launch_rms_norm_grad(const NormGradArgs &a, bool bf16, hipStream_t s) {
  return bf16 ? norm_grad_rows<uint16_t>(a, s) : norm_grad_rows<float>(a, s);
}

}  // namespace rvq
