// layer_norm.hip -- layer norm of rows, with the residual's addition and an
// 8-bit output, and its gradient.
//
//   h = x (+ residual),  m = mean(h),  r = 1 / sqrt(mean((h - m)^2) + eps),
//   y = (h - m) r w + b
//
// Everything between the loads and the stores is fp32.  The variance is that of
// the centred values, not a difference of large sums: a row is held in registers,
// its mean taken, and then the sums of c = h - m and of c^2 together.  The sum of
// c is the mean's own rounding error times d; it is taken out of the mean, of c
// and of the variance (which is summed once more where that is much of it), so that
// rows that lie far from zero lose nothing.
//
// Bound by memory, as the RMS norm: one read and one write of a row, shared by W
// lanes of P 16-byte pieces; rows of more than 2048 pieces are read again for each
// pass over them.  bf16 with weight and bias: 39,731 x 4096 129 us (5.0 TB/s; a copy takes 123),
// 37,003 x 1152 38 us (4.5), with residual and sum 277,777 x 1152 505 us (5.1); one row
// of 4096 with residual to 8 bits 4.0 us, which is a launch.
#include "head.h"
#include "lanes.h"
#include "rows.h"

namespace rvq {

namespace {

// Sums and largest values over the W lanes of a row.  For W == kThreads the waves meet
// in LDS, in two places by turns: whoever writes to one again has passed a barrier
// behind everyone's reading of it, so that one barrier a sum is enough.
template <int W>
struct Row {
  float (&red)[2][2 * kThreads / 64];
  int turn = 0;

  __device__ __forceinline__ void sums(float &a, float &b) {
    a = lane_sum<W < 64 ? W : 64>(a);
    b = lane_sum<W < 64 ? W : 64>(b);
    if constexpr (W > 64) {
      float *r = red[turn ^= 1];
      if ((threadIdx.x & 63) == 0) {
        r[2 * (threadIdx.x >> 6)] = a;
        r[2 * (threadIdx.x >> 6) + 1] = b;
      }
      __syncthreads();
      a = b = 0.f;
#pragma unroll
      for (int w = 0; w < W / 64; ++w) {
        a += r[2 * w];
        b += r[2 * w + 1];
      }
    }
  }
  __device__ __forceinline__ float sum(float v) {
    float none = 0.f;
    sums(v, none);
    return v;
  }
  __device__ __forceinline__ uint32_t top(uint32_t v) {
    v = lane_max_bits<W < 64 ? W : 64>(v);
    if constexpr (W > 64) {
      float *r = red[turn ^= 1];
      if ((threadIdx.x & 63) == 0) r[threadIdx.x >> 6] = __uint_as_float(v);
      __syncthreads();
      v = __float_as_uint(r[0]);
#pragma unroll
      for (int w = 1; w < W / 64; ++w) v = max(v, __float_as_uint(r[w]));
    }
    return v;
  }
};

// weight or bias; `none` where there is none
template <int N>
__device__ __forceinline__ void load_param(const void *w, bool bf16, int c, int left, float none, float (&v)[N]) {
  if (!w) {
#pragma unroll
    for (int e = 0; e < N; ++e) v[e] = none;
  } else {
    load_weight<N>(w, bf16, c, left, v);
  }
}

// Rows whose squares leave fp32.  Too large (a mean square that is not below
// 2^100; NaN and infinity come here too and stay what they are): the values are
// taken times kDown before their mean, which brings them below 2^48.  Too small (a
// variance plus eps below 2^-100): the centred values are taken times kUp.
constexpr float kDown = 0x1p-80f, kUp = 0x1p70f;
__device__ __forceinline__ bool too_large(float mean_square) { return !(mean_square < 0x1p100f); }

// 1 / sqrt(var + eps), and what the centred values as taken are multiplied by.
struct Root {
  float rstd, r;
};
// Of values times kDown.  In 64 bits, since eps times kDown^2 is nothing in 32;
// equal values far from zero have a variance of 0 and r at its largest.
__device__ __forceinline__ Root root_down(float var, float eps) {
  const double rstd = 1.0 / sqrt((double)var * 0x1p160 + (double)eps);
  const double r = rstd * 0x1p80;
  return {(float)rstd, r < 3e38 ? (float)r : (r == r ? 3e38f : NAN)};
}
// Of values as they are, or (small) times kUp.
__device__ __forceinline__ Root root_of(float var, float eps, bool down, bool small) {
  if (down) return root_down(var, eps);
  if (small) {
    const float r = 1.f / sqrtf(var + eps * kUp * kUp);
    return {r * kUp, r};
  }
  const float r = 1.f / sqrtf(var + eps);
  return {r, r};
}

// A mean as it is rounded.  Left to the compiler, s * inv_d becomes a part of some of
// the differences h - m (one fma, with the product unrounded) and not of others, and
// rows far from zero are centred at two places.
__device__ __forceinline__ float rounded(float v) {
  asm("" : "+v"(v));
  return v;
}

// fmaxf without NaN's loss
__device__ __forceinline__ float not_negative(float v) { return v < 0.f ? 0.f : v; }

}  // namespace

// What a lane keeps from row to row: its parts of weight and bias (up to 24 values of
// each), which would otherwise be read from the L2 again for every row, four times the bytes of
// a bf16 row, and the next row's bytes, which come while this one is summed.
template <int P, int N>
constexpr bool kKeep = P * N <= 24;
// Workgroups of a launch: as many as are at work at once with these registers (of the
// narrowest shapes, twice as many).  39,731 x 4096 bf16 129 us with four a CU, 152 with five, of
// which one begins when the others end.
template <int P, int N>
constexpr int kAtOnce = 256 * (P * N <= 8 ? 12 : P * N <= 16 ? 4 : P * N <= 24 ? 3 : 16);

template <typename T, int W, int P>
__global__ __launch_bounds__(kThreads) void layer_norm_kernel(LayerNormArgs a) {
  constexpr int N = kPiece<T>, R = kThreads / W;
  constexpr bool keep = kKeep<P, N>;
  __shared__ float red[2][2 * kThreads / 64];
  Row<W> over{red};
  const int lane = threadIdx.x % W;
  const float inv_d = 1.f / (float)a.d;
  float w[P][N], b[P][N];
  const auto params = [&](int p) {
    const int c = (p * W + lane) * N;
    load_param<N>(a.weight, a.w_bf16, c, a.d - c, 1.f, w[p]);
    load_param<N>(a.bias, a.w_bf16, c, a.d - c, 0.f, b[p]);
  };
  u32x4 raw[P], raw_res[P];
  const auto load = [&](int64_t row) {
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int c = (p * W + lane) * N;
      raw[p] = load_piece((const T *)a.x + row * a.d + c, a.d - c);
      if (a.residual) raw_res[p] = load_piece((const T *)a.residual + row * a.d + c, a.d - c);
    }
  };
  const int64_t first = (int64_t)blockIdx.x * R + threadIdx.x / W, stride = (int64_t)gridDim.x * R;
  if (keep && first < a.n) load(first);
  if constexpr (keep) {
#pragma unroll
    for (int p = 0; p < P; ++p) params(p);
  }
  // W == kThreads: the row is the same for the whole workgroup, as the barriers need
  for (int64_t row = first; row < a.n; row += stride) {
    const int64_t at = row * a.d;
    if (!keep) load(row);
    float h[P][N];
#pragma unroll
    for (int p = 0; p < P; ++p) {
      unpack(raw[p], h[p]);
      if (a.residual) {
        float v[N];
        unpack(raw_res[p], v);
#pragma unroll
        for (int e = 0; e < N; ++e) h[p][e] += v[e];
      }
    }
    if (keep && row + stride < a.n) load(row + stride);
    if (a.sum) {  // after this lane's own loads of the piece: sum may be x or residual itself
#pragma unroll
      for (int p = 0; p < P; ++p) {
        const int c = (p * W + lane) * N;
        if (c < a.d) store_n<N>((T *)a.sum + at + c, a.d - c, h[p]);
      }
    }
    float s = 0.f, s2 = 0.f;
#pragma unroll
    for (int p = 0; p < P; ++p)
#pragma unroll
      for (int e = 0; e < N; ++e) {
        s += h[p][e];
        s2 += h[p][e] * h[p][e];
      }
    over.sums(s, s2);
    const bool down = too_large(s2 * inv_d);  // the same for the row's lanes, as what follows from it
    if (down) {
      s = 0.f;
#pragma unroll
      for (int p = 0; p < P; ++p)
#pragma unroll
        for (int e = 0; e < N; ++e) {
          h[p][e] *= kDown;
          s += h[p][e];
        }
      s = over.sum(s);
    }
    float m = rounded(s * inv_d);
    float s1 = 0.f;
    s2 = 0.f;
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int left = a.d - (p * W + lane) * N;
      if (left >= N) {
#pragma unroll
        for (int e = 0; e < N; ++e) h[p][e] -= m;
      } else {  // what is not of the row stays 0
#pragma unroll
        for (int e = 0; e < N; ++e) h[p][e] = e < left ? h[p][e] - m : 0.f;
      }
#pragma unroll
      for (int e = 0; e < N; ++e) {
        s1 += h[p][e];
        s2 += h[p][e] * h[p][e];
      }
    }
    over.sums(s1, s2);
    const float off = rounded(s1 * inv_d);  // what m was short of
    m += off;
    float var = not_negative(s2 * inv_d - off * off);
    float shift = off;
    // a row far from zero, or one of very small differences: its squares are taken again
    const bool small = !down && var + a.eps < 0x1p-100f;
    float up = 1.f;
    if (small || off * off > 0x1p-10f * (down ? var : var + a.eps)) {
      up = small ? kUp : 1.f;
      s2 = 0.f;
#pragma unroll
      for (int p = 0; p < P; ++p) {
        const int left = a.d - (p * W + lane) * N;
#pragma unroll
        for (int e = 0; e < N; ++e) {
          h[p][e] = e < left ? (h[p][e] - off) * up : 0.f;
          s2 += h[p][e] * h[p][e];
        }
      }
      shift = 0.f;
      var = over.sum(s2) * inv_d;
    }
    const Root root = root_of(var, a.eps, down, small);
    if (lane == 0) {
      if (a.mean) a.mean[row] = down ? m * 0x1p80f : m;
      if (a.rstd) a.rstd[row] = root.rstd;
    }
    const float r = root.r;
    const bool f8 = a.y_type == RVQ_F8E4M3;
    uint32_t top = 0;
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int c = (p * W + lane) * N;
      if (c >= a.d) continue;
      if (!keep) params(p);
#pragma unroll
      for (int e = 0; e < N; ++e) h[p][e] = (h[p][e] - shift) * r * w[p][e] + b[p][e];
      if (f8) {
#pragma unroll
        for (int e = 0; e < N; ++e)
          if (c + e < a.d) top = max(top, magnitude_bits(h[p][e]));
      } else if (a.y_type == RVQ_BF16) {
        store_n<N>((uint16_t *)a.y + at + c, a.d - c, h[p]);
      } else {
        store_n<N>((float *)a.y + at + c, a.d - c, h[p]);
      }
    }
    if (f8) {
      const float scale = row_scale_of(over.top(top));
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
// each pass over it, by elements.  Bound by these loads: 4000 x 20,000 bf16 300 us (1.1 TB/s of
// its bytes once), 1000 x 65,536 298, 2000 x 20,000 fp32 174; the gradient 304, 446 and 232.
template <typename T>
__global__ __launch_bounds__(kThreads) void layer_norm_wide_kernel(LayerNormArgs a) {
  __shared__ float red[2][2 * kThreads / 64];
  Row<kThreads> over{red};
  const T *x = (const T *)a.x, *res = (const T *)a.residual;
  const float inv_d = 1.f / (float)a.d;
  for (int64_t row = blockIdx.x; row < a.n; row += gridDim.x) {
    const int64_t at = row * a.d;
    const auto h_of = [&](int i) {
      float h = load_f32(x, at + i);
      if (res) h += load_f32(res, at + i);
      return h;
    };
    float s = 0.f, s2 = 0.f;
    for (int i = threadIdx.x; i < a.d; i += kThreads) {
      const float h = h_of(i);
      s += h;
      s2 += h * h;
    }
    over.sums(s, s2);
    const bool down = too_large(s2 * inv_d);
    const float f = down ? kDown : 1.f;
    if (down) {
      s = 0.f;
      for (int i = threadIdx.x; i < a.d; i += kThreads) s += h_of(i) * f;
      s = over.sum(s);
    }
    float m = rounded(s * inv_d), s1 = 0.f;
    s2 = 0.f;
    for (int i = threadIdx.x; i < a.d; i += kThreads) {
      const float c = h_of(i) * f - m;
      s1 += c;
      s2 += c * c;
    }
    over.sums(s1, s2);
    const float off = rounded(s1 * inv_d);
    float var = not_negative(s2 * inv_d - off * off), up = 1.f;
    const bool small = !down && var + a.eps < 0x1p-100f;
    if (small || off * off > 0x1p-10f * (down ? var : var + a.eps)) {
      up = small ? kUp : 1.f;
      s2 = 0.f;
      for (int i = threadIdx.x; i < a.d; i += kThreads) {
        const float c = ((h_of(i) * f - m) - off) * up;
        s2 += c * c;
      }
      var = over.sum(s2) * inv_d;
    }
    const Root root = root_of(var, a.eps, down, small);
    if (threadIdx.x == 0) {
      if (a.mean) a.mean[row] = down ? (m + off) * 0x1p80f : m + off;
      if (a.rstd) a.rstd[row] = root.rstd;
    }
    const auto y_of = [&](float h, int i) {
      const float w = a.weight ? load_either(a.weight, a.w_bf16, i) : 1.f;
      const float b = a.bias ? load_either(a.bias, a.w_bf16, i) : 0.f;
      return ((h * f - m) - off) * up * root.r * w + b;
    };
    float scale = 1.f, inv = 1.f;
    if (a.y_type == RVQ_F8E4M3) {
      uint32_t top = 0;
      for (int i = threadIdx.x; i < a.d; i += kThreads) top = max(top, magnitude_bits(y_of(h_of(i), i)));
      scale = row_scale_of(over.top(top));
      inv = 1.f / scale;
      if (threadIdx.x == 0) a.scale[row] = scale;
    }
    for (int i = threadIdx.x; i < a.d; i += kThreads) {
      const float h = h_of(i);
      const float y = y_of(h, i);
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
static hipError_t layer_norm_rows(const LayerNormArgs &a, hipStream_t s) {
  const Shape sh = shape_of(ceil_div(a.d, kPiece<T>));
  const int64_t groups = sh.w ? ceil_div(a.n, kThreads / sh.w) : a.n;
  const auto grid = [&](int64_t most) { return dim3((unsigned)(groups < most ? groups : most)); };
#define RVQ_NORM(W, P)                                                                                \
  if (sh.w == W && sh.p == P) {                                                                       \
    layer_norm_kernel<T, W, P><<<grid(kAtOnce<P, kPiece<T>>), kThreads, 0, s>>>(a);                   \
    return hipGetLastError();                                                                         \
  }
  RVQ_NORM_SHAPES(RVQ_NORM)
#undef RVQ_NORM
  layer_norm_wide_kernel<T><<<grid(kMaxGroups), kThreads, 0, s>>>(a);
  return hipGetLastError();
}

hipError_t launch_layer_norm(const LayerNormArgs &a, bool x_bf16, hipStream_t s) {
  if (a.n == 0) return hipSuccess;
  return x_bf16 ? layer_norm_rows<uint16_t>(a, s) : layer_norm_rows<float>(a, s);
}

// ---- gradient ----
//   dx = r (g - mean(g) - u mean(g u)) + dsum with g = dy w, u = (h - m) r;
//   dw = sum over rows of dy u,  db = sum over rows of dy
// One pass: a workgroup takes rows blockIdx.x, + gridDim.x, ... and keeps its
// parts of dw and db in registers; the parts are added in order by a second
// launch.  The number of parts depends on n, d and the type alone, so the result
// does too.
// h - m can be beyond fp32 where h and m are not (values of both signs near its largest):
// where m is large, both are halved and r is doubled, for the cost of an fma in place of a
// difference and with the same bits.
// Bound by memory: 39,731 x 4096 bf16 with dsum 236 us (5.6 TB/s) and 6 for the parts; 1024 x
// 1152 fp32, two rows in turn, 7.2 and 4.4.

namespace {

// u = (h - m) r = (h f - m f) (r / f); h f is exact inside the fma
struct Centre {
  float f, mf, rf;
  __device__ __forceinline__ Centre(float m, float r) : f(fabsf(m) > 0x1p100f ? 0.5f : 1.f) {
    mf = m * f;
    rf = f < 1.f ? r * 2.f : r;
  }
  __device__ __forceinline__ float u(float h) const { return __builtin_fmaf(h, f, -mf) * rf; }
};

// Workgroups of a launch, and with them the parts: three a CU, which are at work at once
// with most shapes' registers (277,777 x 1152 bf16 476 us, 621 with four; 78,125 x 4096 459 and
// 474; 39,062 x 4096 fp32 464 and 541; the other way round 138,888 x 1152 fp32 501 and
// 488).  Four of the widest, which two or one a CU are at work on (52,083 x 6144 bf16 480, 564
// with three; without parameters, where it is three, 564 and 458).
int most_at_once(const Shape &sh, int piece, bool params) {
  const int values = sh.p * piece;
  return values < 32 || (values == 32 && piece == 8 && !params) ? 768 : 1024;
}
constexpr int kWideParts = 256;

}  // namespace

int64_t layer_norm_grad_parts(int64_t n, int d, bool bf16) {
  const Shape sh = shape_of(ceil_div(d, bf16 ? kPiece<uint16_t> : kPiece<float>));
  if (n == 0) return 1;
  if (!sh.w) return n < kWideParts ? n : kWideParts;
  // two rows in turn before there are as many workgroups as the device holds
  const int64_t groups = ceil_div(n, 2 * (kThreads / sh.w));
  const int most = most_at_once(sh, bf16 ? kPiece<uint16_t> : kPiece<float>, true);
  return groups < most ? groups : most;
}

template <typename T, int W, int P, bool DW>
__global__ __launch_bounds__(kThreads) void layer_norm_grad_kernel(LayerNormGradArgs a) {
  constexpr int N = kPiece<T>, R = kThreads / W;
  __shared__ float red[2][2 * kThreads / 64];
  Row<W> over{red};
  const int lane = threadIdx.x % W;
  float acc[P][N], accb[P][N];
#pragma unroll
  for (int p = 0; p < P; ++p)
#pragma unroll
    for (int e = 0; e < N; ++e) acc[p][e] = accb[p][e] = 0.f;
  for (int64_t row = (int64_t)blockIdx.x * R + threadIdx.x / W; row < a.n; row += (int64_t)gridDim.x * R) {
    const int64_t at = row * a.d;
    const float r = a.rstd[row];
    const Centre centre(a.mean[row], r);
    u32x4 q[P][3];
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int c = (p * W + lane) * N;
      q[p][0] = load_piece((const T *)a.dy + at + c, a.d - c);
      q[p][1] = load_piece((const T *)a.h + at + c, a.d - c);
      if (a.dsum) q[p][2] = load_piece((const T *)a.dsum + at + c, a.d - c);
    }
    float g[P][N], u[P][N];
    float sum = 0.f, dot = 0.f;
#pragma unroll
    for (int p = 0; p < P; ++p) {
      unpack(q[p][0], g[p]);
      unpack(q[p][1], u[p]);
      const int c = (p * W + lane) * N;
      if (c >= a.d) continue;
      float w[N];
      load_weight<N>(a.weight, a.w_bf16, c, a.d - c, w);
#pragma unroll
      for (int e = 0; e < N; ++e) u[p][e] = centre.u(u[p][e]);
      if (a.d - c < N) {  // what is not of the row: 0, where m times r may be beyond fp32 (and dy, 0, is no help)
#pragma unroll
        for (int e = 1; e < N; ++e)
          if (c + e >= a.d) u[p][e] = 0.f;
      }
#pragma unroll
      for (int e = 0; e < N; ++e) {
        if (DW) {
          acc[p][e] += g[p][e] * u[p][e];
          accb[p][e] += g[p][e];
        }
        g[p][e] *= w[e];
        sum += g[p][e];
        dot += g[p][e] * u[p][e];
      }
    }
    over.sums(sum, dot);
    const float mg = sum / (float)a.d, mu = dot / (float)a.d;
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
      for (int e = 0; e < N; ++e) v[e] += r * ((g[p][e] - mg) - u[p][e] * mu);
      // dx may be dy or dsum itself: both were loaded by this lane
      store_n<N>((T *)a.dx + at + c, a.d - c, v);
    }
  }
  if constexpr (DW) {
    float *part = a.part + (int64_t)blockIdx.x * 2 * a.d;
    if constexpr (R == 1) {
#pragma unroll
      for (int p = 0; p < P; ++p) {
        const int c = (p * W + lane) * N;
        if (c >= a.d) continue;
        store_n<N>(part + c, a.d - c, acc[p]);
        store_n<N>(part + a.d + c, a.d - c, accb[p]);
      }
    } else {  // the workgroup's rows, in order
      constexpr int C = W * P * N;  // padded width
      __shared__ float sums[R * C];
#pragma unroll
      for (int which = 0; which < 2; ++which) {
        __syncthreads();
#pragma unroll
        for (int p = 0; p < P; ++p)
#pragma unroll
          for (int e = 0; e < N; ++e)
            sums[(threadIdx.x / W) * C + (p * W + lane) * N + e] = which ? accb[p][e] : acc[p][e];
        __syncthreads();
        for (int c = threadIdx.x; c < a.d; c += kThreads) {
          float s = 0.f;
#pragma unroll
          for (int q = 0; q < R; ++q) s += sums[q * C + c];
          part[which * a.d + c] = s;
        }
      }
    }
  }
}

template <typename T>
__global__ __launch_bounds__(kThreads) void layer_norm_grad_wide_kernel(LayerNormGradArgs a) {
  __shared__ float red[2][2 * kThreads / 64];
  Row<kThreads> over{red};
  const T *dy = (const T *)a.dy, *h = (const T *)a.h, *ds = (const T *)a.dsum;
  for (int64_t row = blockIdx.x; row < a.n; row += gridDim.x) {
    const int64_t at = row * a.d;
    const float r = a.rstd[row];
    const Centre centre(a.mean[row], r);
    const auto g_of = [&](int i) {
      return load_f32(dy, at + i) * (a.weight ? load_either(a.weight, a.w_bf16, i) : 1.f);
    };
    const auto u_of = [&](int i) { return centre.u(load_f32(h, at + i)); };
    float sum = 0.f, dot = 0.f;
    for (int i = threadIdx.x; i < a.d; i += kThreads) {
      const float g = g_of(i);
      sum += g;
      dot += g * u_of(i);
    }
    over.sums(sum, dot);
    const float mg = sum / (float)a.d, mu = dot / (float)a.d;
    for (int i = threadIdx.x; i < a.d; i += kThreads) {
      float v = r * ((g_of(i) - mg) - u_of(i) * mu);
      if (ds) v += load_f32(ds, at + i);
      store_f32((T *)a.dx, at + i, v);
    }
  }
}

template <typename T>
__global__ __launch_bounds__(kThreads) void layer_norm_params_wide_kernel(LayerNormGradArgs a, int64_t parts) {
  const int c = blockIdx.x * kThreads + threadIdx.x;
  const int64_t part = blockIdx.y;
  if (c >= a.d) return;
  const int64_t r0 = a.n * part / parts, r1 = a.n * (part + 1) / parts;
  float s = 0.f, b = 0.f;
  for (int64_t r = r0; r < r1; ++r) {
    const float dy = load_f32((const T *)a.dy, r * a.d + c);
    s += dy * Centre(a.mean[r], a.rstd[r]).u(load_f32((const T *)a.h, r * a.d + c));
    b += dy;
  }
  a.part[part * 2 * a.d + c] = s;
  a.part[(part * 2 + 1) * a.d + c] = b;
}

// Columns' sums over the parts: 64 columns a workgroup, a wave for every 1/16
// of the parts; columns d .. 2d - 1 are dbias'.  In 64 bits: the parts of few rows are many
// beside what each of them sums (1024 x 1152 fp32: 512 of two rows, the result's error 4e-8 and
// 2.3e-7 in 32 bits), and the kernel waits for its loads (4.0 us there in 32 bits, 4.4 in 64).
__global__ __launch_bounds__(1024) void layer_norm_params_join_kernel(const float *part, int64_t parts, int d,
                                                                      float *dweight, float *dbias) {
  __shared__ double sums[16][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int c = blockIdx.x * 64 + lane;
  double s = 0.0;
  if (c < 2 * d) {
    const int p1 = (int)(parts * (wave + 1) / 16);
#pragma unroll 8
    for (int p = (int)(parts * wave / 16); p < p1; ++p) s += (double)part[(int64_t)p * 2 * d + c];
  }
  sums[wave][lane] = s;
  __syncthreads();
  if (wave == 0 && c < 2 * d) {
    s = 0.0;
#pragma unroll
    for (int w = 0; w < 16; ++w) s += sums[w][lane];
    if (c < d) {
      if (dweight) dweight[c] = (float)s;
    } else if (dbias) {
      dbias[c - d] = (float)s;
    }
  }
}

template <typename T>
static hipError_t layer_norm_grad_rows(const LayerNormGradArgs &a, hipStream_t s) {
  const int64_t parts = layer_norm_grad_parts(a.n, a.d, sizeof(T) == 2);
  const Shape sh = shape_of(ceil_div(a.d, kPiece<T>));
  const bool params = a.dweight || a.dbias;
  if (!sh.w || a.n == 0) {
    if (params)  // before dx, which may take the place of dy
      layer_norm_params_wide_kernel<T>
          <<<dim3((unsigned)ceil_div(a.d, kThreads), (unsigned)parts), kThreads, 0, s>>>(a, parts);
    if (a.n > 0)
      layer_norm_grad_wide_kernel<T>
          <<<dim3((unsigned)(a.n < kMaxGroups ? a.n : kMaxGroups)), kThreads, 0, s>>>(a);
  }
  const int64_t most = most_at_once(sh, kPiece<T>, params);
  const dim3 grid((unsigned)(params || parts < most ? parts : most));
#define RVQ_NORM(W, P)                                                                    \
  if (a.n > 0 && sh.w == W && sh.p == P) {                                                \
    if (params)                                                                           \
      layer_norm_grad_kernel<T, W, P, true><<<grid, kThreads, 0, s>>>(a);                 \
    else                                                                                  \
      layer_norm_grad_kernel<T, W, P, false><<<grid, kThreads, 0, s>>>(a);                \
  }
  RVQ_NORM_SHAPES(RVQ_NORM)
#undef RVQ_NORM
  if (params)
    layer_norm_params_join_kernel<<<dim3((unsigned)ceil_div(2 * (int64_t)a.d, 64)), 1024, 0, s>>>(
        a.part, parts, a.d, a.dweight, a.dbias);
  return hipGetLastError();
}

hipError_t launch_layer_norm_grad(const LayerNormGradArgs &a, bool bf16, hipStream_t s) {
  return bf16 ? layer_norm_grad_rows<uint16_t>(a, s) : layer_norm_grad_rows<float>(a, s);
}

}  // namespace rvq
