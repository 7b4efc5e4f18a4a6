// norm.hip -- root-mean-square norm of rows, with the residual's addition
// and an 8-bit output, and its gradient.
//
//   h = x (+ residual),  r = 1 / sqrt(mean(h^2) + eps),  y = h r w
//
// Everything between the loads and the stores is fp32; h is rounded to the
// rows' type only where it is stored, and the norm uses the unrounded sum.
#include "learn.h"

namespace rvq {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxGroups = 1 << 20;  // workgroups of a launch; rows beyond are looped over

__device__ __forceinline__ float block_sum(float v, float *red) {
  v = wave_sum_f32(v);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  float s = 0.f;
#pragma unroll
  for (int w = 0; w < kThreads / 64; ++w) s += red[w];
  return s;
}

__device__ __forceinline__ float block_max(float v, float *red) {
  v = wave_max_f32(v);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  float s = red[0];
#pragma unroll
  for (int w = 1; w < kThreads / 64; ++w) s = fmaxf(s, red[w]);
  return s;
}

}  // namespace

// One workgroup per row, which is read again for each pass over it.
template <typename T>
__global__ __launch_bounds__(kThreads) void rms_norm_kernel(NormArgs a) {
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
    float ss = 0.f;
    for (int i = threadIdx.x; i < a.d; i += kThreads) {
      const float h = h_of(i);
      ss += h * h;
    }
    ss = block_sum(ss, red);
    const float r = 1.f / sqrtf(ss / (float)a.d + a.eps);
    if (a.rstd && threadIdx.x == 0) a.rstd[row] = r;
    float inv = 1.f;
    if (a.y_type == RVQ_F8E4M3) {
      float top = 0.f;
      for (int i = threadIdx.x; i < a.d; i += kThreads) top = fmaxf(top, fabsf(h_of(i) * r * w_of(i)));
      top = block_max(top, red);
      // a row that holds NaN or infinity gets the scale NaN
      const float scale = fmaxf(top / kF8Max, kScaleMin) + (ss - ss);
      inv = 1.f / scale;
      if (threadIdx.x == 0) a.scale[row] = scale;
    }
    for (int i = threadIdx.x; i < a.d; i += kThreads) {
      const float h = h_of(i);
      const float y = h * r * w_of(i);
      // stored after this thread's own loads of the element: sum may be x or residual itself
      if (a.sum) store_f32((T *)a.sum, at + i, h);
      if (a.y_type == RVQ_F8E4M3)
        ((uint8_t *)a.y)[at + i] = f32_to_f8(clamp_f8(y * inv));
      else if (a.y_type == RVQ_BF16)
        store_f32((uint16_t *)a.y, at + i, y);
      else
        store_f32((float *)a.y, at + i, y);
    }
  }
}

hipError_t launch_rms_norm(const NormArgs &a, bool x_bf16, hipStream_t s) {
  if (a.n == 0) return hipSuccess;
  const dim3 grid((unsigned)(a.n < kMaxGroups ? a.n : kMaxGroups));
  if (x_bf16)
    rms_norm_kernel<uint16_t><<<grid, kThreads, 0, s>>>(a);
  else
    rms_norm_kernel<float><<<grid, kThreads, 0, s>>>(a);
  return hipGetLastError();
}

// ---- gradient ----
//   dx = r (g - h r mean(g h r)) + dsum with g = dy w;  dw = sum over rows of dy h r
// The rows' sum is taken in fixed parts of consecutive rows, and the parts
// in order, so it depends on n alone.

template <typename T>
__global__ __launch_bounds__(kThreads) void rms_norm_grad_kernel(NormGradArgs a) {
  __shared__ float red[kThreads / 64];
  const T *dy = (const T *)a.dy, *h = (const T *)a.h, *ds = (const T *)a.dsum;
  for (int64_t row = blockIdx.x; row < a.n; row += gridDim.x) {
    const int64_t at = row * a.d;
    const float r = a.rstd[row];
    const auto w_of = [&](int i) { return a.weight ? load_either(a.weight, a.w_bf16, i) : 1.f; };
    float dot = 0.f;
    for (int i = threadIdx.x; i < a.d; i += kThreads)
      dot += load_f32(dy, at + i) * w_of(i) * (load_f32(h, at + i) * r);
    const float mean = block_sum(dot, red) / (float)a.d;
    for (int i = threadIdx.x; i < a.d; i += kThreads) {
      float v = r * (load_f32(dy, at + i) * w_of(i) - load_f32(h, at + i) * r * mean);
      if (ds) v += load_f32(ds, at + i);
      store_f32((T *)a.dx, at + i, v);
    }
  }
}

template <typename T>
__global__ __launch_bounds__(kThreads) void rms_norm_dweight_kernel(NormGradArgs a, int64_t parts) {
  const int c = blockIdx.x * kThreads + threadIdx.x;
  const int64_t part = blockIdx.y;
  if (c >= a.d) return;
  const int64_t r0 = a.n * part / parts, r1 = a.n * (part + 1) / parts;
  float s = 0.f;
  for (int64_t r = r0; r < r1; ++r)
    s += load_f32((const T *)a.dy, r * a.d + c) * (load_f32((const T *)a.h, r * a.d + c) * a.rstd[r]);
  a.part[part * a.d + c] = s;
}

__global__ __launch_bounds__(kThreads) void rms_norm_dweight_join_kernel(const float *part,
                                                                         int64_t parts, int d,
                                                                         float *dweight) {
  const int c = blockIdx.x * kThreads + threadIdx.x;
  if (c >= d) return;
  float s = 0.f;
  for (int64_t p = 0; p < parts; ++p) s += part[p * d + c];
  dweight[c] = s;
}

int64_t norm_grad_parts(int64_t n) { return n < 256 ? (n > 0 ? n : 1) : 256; }

hipError_t launch_rms_norm_grad(const NormGradArgs &a, bool bf16, hipStream_t s) {
  const unsigned cols = (unsigned)ceil_div(a.d, kThreads);
  if (a.dweight) {  // before dx, which may take the place of dy
    const int64_t parts = norm_grad_parts(a.n);
    const dim3 grid(cols, (unsigned)parts);
    if (bf16)
      rms_norm_dweight_kernel<uint16_t><<<grid, kThreads, 0, s>>>(a, parts);
    else
      rms_norm_dweight_kernel<float><<<grid, kThreads, 0, s>>>(a, parts);
    rms_norm_dweight_join_kernel<<<cols, kThreads, 0, s>>>(a.part, parts, a.d, a.dweight);
  }
  if (a.n == 0) return hipGetLastError();
  const dim3 grid((unsigned)(a.n < kMaxGroups ? a.n : kMaxGroups));
  if (bf16)
    rms_norm_grad_kernel<uint16_t><<<grid, kThreads, 0, s>>>(a);
  else
    rms_norm_grad_kernel<float><<<grid, kThreads, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace rvq
