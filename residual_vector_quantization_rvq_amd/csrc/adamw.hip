// adamw.hip -- one AdamW step over many tensors at once.
//
//   g' = c g,  c = grad_scale min(1, max_norm / (norm + 1e-6))
//   m = b1 m + (1 - b1) g',   v = b2 v + (1 - b2) g'^2
//   p = p (1 - lr wd) - lr / (1 - b1^t) m / (sqrt(v) / sqrt(1 - b2^t) + eps)
//
// All in fp32 and with the moments as they are before they are stored.
//
// 8-bit states.  m and sqrt(v) are held as e4m3 with an fp32 scale for every
// kBlock elements (the block's largest value / 448).  The root is stored, and
// not v, because its range is half of v's in powers of two: e4m3 with a scale
// spans 2^-18 of the block's largest root, 2^-36 of its largest v.  With
// b2 = 0.999 one step moves sqrt(v) by about 1/2000 of itself and the grid's
// step is 1/16 to 1/8 of the value: rounded to nearest it would never move.
// So a step that is given a seed rounds at random, up with the probability of
// the remainder, from bits that are a hash of (seed, step, tensor, element);
// bf16 parameters, where lr times the update is often under half a step, are
// rounded the same way.
//
// The tensors' pointers travel as kernel arguments, kTable tensors a launch:
// nothing is copied, allocated or kept between calls.
#include "learn.h"

namespace rvq {

namespace {

constexpr int kThreads = 256;
constexpr int kTable = 40;          // tensors of one launch (kernel arguments: 4 KB)
constexpr int kChunk = 2048;        // elements of one workgroup; a multiple of kBlock
constexpr int kBlock = 256;         // elements that share a scale
constexpr int kNormGroups = 1024;   // partial sums of squares of one launch

struct Entry {
  void *p;
  const void *g;
  void *m, *v;
  float *ms, *vs;
  uint16_t *copy;
  int64_t n;
  int64_t chunk0;   // first workgroup of this tensor
  float decay;      // 1 - lr wd
  uint32_t base;    // rounding bits: mixed from (seed, step, tensor)
};
struct Table {
  Entry e[kTable];
  int count;
  int64_t chunks;
};
struct Consts {
  float b1, c1, b2, c2;  // c = 1 - b, from the 64-bit b: 1.f - 0.999f is 1e-5 off
  float eps, lr1, rk2, grad_scale, max_norm;
  bool stochastic;
};

// 32 bits mixed from 32: xor of the high half, odd multipliers from the
// fractions of sqrt(2) and sqrt(3)
__host__ __device__ inline uint32_t mix(uint32_t x) {
  x ^= x >> 16;
  x *= 0x3504F333u;
  x ^= x >> 15;
  x *= 0x5DB3D743u;
  return x ^ (x >> 16);
}
__device__ __forceinline__ uint32_t round_bits(uint32_t base, int64_t i) {
  return mix(base + (uint32_t)i * 0x9E3779B1u + (uint32_t)(i >> 32) * 0x3504F333u);
}

// |v| <= 448 rounded to the e4m3 grid at random: 20 random bits are added
// under the three bits of the mantissa that stay.  Below 2^-6 the grid is
// that of 2^-6, reached by adding it for the rounding.
__device__ __forceinline__ float round_f8(float v, uint32_t random20) {
  const float a = fabsf(v);
  const bool small = a < 0x1p-6f;
  float r = __uint_as_float((__float_as_uint(small ? a + 0x1p-6f : a) + random20) & 0xfff00000u);
  r = fminf(small ? r - 0x1p-6f : r, kF8Max);
  return copysignf(r, v);
}
__device__ __forceinline__ float round_bf16(float v, uint32_t random16) {
  return __uint_as_float((__float_as_uint(v) + random16) & 0xffff0000u);
}

// the entry of a workgroup's chunk
__device__ __forceinline__ int entry_of(const Table &t, int64_t chunk) {
  int lo = 0, hi = t.count;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (t.e[mid].chunk0 <= chunk) lo = mid; else hi = mid;
  }
  return lo;
}

__device__ __forceinline__ void update(float &p, float g, float &m, float &v, const Consts &k,
                                       float decay) {
  m = k.b1 * m + k.c1 * g;
  v = k.b2 * v + k.c2 * (g * g);
  p = p * decay - k.lr1 * m / (sqrtf(v) * k.rk2 + k.eps);
}

}  // namespace

// Sums of squares of the gradients: a workgroup's chunks in order, in fp64.
template <typename G>
__global__ __launch_bounds__(kThreads) void adamw_norm_kernel(Table t, double *part) {
  __shared__ double red[kThreads / 64];
  double s = 0.0;
  for (int64_t chunk = blockIdx.x; chunk < t.chunks; chunk += gridDim.x) {
    const Entry &e = t.e[entry_of(t, chunk)];
    const int64_t i0 = (chunk - e.chunk0) * kChunk;
    const int64_t i1 = i0 + kChunk < e.n ? i0 + kChunk : e.n;
    float c = 0.f;
    for (int64_t i = i0 + threadIdx.x; i < i1; i += kThreads) {
      const float g = load_f32((const G *)e.g, i);
      c += g * g;
    }
    s += (double)c;
  }
  s = wave_sum_f64(s);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    double v = 0.0;
    for (int w = 0; w < kThreads / 64; ++w) v += red[w];
    part[blockIdx.x] = v;
  }
}

// The norm, and the factor of every gradient: NaN where the norm is not
// finite, which leaves the parameters and states as they are.
__global__ __launch_bounds__(kThreads) void adamw_clip_kernel(const double *part, int64_t n, Consts k,
                                                              float *clip, float *grad_norm) {
  __shared__ double red[kThreads / 64];
  double s = 0.0;
  for (int64_t i = threadIdx.x; i < n; i += kThreads) s += part[i];
  s = wave_sum_f64(s);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    double v = 0.0;
    for (int w = 0; w < kThreads / 64; ++w) v += red[w];
    const float norm = (float)(sqrt(v) * (double)fabsf(k.grad_scale));
    if (grad_norm) *grad_norm = norm;
    const float f = k.max_norm / (norm + 1e-6f);
    *clip = !(norm < INFINITY) ? NAN : k.max_norm > 0.f ? k.grad_scale * fminf(f, 1.f) : k.grad_scale;
  }
}

template <typename P, typename G>
__global__ __launch_bounds__(kThreads) void adamw_32_kernel(Table t, Consts k, const float *clip) {
  const float c = clip ? *clip : k.grad_scale;
  if (!(c == c)) return;
  const Entry &e = t.e[entry_of(t, blockIdx.x)];
  const int64_t i0 = (blockIdx.x - e.chunk0) * kChunk;
  const int64_t i1 = i0 + kChunk < e.n ? i0 + kChunk : e.n;
  for (int64_t i = i0 + threadIdx.x; i < i1; i += kThreads) {
    float p = load_f32((const P *)e.p, i), m = ((float *)e.m)[i], v = ((float *)e.v)[i];
    update(p, load_f32((const G *)e.g, i) * c, m, v, k, e.decay);
    if (sizeof(P) == 2 && k.stochastic) p = round_bf16(p, ((round_bits(e.base, i) >> 21) << 5) + 16);
    store_f32((P *)e.p, i, p);
    ((float *)e.m)[i] = m;
    ((float *)e.v)[i] = v;
    if (e.copy) e.copy[i] = f32_to_bf16_bits(p);
  }
}

// One wave per block of kBlock elements, four of them per lane.
template <typename P, typename G>
__global__ __launch_bounds__(kThreads) void adamw_8_kernel(Table t, Consts k, const float *clip) {
  const float c = clip ? *clip : k.grad_scale;
  if (!(c == c)) return;
  const Entry &e = t.e[entry_of(t, blockIdx.x)];
  const int lane = threadIdx.x & 63;
  for (int b = threadIdx.x >> 6; b < kChunk / kBlock; b += kThreads / 64) {
    const int64_t block = (blockIdx.x - e.chunk0) * (kChunk / kBlock) + b;
    const int64_t i0 = block * kBlock;
    if (i0 >= e.n) return;
    const float sm = e.ms[block], sv = e.vs[block];
    float m[4], r[4], mtop = 0.f, rtop = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t i = i0 + 64 * j + lane;
      m[j] = r[j] = 0.f;
      if (i >= e.n) continue;
      float p = load_f32((const P *)e.p, i);
      const float root = f8_to_f32(((uint8_t *)e.v)[i]) * sv;
      float v = root * root;
      m[j] = f8_to_f32(((uint8_t *)e.m)[i]) * sm;
      update(p, load_f32((const G *)e.g, i) * c, m[j], v, k, e.decay);
      r[j] = sqrtf(v);
      mtop = fmaxf(mtop, fabsf(m[j]));
      rtop = fmaxf(rtop, r[j]);
      if (sizeof(P) == 2 && k.stochastic) p = round_bf16(p, ((round_bits(e.base, i) >> 21) << 5) + 16);
      store_f32((P *)e.p, i, p);
      if (e.copy) e.copy[i] = f32_to_bf16_bits(p);
    }
    const float nsm = fmaxf(wave_max_f32(mtop) / kF8Max, kScaleMin);
    const float nsv = fmaxf(wave_max_f32(rtop) / kF8Max, kScaleMin);
    if (lane == 0) {
      e.ms[block] = nsm;
      e.vs[block] = nsv;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t i = i0 + 64 * j + lane;
      if (i >= e.n) continue;
      float qm = clamp_f8(m[j] / nsm), qr = clamp_f8(r[j] / nsv);
      if (k.stochastic) {
        const uint32_t bits = round_bits(e.base, i);
        qm = round_f8(qm, ((bits & 0x3ff) << 10) + 512);
        qr = round_f8(qr, (((bits >> 10) & 0x7ff) << 9) + 256);
      }
      ((uint8_t *)e.m)[i] = f32_to_f8(qm);
      ((uint8_t *)e.v)[i] = f32_to_f8(qr);
    }
  }
}

size_t adam_part_count(int count) { return (size_t)ceil_div(count > 0 ? count : 1, kTable) * kNormGroups; }

hipError_t launch_adamw(const rvq_adamw_tensor *t, const AdamArgs &a, hipStream_t s) {
  const Consts k = {a.b1, a.c1, a.b2, a.c2, a.eps, a.lr1, a.rk2, a.grad_scale, a.max_norm, a.stochastic};
  const bool norm = a.clip != nullptr;
  int64_t parts = 0;
  for (int pass = norm ? 0 : 1; pass < 2; ++pass) {
    for (int first = 0; first < a.count;) {
      Table tab;
      tab.count = 0;
      tab.chunks = 0;
      int i = first;
      for (; i < a.count && tab.count < kTable; ++i) {
        if (t[i].numel == 0) continue;
        Entry &e = tab.e[tab.count++];
        e.p = t[i].param;
        e.g = t[i].grad;
        e.m = t[i].m;
        e.v = t[i].v;
        e.ms = t[i].m_scale;
        e.vs = t[i].v_scale;
        e.copy = (uint16_t *)t[i].copy;
        e.n = t[i].numel;
        e.chunk0 = tab.chunks;
        e.decay = (float)(1.0 - a.lr * (double)t[i].weight_decay);
        e.base = mix(a.key + (uint32_t)i);
        tab.chunks += ceil_div(e.n, kChunk);
      }
      first = i;
      if (tab.count == 0) continue;
      if (pass == 0) {
        const unsigned groups = (unsigned)(tab.chunks < kNormGroups ? tab.chunks : kNormGroups);
        if (a.g_bf16)
          adamw_norm_kernel<uint16_t><<<groups, kThreads, 0, s>>>(tab, a.part + parts);
        else
          adamw_norm_kernel<float><<<groups, kThreads, 0, s>>>(tab, a.part + parts);
        parts += groups;
        continue;
      }
      const dim3 grid((unsigned)tab.chunks);
#define RVQ_ADAM(P, G)                                                      \
  do {                                                                      \
    if (a.eight)                                                            \
      adamw_8_kernel<P, G><<<grid, kThreads, 0, s>>>(tab, k, a.clip);       \
    else                                                                    \
      adamw_32_kernel<P, G><<<grid, kThreads, 0, s>>>(tab, k, a.clip);      \
  } while (0)
      if (a.p_bf16) {
        if (a.g_bf16) RVQ_ADAM(uint16_t, uint16_t); else RVQ_ADAM(uint16_t, float);
      } else {
        if (a.g_bf16) RVQ_ADAM(float, uint16_t); else RVQ_ADAM(float, float);
      }
#undef RVQ_ADAM
    }
    if (pass == 0) adamw_clip_kernel<<<1, kThreads, 0, s>>>(a.part, parts, k, a.clip, a.grad_norm);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

uint32_t adam_key(uint32_t seed, uint32_t step) { return mix(seed ^ (step * 0x9E3779B1u)); }

}  // namespace rvq
