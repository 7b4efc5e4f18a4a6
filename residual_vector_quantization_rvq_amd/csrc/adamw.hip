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
// rounded the same way.  Near the bottom of a block's grid m and the root go up or
// down apart; a root is never stored as 0 beside an m that is not (kF8Least).
//
// The tensors' pointers travel as kernel arguments, kTable tensors a launch:
// nothing is copied, allocated or kept between calls.
//
// Bound by memory, every element read and written once (the gradients twice
// where the norm is asked for).  Bytes moved and time: 537 M fp32 parameters,
// 32-bit states, clipped, with bf16 copies 18.3 GB, 3.44 ms, 5.3 TB/s; 537 M
// bf16 parameters with 8-bit states 5.4 GB, 0.97 to 1 ms by the card, 5.5 TB/s; 20 M fp32
// parameters with 8-bit states, clipped, with copies 361 MB, 79 us.  96 tensors
// of 200,003 elements: three launches of 5 to 6 us (42 us a call, most of it the
// caller's side).  Streaming stores change nothing (within 1%).
#include "learn.h"

namespace rvq {

namespace {

constexpr int kThreads = 256;
constexpr int kTable = 54;          // tensors of one launch, and of one launch of the norm:
constexpr int kNormTable = 160;     // as many as 4 KB of kernel arguments hold
constexpr int kChunk = 2048;        // elements of one workgroup; a multiple of kBlock
constexpr int kBlock = 256;         // elements that share a scale
constexpr int kNormGroups = 2048;   // partial sums of squares of one launch

struct Entry {
  void *p;
  const void *g;
  void *m, *v;
  float *ms, *vs;
  uint16_t *copy;
  int64_t n;
  uint32_t chunk0;  // first workgroup of this tensor
  float decay;      // 1 - lr wd
};
struct NormEntry {
  const void *g;
  int64_t n;
  uint32_t chunk0;
};
template <typename E, int Size>
struct TableOf {
  E e[Size];
  int count;
  int first;        // place in the call of the first entry; an empty tensor has an entry too
  uint32_t chunks;
};
using Table = TableOf<Entry, kTable>;
using NormTable = TableOf<NormEntry, kNormTable>;
struct Consts {
  float b1, c1, b2, c2;  // c = 1 - b, from the 64-bit b: 1.f - 0.999f is 1e-5 off
  float eps, lr1, rk2, grad_scale, max_norm;
  uint32_t key;      // of the rounding bits: mixed from seed and step
  bool stochastic;
};
// Where a step has its gradients' factor from: the partial sums themselves,
// where they are few (each workgroup adds them up, which saves a launch), the
// clip kernel's result, or (neither) grad_scale.
struct Clip {
  const double *part;
  int64_t parts;
  const float *factor;
  float *grad_norm;   // with part: written by the launch's first workgroup
};
constexpr int64_t kFewParts = 1024;
static_assert(sizeof(Table) + sizeof(Consts) + sizeof(Clip) + 16 <= 4096 && sizeof(NormTable) + 16 <= 4096,
              "kernel arguments");

// 32 bits mixed from 32: xor of the high half, odd multipliers from the
// fractions of sqrt(2) and sqrt(3)
__host__ __device__ inline uint32_t mix(uint32_t x) {
  x ^= x >> 16;
  x *= 0x3504F333u;
  x ^= x >> 15;
  x *= 0x5DB3D743u;
  return x ^ (x >> 16);
}
__device__ __forceinline__ uint32_t tensor_bits(uint32_t key, int tensor) {
  return mix(key + (uint32_t)tensor);
}
// element i's bits are mix(word), word + kWordStep the next element's
constexpr uint32_t kWordStep = 0x9E3779B1u;
__device__ __forceinline__ uint32_t round_word(uint32_t base, int64_t i) {
  return base + (uint32_t)i * kWordStep + (uint32_t)(i >> 32) * 0x3504F333u;
}

// |v| <= 448 (or a few units of the last place above it: both roundings bring
// that to 448) rounded to the e4m3 grid at random, into byte `Byte` of `w`.  The
// instruction adds the upper 20 of the random bits under the three bits of
// the mantissa that stay; below 2^-6 the grid is that of 2^-6, and the bits
// stand for the same share of its step.
template <int Byte>
__device__ __forceinline__ int random_f8(float v, uint32_t random, int w) {
  return __builtin_amdgcn_cvt_sr_fp8_f32(v, (int)random, w, Byte);
}
// v[q0 .. q0 + 3] with the bits of each
template <int N, typename Bits>
__device__ __forceinline__ uint32_t random_f8x4(const float (&v)[N], int q0, Bits bits) {
  int w = random_f8<0>(v[q0], bits(q0), 0);
  w = random_f8<1>(v[q0 + 1], bits(q0 + 1), w);
  w = random_f8<2>(v[q0 + 2], bits(q0 + 2), w);
  return (uint32_t)random_f8<3>(v[q0 + 3], bits(q0 + 3), w);
}
// v rounded to bf16 at random: of a NaN, only one with zeros in the places that go,
// out of whose significand the bits cannot carry
__device__ __forceinline__ float round_number_bf16(float v, uint32_t random16) {
  return __uint_as_float((__float_as_uint(v) + random16) & 0xffff0000u);
}
// ... of any NaN
__device__ __forceinline__ float round_bf16(float v, uint32_t random16) {
  return v == v ? round_number_bf16(v, random16) : v;
}

// The least e4m3 value.  A root above 0 is stored as it and not as 0 where its m
// is not stored as 0.  The two are rounded apart, and m / 0 would make the next
// step lr m / eps: over 10^6 times lr in blocks with elements 10^4 times larger.
// A state that comes with such a pair is stepped as it is, by the formula alone.
constexpr float kF8Least = 0x1p-9f;
// e4m3 byte q of 8 is not 0, of either sign
__device__ __forceinline__ bool byte_set(u32x2 w, int q) { return (w[q >> 2] >> (8 * (q & 3))) & 0x7f; }

// op over the 32 lanes of a half wave
template <typename Op>
__device__ __forceinline__ int over_half_wave(int v, Op op) {
#define RVQ_ROR(N) v = op(v, __builtin_amdgcn_mov_dpp(v, 0x120 + N, 0xf, 0xf, false))
  RVQ_ROR(8);
  RVQ_ROR(4);
  RVQ_ROR(2);
  RVQ_ROR(1);
#undef RVQ_ROR
  return op(v, __builtin_amdgcn_ds_swizzle(v, 0x401f));  // lane ^ 16
}
__device__ __forceinline__ float half_wave_max(float v) {
  return __int_as_float(over_half_wave(
      __float_as_int(v), [](int a, int b) { return __float_as_int(fmaxf(__int_as_float(a), __int_as_float(b))); }));
}
__device__ __forceinline__ uint32_t half_wave_max(uint32_t v) {
  return (uint32_t)over_half_wave((int)v, [](int a, int b) { return (int)max((uint32_t)a, (uint32_t)b); });
}

// 8 e4m3 bytes at p; `left` of them exist (the others read as zero)
__device__ __forceinline__ u32x2 load_8_bytes(const uint8_t *p, int left) {
  u32x2 q = {0, 0};
  if (left >= 8) {
    q = *(const u32x2_at1 *)p;
  } else {
    for (int e = 0; e < left; ++e) q[e >> 2] |= (uint32_t)p[e] << (8 * (e & 3));
  }
  return q;
}
__device__ __forceinline__ void load_f8x8(const uint8_t *p, int left, float (&v)[8]) {
  const u32x2 q = load_8_bytes(p, left);
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)q[j], false);
    const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)q[j], true);
    v[4 * j] = lo[0];
    v[4 * j + 1] = lo[1];
    v[4 * j + 2] = hi[0];
    v[4 * j + 3] = hi[1];
  }
}
__device__ __forceinline__ void store_8_bytes(uint8_t *p, int left, u32x2 q) {
  if (left >= 8) {
    *(u32x2_at1 *)p = q;
  } else {
    for (int e = 0; e < left; ++e) p[e] = (uint8_t)(q[e >> 2] >> (8 * (e & 3)));
  }
}

// the entry of a workgroup's chunk
template <typename TableT>
__device__ __forceinline__ int entry_of(const TableT &t, uint32_t chunk) {
  int lo = 0, hi = t.count;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (t.e[mid].chunk0 <= chunk) lo = mid; else hi = mid;
  }
  return lo;
}

// m and v with every operation rounded by itself, in the order of the formula
// above: a stored 8-bit moment turns on the last place of what is rounded.
__device__ __forceinline__ void moments(float g, float &m, float &v, const Consts &k) {
#pragma clang fp contract(off)
  m = k.b1 * m + k.c1 * g;
  v = k.b2 * v + k.c2 * (g * g);
}

// Root and quotient are the hardware's (one unit in the last place): they act
// on lr times the update alone.
__device__ __forceinline__ float updated(float p, float m, float root, const Consts &k, float decay) {
  return p * decay - k.lr1 * m * __builtin_amdgcn_rcpf(root * k.rk2 + k.eps);
}

// The nearest fp32 to sqrt(v), by one Newton step from the hardware's 1 /
// sqrt(v), for v of 2^-96 (whose remainder fp32 still holds) and up; smaller
// ones count as zero, and infinity and NaN give NaN.
__device__ __forceinline__ float nearest_sqrt(float v) {
  const float y = __builtin_amdgcn_rsqf(v), s = v * y;
  const float r = __builtin_fmaf(-s, s, v);
  return v < 0x1p-96f ? 0.f : __builtin_fmaf(r, 0.5f * y, s);
}
// A factor for roots of an element whose old root and gradient are `largest` at
// most.  Large squares lie between 2^16 and 2^124 then, so that (1 - b2) times
// them, 2^-53 at least, is no v that counts as zero; small ones are 2^64 times what
// they are.  A power of two changes no digit.
constexpr float kRootUnit = 0x1p32f, kLargeUnit = 0x1p-66f;
__device__ __forceinline__ float root_unit(float largest) {
  return largest < 0x1p29f ? kRootUnit : largest < 0x1p74f ? 0x1p-12f : kLargeUnit;
}

// An element's step where squares leave fp32, in the unit u: vu is the old and
// then the new v times u^2, root the new root times u.  Returns the new parameter.
__device__ __forceinline__ float large_step(float p, float g, float m, float &vu, float &root, float u,
                                            const Consts &k, float decay) {
  Consts ku = k;
  ku.eps *= u;
  m *= u;
  moments(g * u, m, vu, ku);
  root = vu < INFINITY ? nearest_sqrt(vu) : vu;
  return updated(p, m, root, ku, decay);
}
constexpr float kLargest = 0x1.fffffep127f;

}  // namespace

// Sums of squares of the gradients, in fp64: in fp32 an element above 1.8e19 would
// make a finite norm infinite and the step be skipped, and those below 1e-23
// would be lost.  A workgroup takes consecutive chunks.
template <typename G>
__global__ __launch_bounds__(kThreads) void adamw_norm_kernel(NormTable t, double *part) {
  __shared__ double red[kThreads / 64];
  double s = 0.0;
  const int64_t c0 = (int64_t)t.chunks * blockIdx.x / gridDim.x;
  const int64_t c1 = (int64_t)t.chunks * (blockIdx.x + 1) / gridDim.x;
  int at = entry_of(t, (uint32_t)c0);
  for (int64_t chunk = c0; chunk < c1; ++chunk) {
    while (at + 1 < t.count && t.e[at + 1].chunk0 <= chunk) ++at;
    const NormEntry &e = t.e[at];
    const int64_t i = (chunk - e.chunk0) * kChunk + threadIdx.x * 8;
    if (i < e.n) {
      float g[8];
      load_n<8>((const G *)e.g + i, (int)(e.n - i < 8 ? e.n - i : 8), g);
#pragma unroll
      for (int j = 0; j < 8; ++j) s = __builtin_fma((double)g[j], (double)g[j], s);
    }
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

namespace {

// The norm of all gradients out of the workgroups' sums, added by a workgroup
// of T threads in an order that depends on their number alone.
template <int T>
__device__ __forceinline__ float norm_of(const double *part, int64_t n, float grad_scale) {
  __shared__ double red[T / 64];
  double s = 0.0;
  for (int64_t i = threadIdx.x; i < n; i += T) s += part[i];
  s = wave_sum_f64(s);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = s;
  __syncthreads();
  double v = 0.0;
#pragma unroll
  for (int w = 0; w < T / 64; ++w) v += red[w];
  return (float)(sqrt(v) * (double)fabsf(grad_scale));
}
// The factor of every gradient: NaN where the norm is not finite, which leaves
// the parameters and states as they are.
__device__ __forceinline__ float factor_of(float norm, const Consts &k) {
  const float f = k.max_norm / (norm + 1e-6f);
  return !(norm < INFINITY) ? NAN : k.max_norm > 0.f ? k.grad_scale * fminf(f, 1.f) : k.grad_scale;
}
// for every thread of a workgroup of the step
__device__ __forceinline__ float step_factor(const Clip &c, const Consts &k) {
  if (!c.part) return c.factor ? *c.factor : k.grad_scale;
  const float norm = norm_of<kThreads>(c.part, c.parts, k.grad_scale);
  if (c.grad_norm && blockIdx.x == 0 && threadIdx.x == 0) *c.grad_norm = norm;
  return factor_of(norm, k);
}

}  // namespace

__global__ __launch_bounds__(1024) void adamw_clip_kernel(const double *part, int64_t n, Consts k,
                                                          float *factor, float *grad_norm) {
  const float norm = norm_of<1024>(part, n, k.grad_scale);
  if (threadIdx.x == 0) {
    if (grad_norm) *grad_norm = norm;
    *factor = factor_of(norm, k);
  }
}

// 32-bit states: two pieces of four elements a lane, all of whose loads are
// issued before the first is used.
template <typename P, typename G>
__global__ __launch_bounds__(kThreads) void adamw_32_kernel(Table t, Consts k, Clip clip) {
  constexpr int N = 4, J = kChunk / (kThreads * N);
  const int at = entry_of(t, blockIdx.x);
  const Entry &e = t.e[at];
  const int64_t i0 = (int64_t)(blockIdx.x - e.chunk0) * kChunk + threadIdx.x * N;
  float p[J][N], g[J][N], m[J][N], v[J][N];
  int left[J];
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const int64_t i = i0 + j * kThreads * N;
    left[j] = (int)(e.n - i < 0 ? 0 : e.n - i < N ? e.n - i : N);
    load_n<N>((const P *)e.p + i, left[j], p[j]);
    load_n<N>((const G *)e.g + i, left[j], g[j]);
    load_n<N>((const float *)e.m + i, left[j], m[j]);
    load_n<N>((const float *)e.v + i, left[j], v[j]);
  }
  const float c = step_factor(clip, k);
  if (!(c == c)) return;
  const uint32_t base = tensor_bits(k.key, t.first + at);
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const int64_t i = i0 + j * kThreads * N;
    const uint32_t word = round_word(base, i);  // a piece does not reach over a multiple of 2^32
    float top = 0.f;
#pragma unroll
    for (int q = 0; q < N; ++q) {
      moments(g[j][q] * c, m[j][q], v[j][q], k);
      p[j][q] = updated(p[j][q], m[j][q], __builtin_amdgcn_sqrtf(v[j][q]), k, e.decay);
      top = fmaxf(top, v[j][q]);
    }
    if (top == INFINITY) {
      // Squares beyond fp32: once more, in a smaller unit; a finite v is held at
      // the largest fp32 at most.
#pragma unroll
      for (int q = 0; q < N; ++q) {
        if (v[j][q] != INFINITY) continue;
        float vu = ((const float *)e.v)[i + q] * kLargeUnit * kLargeUnit, root;
        p[j][q] = large_step(load_f32((const P *)e.p, i + q), g[j][q] * c, ((const float *)e.m)[i + q], vu, root,
                             kLargeUnit, k, e.decay);
        v[j][q] = vu * (1.f / kLargeUnit) * (1.f / kLargeUnit);
        if (v[j][q] == INFINITY && vu < INFINITY) v[j][q] = kLargest;
      }
    }
    if (sizeof(P) == 2 && k.stochastic) {
#pragma unroll
      for (int q = 0; q < N; ++q)
        p[j][q] = round_bf16(p[j][q], ((mix(word + q * kWordStep) >> 21) << 5) + 16);
    }
    store_n<N>((P *)e.p + i, left[j], p[j]);
    store_n<N>((float *)e.m + i, left[j], m[j]);
    store_n<N>((float *)e.v + i, left[j], v[j]);
    if (e.copy) store_n<N>(e.copy + i, left[j], p[j]);
  }
}

// 8-bit states: a half wave per block of kBlock elements, eight a lane.  The
// root and the quotients that are stored are the nearest fp32 values, so that
// the state is the definition's to the bit: one that is a unit off is stored as
// the neighbour on the grid about once in 10^6 values, 6 to 12% away.  Where
// parameters are bf16, arithmetic is nearly as long as 10 bytes of traffic: what
// is for rare elements alone is left to branches that a block without them does
// not take (537 M, on one card: 981 us with none of it, 996 as it is; small roots
// looked for and NaN kept element by element, and the bits of low roots chosen so,
// cost 2% each).
template <typename P, typename G>
__global__ __launch_bounds__(kThreads) void adamw_8_kernel(Table t, Consts k, Clip clip) {
  constexpr int N = kChunk / kThreads;
  static_assert(N == 8 && kBlock == 32 * N, "a half wave holds a block");
  const int at = entry_of(t, blockIdx.x);
  const Entry &e = t.e[at];
  const int64_t i = (int64_t)(blockIdx.x - e.chunk0) * kChunk + threadIdx.x * N, block = i / kBlock;
  float c = 0.f;
  if (clip.part) c = step_factor(clip, k);  // a barrier: before any lane leaves
  if (block * kBlock >= e.n) return;        // the whole half wave
  const int left = (int)(e.n - i < 0 ? 0 : e.n - i < N ? e.n - i : N);
  float p[N], g[N], m[N], v[N];
  load_n<N>((const P *)e.p + i, left, p);
  load_n<N>((const G *)e.g + i, left, g);
  load_f8x8((const uint8_t *)e.m + i, left, m);
  load_f8x8((const uint8_t *)e.v + i, left, v);
  const float sm = e.ms[block], sv = e.vs[block];
  if (!clip.part) c = step_factor(clip, k);
  if (!(c == c)) return;
  const uint32_t base = tensor_bits(k.key, t.first + at);
  float mtop = 0.f;
  uint32_t rtop = 0;
  const uint32_t word = round_word(base, i);
  uint32_t bits[N];
  // Roots times kRootUnit, and v times its square: nothing in fp32's range is
  // too small then, and where v times that overflows the root is NaN.
  Consts ku = k;
  ku.c2 *= kRootUnit * kRootUnit;
  ku.rk2 *= 1.f / kRootUnit;
  const float svu = sv * kRootUnit;
#pragma unroll
  for (int q = 0; q < N; ++q) {
    m[q] *= sm;
    v[q] *= svu;
    v[q] *= v[q];
    moments(g[q] * c, m[q], v[q], ku);
    v[q] = nearest_sqrt(v[q]);  // the root from here on
    p[q] = updated(p[q], m[q], v[q], ku, e.decay);
    mtop = fmaxf(mtop, fabsf(m[q]));
    rtop = max(rtop, __float_as_uint(v[q]));  // of either sign, NaN is above the rest
    if (k.stochastic) {
      bits[q] = mix(word + q * kWordStep);
      // a NaN of the gradient or a scale is seen to below, those of e4m3 and bf16 have zeros
      if (sizeof(P) == 2) p[q] = round_number_bf16(p[q], ((bits[q] >> 21) << 5) + 16);
    }
  }
  float nsm = half_wave_max(mtop), nsv = __uint_as_float(half_wave_max(rtop)), unit = kRootUnit;
  if (!(nsv < INFINITY && sm == sm)) {
    // v times kRootUnit^2 beyond fp32, infinity or NaN in the block: its elements
    // once more, each in a unit of its own.  What is not finite is stored as NaN,
    // and its block's scales are the others'.
    unit = 1.f;
#pragma unroll 1
    for (int at = 0; at < N; ++at) {  // not unrolled: hardly ever run, and it would take the registers of two waves
      const float gq = at < left ? load_f32((const G *)e.g, i + at) * c : 0.f;
      const float m0 = at < left ? f8_to_f32(((const uint8_t *)e.m)[i + at]) * sm : 0.f;
      const float r0 = at < left ? f8_to_f32(((const uint8_t *)e.v)[i + at]) * sv : 0.f;
      const float u = root_unit(fmaxf(r0, fabsf(gq)));
      float vu = (r0 * u) * (r0 * u), root;
      float pq = large_step(at < left ? load_f32((const P *)e.p, i + at) : 0.f, gq, m0, vu, root, u, k, e.decay);
      if (sizeof(P) == 2 && k.stochastic) pq = round_bf16(pq, ((mix(word + at * kWordStep) >> 21) << 5) + 16);
      root = fminf(root * (1.f / u), kLargest) + (root - root);  // above it by rounding alone
#pragma unroll
      for (int q = 0; q < N; ++q) {
        p[q] = q == at ? pq : p[q];
        v[q] = q == at ? root : v[q];
      }
    }
    mtop = 0.f;
    float top = 0.f;
#pragma unroll
    for (int q = 0; q < N; ++q) {
      if (!(fabsf(m[q]) < INFINITY)) m[q] = NAN;
      mtop = fmaxf(mtop, fabsf(m[q]));
      top = fmaxf(top, v[q]);
    }
    nsm = half_wave_max(mtop);
    nsv = half_wave_max(top);
  }
  store_n<N>((P *)e.p + i, left, p);
  if (e.copy) store_n<N>(e.copy + i, left, p);
  nsm = fmaxf(nsm * kF8Unit, kScaleMin);
  nsv = fmaxf(nsv * kF8Unit, kScaleMin * unit);
  const float im = 1.f / nsm, iv = 1.f / nsv;
#pragma unroll
  for (int q = 0; q < N; ++q) {
    m[q] = nearest_quotient(m[q], nsm, im);
    v[q] = nearest_quotient(v[q], nsv, iv);
  }
  u32x2 qm, qv;
  const auto m_bits = [&](int q) { return (bits[q] << 22) | 0x200000u; };
  const auto v_bits = [&](int q) { return ((bits[q] << 11) & 0xffe00000u) | 0x100000u; };
  if (k.stochastic) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      qm[h] = random_f8x4(m, 4 * h, m_bits);
      qv[h] = random_f8x4(v, 4 * h, v_bits);
    }
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      qm[h] = pack_f8x4(m[4 * h], m[4 * h + 1], m[4 * h + 2], m[4 * h + 3]);
      qv[h] = pack_f8x4(v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]);
    }
  }
  // roots above 0 and below the least value: those alone can have become 0.  Zeros,
  // of rows that nothing touched, are told apart at a second look.
  uint32_t low = UINT32_MAX;  // the least root above 0, less 1 in its bits
#pragma unroll
  for (int q = 0; q < N; ++q) low = min(low, __float_as_uint(v[q]) - 1);
  if (low < __float_as_uint(kF8Least) - 1) {  // only a root below kF8Least can have become 0
    const u32x2 m0 = load_8_bytes((const uint8_t *)e.m + i, left), v0 = load_8_bytes((const uint8_t *)e.v + i, left);
    const auto paired = [&](int q) { return v[q] < kF8Least && (byte_set(v0, q) || !byte_set(m0, q)); };
    if (k.stochastic) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
        qv[h] = random_f8x4(v, 4 * h, [&](int q) { return paired(q) ? m_bits(q) : v_bits(q); });
    }
#pragma unroll
    for (int q = 0; q < N; ++q)
      if (paired(q) && v[q] > 0.f && byte_set(qm, q) && !byte_set(qv, q)) qv[q >> 2] |= 1u << (8 * (q & 3));
  }
  store_8_bytes((uint8_t *)e.m + i, left, qm);
  store_8_bytes((uint8_t *)e.v + i, left, qv);
  if ((threadIdx.x & 31) == 0) {
    e.ms[block] = nsm;
    e.vs[block] = nsv * (1.f / unit);
  }
}

// every launch of the norm but the last takes kNormTable tensors
size_t adam_part_count(int count) { return (size_t)(count > 0 ? ceil_div(count, kNormTable) : 1) * kNormGroups; }

namespace {

// Consecutive tables of all tensors, one launch(table) each, of at most `most`
// chunks.  A step has a workgroup for each: kMaxChunks, as many as one tensor has
// (2^34 elements).  The norm's workgroups take many each.
constexpr int64_t kMaxChunks = (int64_t)1 << 23;
static_assert(kNormTable * kMaxChunks < (int64_t)1 << 32, "chunk0 is 32-bit");
template <typename TableT, typename Fill, typename Launch>
void for_each_table(const rvq_adamw_tensor *t, int count, int size, int64_t most, Fill fill, Launch launch) {
  for (int first = 0; first < count;) {
    TableT tab;
    tab.first = first;
    int64_t chunks = 0;
    int i = 0;
    for (; i < size && first + i < count; ++i) {
      const int64_t n = t[first + i].numel, more = ceil_div(n, kChunk);
      if (i > 0 && chunks + more > most) break;
      fill(tab.e[i], t[first + i]);
      tab.e[i].n = n;
      tab.e[i].chunk0 = (uint32_t)chunks;
      chunks += more;
    }
    tab.count = i;
    tab.chunks = (uint32_t)chunks;
    first += i;
    if (chunks > 0) launch(tab);
  }
}

template <typename P, typename G>
void launch_step(const rvq_adamw_tensor *t, const AdamArgs &a, const Consts &k, Clip clip,
                 hipStream_t s) {
  for_each_table<Table>(
      t, a.count, kTable, kMaxChunks,
      [&](Entry &e, const rvq_adamw_tensor &x) {
        e.p = x.param;
        e.g = x.grad;
        e.m = x.m;
        e.v = x.v;
        e.ms = x.m_scale;
        e.vs = x.v_scale;
        e.copy = (uint16_t *)x.copy;
        e.decay = (float)(1.0 - a.lr * (double)x.weight_decay);
      },
      [&](const Table &tab) {
        if (a.eight)
          adamw_8_kernel<P, G><<<dim3(tab.chunks), kThreads, 0, s>>>(tab, k, clip);
        else
          adamw_32_kernel<P, G><<<dim3(tab.chunks), kThreads, 0, s>>>(tab, k, clip);
        clip.grad_norm = nullptr;  // written by the first launch
      });
}

template <typename G>
int64_t launch_norm(const rvq_adamw_tensor *t, const AdamArgs &a, hipStream_t s) {
  int64_t parts = 0;
  for_each_table<NormTable>(
      t, a.count, kNormTable, kNormTable * kMaxChunks, [&](NormEntry &e, const rvq_adamw_tensor &x) { e.g = x.grad; },
      [&](const NormTable &tab) {
        const unsigned groups = tab.chunks < (unsigned)kNormGroups ? tab.chunks : kNormGroups;
        adamw_norm_kernel<G><<<dim3(groups), kThreads, 0, s>>>(tab, a.part + parts);
        parts += groups;
      });
  return parts;
}

}  // namespace

hipError_t launch_adamw(const rvq_adamw_tensor *t, const AdamArgs &a, hipStream_t s) {
  const Consts k = {a.b1, a.c1, a.b2, a.c2, a.eps, a.lr1, a.rk2, a.grad_scale, a.max_norm, a.key,
                    a.stochastic};
  Clip clip = {nullptr, 0, nullptr, nullptr};
  if (a.clip) {
    const int64_t parts = a.g_bf16 ? launch_norm<uint16_t>(t, a, s) : launch_norm<float>(t, a, s);
    if (parts > 0 && parts <= kFewParts) {
      clip = {a.part, parts, nullptr, a.grad_norm};
    } else {
      adamw_clip_kernel<<<1, 1024, 0, s>>>(a.part, parts, k, a.clip, a.grad_norm);
      clip.factor = a.clip;
    }
  }
  if (a.p_bf16) {
    if (a.g_bf16) launch_step<uint16_t, uint16_t>(t, a, k, clip, s);
    else launch_step<uint16_t, float>(t, a, k, clip, s);
  } else {
    if (a.g_bf16) launch_step<float, uint16_t>(t, a, k, clip, s);
    else launch_step<float, float>(t, a, k, clip, s);
  }
  return hipGetLastError();
}

uint32_t adam_key(uint32_t seed, uint32_t step) { return mix(seed ^ (step * 0x9E3779B1u)); }

}  // namespace rvq
