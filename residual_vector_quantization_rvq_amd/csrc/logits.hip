// logits.hip -- rows of logits x over V tokens at temperature T: log probabilities
// of given tokens, entropies and top alternatives, the distillation loss of a
// teacher's top logits, and the gradients of both.
//
//   M = max x,  d_j = (M - x_j) / T >= 0,  S = sum exp(-d_j)
//   log p_j = -d_j - log S,   H = log S + sum d_j exp(-d_j) / S
//
// H is a sum of two terms that are not negative, and log S is log1p of the sum
// without one of its largest terms, so that a row that is all but certain keeps the
// precision of its small numbers.  Sums are fp32: a thread adds its elements in
// four chains, lanes and waves join them in a tree; exponentials are the
// hardware's of base 2 (the factor log2(e) / T is one multiplication).
//
// Bound by memory, and for bf16 nearly by the arithmetic too (about eleven
// instructions an element, four of them the exponential): each row is read once,
// with a running maximum and sum.  What a row needs after that (top alternatives, the
// sum of an all but certain row) is read again by the few threads whose largest
// value says that they hold it.  4577 x 65,536 bf16 110 us (5.5 TB/s), with five alternatives
// 119, fp32 201 (6.0); 36,621 x 8192 bf16 108 (5.6) and its gradient 200 (6.0); 1,171,875 x
// 256 174 (3.5), where what is done once a row takes longer than its bytes.
#include "head.h"
#include "lanes.h"

namespace rvq {

namespace {

constexpr int kMaxGroups = 1 << 20;  // workgroups of a launch; rows beyond are looped over
constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;
constexpr float kFar = 300.f;        // powers of two: beyond it nothing is left of an fp32 number
constexpr int kPieces = 4;           // 16-byte pieces that a thread loads at once

__device__ __forceinline__ float exp2_neg(float d) { return __builtin_amdgcn_exp2f(-d); }

// A row (or a part of one) as it is summed: the largest value m, t = sum exp2((x - m) c)
// and q = sum (m - x) c exp2((x - m) c).  Nothing yet (or -inf alone): m = -inf, t = 0.
struct Sums {
  float m, t, q;
};

template <typename T>
__device__ __forceinline__ void load_values(const T *row, int at, int left, float (&v)[kPiece<T>]) {
  unpack(load_piece(row + (left > 0 ? at : 0), left), v);
#pragma unroll
  for (int e = 0; e < kPiece<T>; ++e)
    if (e >= left) v[e] = -INFINITY;
}

template <int N, bool ENT>
__device__ __forceinline__ void add_values(const float (&v)[N], float c, Sums &s) {
  float mc = v[0];
#pragma unroll
  for (int e = 1; e < N; ++e) mc = fmaxf(mc, v[e]);
  if (mc > s.m) {
    if (s.m > -INFINITY) {
      const float d = fminf((mc - s.m) * c, kFar), f = exp2_neg(d);
      if (ENT) s.q = (s.q + d * s.t) * f;
      s.t *= f;
    }
    s.m = mc;
  }
  const float m = s.m == -INFINITY ? 0.f : s.m;
  float t[4] = {0.f, 0.f, 0.f, 0.f}, q[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int e = 0; e < N; ++e) {
    const float d = (m - v[e]) * c, x = exp2_neg(d);
    t[e & 3] += x;
    if (ENT) q[e & 3] += fminf(d, kFar) * x;  // a masked value: 0
  }
  s.t += (t[0] + t[1]) + (t[2] + t[3]);
  if (ENT) s.q += (q[0] + q[1]) + (q[2] + q[3]);
}

// P pieces of a row, W pieces apart, the first at column `at`.  With BITS, columns whose
// bit is set in `bits` are left out.  At a row's end (TAIL) the last N columns are read
// in place of a piece that goes past them, and what an earlier piece holds is left
// out: no load waits for a branch.  (Rows of N columns or more; `bits` has a byte more.)
template <typename T, int W, int P, bool ENT, bool BITS, bool TAIL>
__device__ __forceinline__ void stream_pieces(const T *row, int cols, int at, float c, const uint8_t *bits, Sums &s) {
  constexpr int N = kPiece<T>;
  u32x4 raw[P];
  int from[P];
#pragma unroll
  for (int p = 0; p < P; ++p) {
    from[p] = at + p * W * N;
    if (TAIL) from[p] = min(from[p], cols - N);
    raw[p] = load16(row + from[p]);
  }
  float v[P * N];
#pragma unroll
  for (int p = 0; p < P; ++p) {
    float u[N];
    unpack(raw[p], u);
    uint32_t out = 0;  // a bit for each column that is left out
    if constexpr (BITS) {
      out = bits[from[p] >> 3];
      if (TAIL) out |= (uint32_t)bits[(from[p] >> 3) + 1] << 8;
      if (TAIL || N == 4) out >>= from[p] & 7;
    }
    if (TAIL) out |= (1u << min(at + p * W * N - from[p], N)) - 1;
    if (TAIL || BITS) {
#pragma unroll
      for (int e = 0; e < N; ++e)
        if (out >> e & 1) u[e] = -INFINITY;
    }
#pragma unroll
    for (int e = 0; e < N; ++e) v[p * N + e] = u[e];
  }
  add_values<P * N, ENT>(v, c, s);
}

// The values of columns [0, cols) of a row that are this thread's: pieces lane,
// lane + W, ...  ONE_SUM: inner pieces and a row's end are summed by the same instructions;
// beside the search for the top alternatives that is faster (16,384 x 65,536 bf16 400 us, 450
// with a sum for each), without it slower (16,384 x 2,049 bf16 35 us, 17 with a sum for each).
template <typename T, int W, bool ENT, bool BITS, bool ONE_SUM>
__device__ __forceinline__ void stream_row(const T *row, int cols, int lane, float c, const uint8_t *bits, Sums &s) {
  constexpr int N = kPiece<T>, P = kPieces;
  if (cols < N) {
    float v[N];
    load_values(row, lane * N, cols - lane * N, v);
    if constexpr (BITS) {
#pragma unroll
      for (int e = 0; e < N; ++e)
        if (bits[0] >> e & 1) v[e] = -INFINITY;
    }
    add_values<N, ENT>(v, c, s);
    return;
  }
  if constexpr (ONE_SUM) {
    for (int base = 0; base < cols; base += W * P * N) {
      float v[P * N];
      const int at = base + lane * N;
      if (base + W * P * N <= cols) {
        u32x4 raw[P];
#pragma unroll
        for (int p = 0; p < P; ++p) raw[p] = load16(row + at + p * W * N);
#pragma unroll
        for (int p = 0; p < P; ++p) {
          float u[N];
          unpack(raw[p], u);
#pragma unroll
          for (int e = 0; e < N; ++e) v[p * N + e] = u[e];
        }
      } else {
#pragma unroll
        for (int p = 0; p < P; ++p) {
          float u[N];
          load_values(row, at + p * W * N, cols - (at + p * W * N), u);
#pragma unroll
          for (int e = 0; e < N; ++e) v[p * N + e] = u[e];
        }
      }
      add_values<P * N, ENT>(v, c, s);
    }
    return;
  }
  int base = 0;
  for (; base + W * P * N <= cols; base += W * P * N)
    stream_pieces<T, W, P, ENT, BITS, false>(row, cols, base + lane * N, c, bits, s);
  if (cols - base > 2 * W * N) {
    stream_pieces<T, W, P, ENT, BITS, true>(row, cols, base + lane * N, c, bits, s);
  } else if (cols - base > W * N) {
    stream_pieces<T, W, 2, ENT, BITS, true>(row, cols, base + lane * N, c, bits, s);
  } else if (base < cols) {
    stream_pieces<T, W, 1, ENT, BITS, true>(row, cols, base + lane * N, c, bits, s);
  }
}

// ---- over the W threads of a row; W > 64: the whole workgroup ----
template <int W>
__device__ __forceinline__ float all_max(float v, float *red) {
  v = lane_max<W < 64 ? W : 64>(v);
  if constexpr (W > 64) {
    __syncthreads();
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    v = red[0];
#pragma unroll
    for (int w = 1; w < W / 64; ++w) v = fmaxf(v, red[w]);
  }
  return v;
}
template <int W, typename F>
__device__ __forceinline__ F all_sum(F v, F *red) {
  if constexpr (sizeof(F) == 4) {
    v = lane_sum<W < 64 ? W : 64>(v);
  } else {
#pragma unroll
    for (int off = (W < 64 ? W : 64) / 2; off >= 1; off >>= 1) v += __shfl_xor(v, off, 64);
  }
  if constexpr (W > 64) {
    __syncthreads();
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    v = red[0];
#pragma unroll
    for (int w = 1; w < W / 64; ++w) v += red[w];
  }
  return v;
}
// two at once; `red` holds 2 W / 64
template <int W>
__device__ __forceinline__ void all_sum2(float &a, float &b, float *red) {
  a = lane_sum<W < 64 ? W : 64>(a);
  b = lane_sum<W < 64 ? W : 64>(b);
  if constexpr (W > 64) {
    __syncthreads();
    if ((threadIdx.x & 63) == 0) {
      red[2 * (threadIdx.x >> 6)] = a;
      red[2 * (threadIdx.x >> 6) + 1] = b;
    }
    __syncthreads();
    a = red[0];
    b = red[1];
#pragma unroll
    for (int w = 1; w < W / 64; ++w) {
      a += red[2 * w];
      b += red[2 * w + 1];
    }
  }
}
// the smallest
template <int W>
__device__ __forceinline__ int all_min(int v, int *red) {
#pragma unroll
  for (int off = (W < 64 ? W : 64) / 2; off >= 1; off >>= 1) v = min(v, __shfl_xor(v, off, 64));
  if constexpr (W > 64) {
    __syncthreads();
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    v = red[0];
#pragma unroll
    for (int w = 1; w < W / 64; ++w) v = min(v, red[w]);
  }
  return v;
}

// The threads' sums as one: m, t and q of all (a thread's own stay as they are).
template <int W, bool ENT>
__device__ __forceinline__ Sums join_threads(const Sums &s, float c, float *red) {
  Sums r;
  r.m = all_max<W>(s.m, red);
  float t = s.t, q = s.q;
  if (!(t == 0.f)) {  // NaN goes on
    const float d = fminf((r.m - s.m) * c, kFar), f = exp2_neg(d);
    if (ENT) q = (q + d * t) * f;
    t *= f;
    if (r.m != r.m || r.m - s.m != r.m - s.m) t = NAN;  // infinite maxima
  }
  if (ENT) {
    all_sum2<W>(t, q, red);
  } else {
    t = all_sum<W>(t, red);
    q = 0.f;
  }
  r.t = t;
  r.q = q;
  return r;
}

// The sum without one of its largest terms.  Where the rest is small beside that
// term, it is added up anew without it: the thread that holds the term (the first of
// them) gives its values to all.
template <typename T, int W>
__device__ __forceinline__ float rest_of(const T *row, int cols, int lane, float c, const Sums &own, const Sums &all,
                                         float *red) {
  if (!(all.t < 1.5f) || all.t == 0.f) return all.t - 1.f;
  constexpr int N = kPiece<T>;
  const int owner = all_min<W>(own.m == all.m ? lane : W, (int *)red);
  float rest = 0.f;
  if (lane != owner && own.t != 0.f) rest = own.t * exp2_neg(fminf((all.m - own.m) * c, kFar));
  for (int64_t i = ((int64_t)lane * W + owner) * N; i < cols; i += (int64_t)W * W * N) {
    float v[N];
    load_values(row, (int)i, cols - (int)i, v);
#pragma unroll
    for (int e = 0; e < N; ++e)
      if (v[e] != all.m) rest += exp2_neg((all.m - v[e]) * c);
  }
  return all_sum<W>(rest, red);
}

// ---- values and places as one number: larger values first, then lower places ----
// -0 and +0 are one value.
__device__ __forceinline__ uint32_t order_bits(float v) {
  const uint32_t b = __float_as_uint(v + 0.f);
  return b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float from_order_bits(uint32_t k) {
  return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xffffffffu));
}
__device__ __forceinline__ uint64_t order_key(float v, int at) {
  return ((uint64_t)order_bits(v) << 32) | (uint32_t)~at;
}
constexpr uint32_t kNoneBits = 0x007fffffu;  // order_bits(-inf): masked values are no alternatives
constexpr int kMaxCand = 1024, kTopThreads = 256;
static_assert(kMaxTop <= kMaxCand, "the join ranks at least one slice's keys");

// A bound that at least `top` of the `total` numbers in v reach (0 if there are fewer):
// the upper 16 bits of the top-th largest (or the lower, with first = 15 and the upper as
// bound).  By one wave, a bit at a time.
template <int PER>
__device__ __forceinline__ uint32_t bound_of(const uint32_t (&v)[PER], int top, uint32_t bound = 0, int first = 31) {
  for (int bit = first; bit > first - 16; --bit) {
    const uint32_t trial = bound | (1u << bit);
    int reached = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) reached += __popcll(__ballot(v[i] >= trial));
    if (reached >= top) bound = trial;
  }
  return bound;
}
// Ranks `found` different keys: the largest `top` of them to out in order, zeros behind them.
__device__ __forceinline__ void rank_keys(const uint64_t *cand, int found, int top, uint64_t *out) {
  for (int i = threadIdx.x; i < found; i += kTopThreads) {
    const uint64_t key = cand[i];
    int rank = 0;
#pragma unroll 8
    for (int j = 0; j < found; ++j) rank += cand[j] > key;
    if (rank < top) out[rank] = key;
  }
  for (int i = found + threadIdx.x; i < top; i += kTopThreads) out[i] = 0;
}

// The `top` largest of a row's columns [0, cols), larger first, to out[0 .. top - 1]
// (0: none left).
//
// At least `top` threads have a largest value of the top-th largest of these or
// more, so it bounds the answer from below: only the values of threads that reach it
// are looked at again, all threads together, and the few that reach it are ranked by
// counting.  (Of that bound the upper 16 bits are found.)  Should more than kMaxCand
// values reach it, it is mostly because they are equal (tokens masked by the type's lowest
// value): then all of the bound is found, the values above it are ranked, and those that
// equal it come in the row's order until there are enough.  And should more than kMaxCand
// be above it, the largest is taken `top` times over the whole row.
// 4096 x 65,536 bf16 with ten tokens left and five alternatives 184 us (by rounds over the whole
// row 1134), ordinary rows 110.
template <typename T>
__device__ void top_of_row(const T *row, int cols, float own_max, int top, uint32_t *tmax, uint64_t *cand, int *count,
                           uint64_t *out) {
  constexpr int N = kPiece<T>, W = kTopThreads;
  const int lane = threadIdx.x;
  const uint32_t own = order_bits(own_max);
  __syncthreads();
  tmax[lane] = own;
  if (lane == 0) count[0] = count[2] = 0;
  __syncthreads();
  if (lane < 64) {
    uint32_t mine[W / 64];
#pragma unroll
    for (int i = 0; i < W / 64; ++i) mine[i] = tmax[i * 64 + lane];
    const uint32_t bound = bound_of(mine, top);
    if (lane == 0) count[1] = (int)max(bound, kNoneBits + 1);
  }
  __syncthreads();
  const uint32_t bound = (uint32_t)count[1];
  if (own >= bound) tmax[atomicAdd(count + 2, 1)] = lane;  // nobody's tmax is read from here on
  __syncthreads();
  const int holders = count[2], each = (cols + W * N - 1) / (W * N);
  bool room = true;  // all that overflow need to know is that there are too many
  for (int i = lane; room && i < holders * each; i += W) {
    const int j = i / holders, at = (j * W + (int)tmax[i - j * holders]) * N;
    float v[N];
    load_values(row, at, cols - at, v);
#pragma unroll
    for (int e = 0; e < N; ++e)
      if (order_bits(v[e]) >= bound) {
        const int place = atomicAdd(count, 1);  // the order does not matter: ranked below
        if (place < kMaxCand)
          cand[place] = order_key(v[e], at + e);
        else
          room = false;
      }
  }
  __syncthreads();
  const int found = count[0];
  if (found <= kMaxCand) {
    rank_keys(cand, found, top, out);
    __syncthreads();
    return;
  }
  // the whole bound; -inf where fewer than `top` threads hold more
  __syncthreads();
  tmax[lane] = own;
  if (lane == 0) count[0] = 0;
  __syncthreads();
  if (lane < 64) {
    uint32_t mine[W / 64];
#pragma unroll
    for (int i = 0; i < W / 64; ++i) mine[i] = tmax[i * 64 + lane];
    const uint32_t exact = bound_of(mine, top, bound_of(mine, top), 15);
    if (lane == 0) count[1] = (int)max(exact, kNoneBits);
  }
  __syncthreads();
  const uint32_t least = (uint32_t)count[1];
  if (own > least)
    for (int i = lane * N; i < cols; i += W * N) {
      float v[N];
      load_values(row, i, cols - i, v);
#pragma unroll
      for (int e = 0; e < N; ++e)
        if (order_bits(v[e]) > least) {
          const int place = atomicAdd(count, 1);
          if (place < kMaxCand) cand[place] = order_key(v[e], i + e);
        }
    }
  __syncthreads();
  int have = count[0];
  if (have <= kMaxCand) {
    for (int base = 0; base < cols && have < top && least > kNoneBits; base += W * N) {
      const int i = base + lane * N;
      float v[N];
      load_values(row, i, cols - i, v);
      int equal = 0;
#pragma unroll
      for (int e = 0; e < N; ++e) equal += order_bits(v[e]) == least;
      int before = equal;  // of this piece and the lower ones
#pragma unroll
      for (int off = 1; off < 64; off <<= 1) {
        const int o = __shfl_up(before, off, 64);
        if ((lane & 63) >= off) before += o;
      }
      __syncthreads();
      if ((lane & 63) == 63) tmax[lane >> 6] = before;
      __syncthreads();
      int place = have + before - equal, all = 0;
#pragma unroll
      for (int w = 0; w < W / 64; ++w) {
        if (w < lane >> 6) place += (int)tmax[w];
        all += (int)tmax[w];
      }
#pragma unroll
      for (int e = 0; e < N; ++e)
        if (order_bits(v[e]) == least) {
          if (place < top) cand[place] = order_key(v[e], i + e);
          ++place;
        }
      have = min(have + all, top);
    }
    __syncthreads();
    rank_keys(cand, have, top, out);
    __syncthreads();
    return;
  }
  uint64_t last = ~(uint64_t)0;
  for (int r = 0; r < top; ++r) {
    uint64_t best = 0;
    if (own > kNoneBits)
      for (int i = lane * N; i < cols; i += W * N) {
        float v[N];
        load_values(row, i, cols - i, v);
#pragma unroll
        for (int e = 0; e < N; ++e) {
          const uint64_t key = order_key(v[e], i + e);
          if (key < last && key > best && order_bits(v[e]) > kNoneBits) best = key;
        }
      }
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) {
      const uint64_t o = __shfl_xor((unsigned long long)best, off, 64);
      best = o > best ? o : best;
    }
    __syncthreads();
    if ((lane & 63) == 0) cand[lane >> 6] = best;
    __syncthreads();
    best = cand[0];
#pragma unroll
    for (int w = 1; w < W / 64; ++w) best = cand[w] > best ? cand[w] : best;
    if (lane == 0) out[r] = best;
    last = best;
  }
  __syncthreads();
}

// ---- what a row's sums give ----
// log S; NaN of a row that holds NaN or +inf; 0 of a row without a value above -inf
__device__ __forceinline__ float log_sum(float m, float rest) {
  return m == -INFINITY && !(rest != rest) ? 0.f : log1pf(rest);
}
__device__ __forceinline__ float log_prob(float x, float m, float log_s, float inv_t) {
  if (m == -INFINITY && !(log_s != log_s)) return -INFINITY;  // a row without a token
  return -((m - x) * inv_t) - log_s;
}

// The given token of a row and its value.
struct Given {
  int id;  // -1: none
  float x;
};
template <typename T>
__device__ __forceinline__ Given given_of(const LogprobArgs &a, int64_t row, int id, bool report) {
  if (id < 0 || id >= a.V) {
    if (report && id != -1 && a.bad) atomicAdd(a.bad, 1u);
    return {-1, 0.f};
  }
  return {id, load_f32((const T *)a.x, row * a.V + id)};
}
__device__ __forceinline__ void finish_row(const LogprobArgs &a, int64_t row, const Given &given, float m, float rest,
                                           float q) {
  const float log_s = log_sum(m, rest);
  a.stats[2 * row] = m;
  a.stats[2 * row + 1] = log_s;
  if (a.entropy) a.entropy[row] = m == -INFINITY && !(log_s != log_s) ? 0.f : log_s + q * kLn2 / (1.f + rest);
  if (a.ids) a.logprob[row] = given.id >= 0 ? log_prob(given.x, m, log_s, a.inv_t) : 0.f;
}
__device__ __forceinline__ void finish_top(const LogprobArgs &a, int64_t row, int i, uint64_t key, float m,
                                           float log_s) {
  const bool none = key == 0 || log_s != log_s;
  a.top_ids[row * a.top + i] = none ? -1 : (int)~(uint32_t)key;
  a.top_logprob[row * a.top + i] =
      log_s != log_s ? NAN : key == 0 ? -INFINITY : log_prob(from_order_bits((uint32_t)(key >> 32)), m, log_s, a.inv_t);
}

// a slice's sums and top keys in the workspace, in floats
__host__ __device__ constexpr int part_floats(int top) { return 4 + 2 * top; }

}  // namespace

template <typename T, int W, bool ENT, bool TOP>
__global__ __launch_bounds__(256, 6) void logprob_kernel(LogprobArgs a, LogprobPlan plan) {
  constexpr int R = 256 / W;
  __shared__ float red[2 * 256 / 64];
  __shared__ uint32_t tmax[TOP ? kTopThreads : 1];
  __shared__ uint64_t cand[TOP ? kMaxCand : 1];
  __shared__ uint64_t best[TOP ? kMaxTop : 1];
  __shared__ int count[3];
  const int lane = threadIdx.x % W;
  const float c = a.inv_t * kLog2e;
  const int64_t jobs = a.n * plan.slices;
  // W > 64: the job is the same for the whole workgroup, as the barriers need
  for (int64_t job = (int64_t)blockIdx.x * R + threadIdx.x / W; job < jobs; job += (int64_t)gridDim.x * R) {
    const int64_t row = plan.slices == 1 ? job : job / plan.slices;
    const int64_t c0 = (job - row * plan.slices) * plan.slice;
    const int cols = (int)(a.V - c0 < plan.slice ? a.V - c0 : plan.slice);
    const T *x = (const T *)a.x + row * a.V + c0;
    const int id = !TOP && a.ids && plan.slices == 1 ? a.ids[row] : -1;
    Sums s = {-INFINITY, 0.f, 0.f};
    stream_row<T, W, ENT, false, TOP>(x, cols, lane, c, nullptr, s);
    Given given = {-1, 0.f};
    if (!TOP) given = given_of<T>(a, row, id, lane == 0);  // comes while the sums are joined
    const Sums all = join_threads<W, ENT>(s, c, red);
    const float rest = rest_of<T, W>(x, cols, lane, c, s, all, red);
    if constexpr (TOP) top_of_row<T>(x, cols, s.m, a.top, tmax, cand, count, best);
    if (plan.slices == 1) {
      if (lane == 0) {
        if (TOP && a.ids) given = given_of<T>(a, row, a.ids[row], true);
        finish_row(a, row, given, all.m, rest, all.q);
      }
      if constexpr (TOP) {
        const float log_s = log_sum(all.m, rest);
        for (int i = lane; i < a.top; i += W) finish_top(a, row, i, best[i], all.m, log_s);
      }
    } else {
      float *part = a.part + job * part_floats(TOP ? a.top : 0);
      if (lane == 0) {
        part[0] = all.m;
        part[1] = rest;
        part[2] = all.q;
      }
      if constexpr (TOP)
        for (int i = lane; i < a.top; i += W) ((uint64_t *)(part + 4))[i] = best[i] ? best[i] - (uint32_t)c0 : 0;
    }
  }
}

// A row out of its slices: one wave joins their sums, another bounds their keys, and
// the workgroup ranks those that reach the bound.
template <typename T>
__global__ __launch_bounds__(kTopThreads) void logprob_join_kernel(LogprobArgs a, LogprobPlan plan) {
  __shared__ uint64_t cand[kMaxCand], kept[kMaxCand], best[kMaxTop];
  __shared__ float got[2];
  __shared__ int count[2];
  const int64_t row = blockIdx.x;
  const float *part = a.part + row * plan.slices * part_floats(a.top);
  const float c = a.inv_t * kLog2e;
  const int total = plan.slices * a.top;
  // the first wave's part is on its way before the keys are
  const int i = threadIdx.x;
  const bool in = i < plan.slices && i < 64;
  const float *p = part + (in ? i : 0) * part_floats(a.top);
  const float m = in ? p[0] : -INFINITY, rest = in ? p[1] : -1.f, q = in ? p[2] : 0.f;
  const Given given = i == 0 ? given_of<T>(a, row, a.ids ? a.ids[row] : -1, true) : Given{-1, 0.f};
  for (int i = threadIdx.x; i < total; i += kTopThreads) {
    const int slice = i / a.top;
    cand[i] = ((const uint64_t *)(part + slice * part_floats(a.top) + 4))[i - slice * a.top];
  }
  if (threadIdx.x == 0) count[0] = 0;
  if (threadIdx.x < 64) {
    const float top = all_max<64>(m, nullptr);
    // a slice's whole sum, but for the first that holds the largest value
    const uint64_t holds = __ballot(m == top);
    const bool owner = (holds & (((uint64_t)1 << i) - 1)) == 0 && m == top;
    float t = rest + 1.f, r = rest, qq = q;
    if (t != 0.f) {
      const float d = fminf((top - m) * c, kFar), f = exp2_neg(d);
      qq = (q + d * t) * f;
      r = owner ? rest : t * f;
      if (top - m != top - m) r = NAN;
    } else {
      r = 0.f;
      qq = 0.f;
    }
    all_sum2<64>(r, qq, nullptr);
    if (top == -INFINITY && !(r != r)) r = -1.f;
    if (i == 0) {
      finish_row(a, row, given, top, r, qq);
      got[0] = top;
      got[1] = log_sum(top, r);
    }
  }
  if (a.top == 0) return;
  __syncthreads();
  if (threadIdx.x >= 64 && threadIdx.x < 128) {
    // A slice's keys are in order: where `of` slices have a key of the bound or more in place
    // `deep`, at least `top` keys reach it.
    const int deep = (a.top - 1) / plan.slices, of = (a.top + deep) / (deep + 1);
    const int slice = threadIdx.x - 64;
    const uint32_t mine[1] = {slice < plan.slices ? (uint32_t)(cand[slice * a.top + deep] >> 32) : 0};
    const uint32_t bound = bound_of(mine, of);
    if (slice == 0) count[1] = (int)max(bound, kNoneBits + 1);
  }
  __syncthreads();
  const uint32_t bound = (uint32_t)count[1];
  for (int i = threadIdx.x; i < total; i += kTopThreads)
    if ((uint32_t)(cand[i] >> 32) >= bound) kept[atomicAdd(count, 1)] = cand[i];
  __syncthreads();
  rank_keys(kept, count[0], a.top, best);
  __syncthreads();
  for (int i = threadIdx.x; i < a.top; i += kTopThreads) finish_top(a, row, i, best[i], got[0], got[1]);
}

LogprobPlan logprob_plan(int64_t n, int V, int top, bool bf16) {
  // Fewer rows than would fill the device, and so long that a second launch takes less than one
  // workgroup's way along them: several workgroups each (65,536 fp32: one row 5.0 us, 10.7 in one, 255
  // rows 15.5 and 18.7, 400 rows 21.5 and 20.1; 65,536 bf16: one row 5.1 and 8.3, 160 rows 8.7 and 9.1, 200
  // rows 11.6 and 11.2; 16,384 fp32, one row: 5.0 and 4.5; with five alternatives 9.3 and 13.2, 10.2 and
  // 11.9, 9.3 and 7.2).
  int64_t slices = 1;
  const int64_t bytes = (int64_t)V * (bf16 ? 2 : 4);
  if (bytes >= 1 << 17 && n <= (bytes >= 1 << 18 ? 256 : 160)) {
    slices = ceil_div(512, n);
    if (slices > V / 2048) slices = V / 2048;
    if (slices > 64) slices = 64;  // a lane each in the join
    if (top > 0 && slices * top > kMaxCand) slices = kMaxCand / top;
  }
  const int64_t slice = round_up(ceil_div(V, slices), 8);
  return {(int)ceil_div(V, slice), slice};
}
size_t logprob_part_floats(int64_t n, const LogprobPlan &p, int top) {
  return p.slices == 1 ? 0 : (size_t)n * p.slices * part_floats(top);
}

template <typename T, int W, bool TOP>
static void start_logprobs(const LogprobArgs &a, const LogprobPlan &plan, hipStream_t s) {
  const int64_t groups = ceil_div(a.n * plan.slices, 256 / W);
  const dim3 grid((unsigned)(groups < kMaxGroups ? groups : kMaxGroups));
  if (a.entropy)
    logprob_kernel<T, W, true, TOP><<<grid, 256, 0, s>>>(a, plan);
  else
    logprob_kernel<T, W, false, TOP><<<grid, 256, 0, s>>>(a, plan);
}

template <typename T>
static hipError_t logprobs(const LogprobArgs &a, hipStream_t s) {
  const LogprobPlan plan = logprob_plan(a.n, a.V, a.top, sizeof(T) == 2);
  // Threads of a row.  Of short rows what is done once a row weighs most, and a wave does it
  // for four rows as for one: 1,024 bf16 columns of 293,000 rows 112 us with 16 threads, 139
  // with 32, 189 with 64; 2,048 of 146,000 113, 117, 137, but of 6,144 10.0 and 9.1 with 64.  A
  // workgroup for a row of 2,049 takes 311 where a wave takes 163; of 24,576 rows of 8,192
  // 91 where a wave takes 80, but fp32 rows of 4,096 79 where that takes 83, and 512 rows of
  // 4,096 4.6 where that takes 5.2.  The top alternatives are picked by a workgroup.
  const int64_t bytes = (int64_t)a.V * sizeof(T);
  constexpr bool narrow = sizeof(T) == 2;
  if (a.top > 0)
    start_logprobs<T, 256, true>(a, plan, s);
  else if (bytes <= 2048 || (narrow && bytes <= 4096 && a.n >= 16384))
    start_logprobs<T, 16, false>(a, plan, s);
  else if (bytes <= 4096 || (bytes <= (narrow ? 16384 : 12288) && a.n >= 2048))
    start_logprobs<T, 64, false>(a, plan, s);
  else
    start_logprobs<T, 256, false>(a, plan, s);
  if (plan.slices > 1) logprob_join_kernel<T><<<dim3((unsigned)a.n), kTopThreads, 0, s>>>(a, plan);
  return hipGetLastError();
}

hipError_t launch_logprobs(const LogprobArgs &a, bool x_bf16, hipStream_t s) {
  if (a.n == 0) return hipSuccess;
  return x_bf16 ? logprobs<uint16_t>(a, s) : logprobs<float>(a, s);
}

namespace {

template <typename T, int W>
__device__ __forceinline__ void zero_row(T *dx, int cols, int lane) {
  constexpr int N = kPiece<T>;
  const float v[N] = {};
  for (int i = lane * N; i < cols; i += W * N) store_n<N>(dx + i, cols - i, v);
}
// dx = f(x) for a thread's pieces of a row; dx may be x.  At the row's end as above: what
// is read twice is written by the piece that it belongs to, out of that piece's own load.
template <typename T, int W, int P, bool TAIL, typename F>
__device__ __forceinline__ void map_pieces(const T *x, T *dx, int cols, int at, F f) {
  constexpr int N = kPiece<T>;
  u32x4 raw[P];
#pragma unroll
  for (int p = 0; p < P; ++p) {
    const int i = at + p * W * N;
    raw[p] = load16(x + (TAIL ? min(i, cols - N) : i));
  }
#pragma unroll
  for (int p = 0; p < P; ++p) {
    const int i = at + p * W * N;
    if (TAIL && i >= cols) break;
    float v[N];
    unpack(raw[p], v);
#pragma unroll
    for (int e = 0; e < N; ++e) v[e] = f(v[e]);
    if (!TAIL || i + N <= cols) {
      store_n<N>(dx + i, N, v);
    } else {
#pragma unroll
      for (int e = 1; e < N; ++e)
        if (cols - N + e >= i) store_f32(dx, cols - N + e, v[e]);
    }
  }
}
template <typename T, int W, typename F>
__device__ __forceinline__ void map_row(const T *x, T *dx, int cols, int lane, F f) {
  constexpr int N = kPiece<T>, P = kPieces;
  if (cols < N) {
    if (lane > 0) return;
    float v[N];
    unpack(load_piece(x, cols), v);
#pragma unroll
    for (int e = 0; e < N; ++e) v[e] = f(v[e]);
    store_n<N>(dx, cols, v);
    return;
  }
  int base = 0;
  for (; base + W * P * N <= cols; base += W * P * N)
    map_pieces<T, W, P, false>(x, dx, cols, base + lane * N, f);
  if (cols - base > 2 * W * N)
    map_pieces<T, W, P, true>(x, dx, cols, base + lane * N, f);
  else if (base < cols)
    map_pieces<T, W, 2, true>(x, dx, cols, base + lane * N, f);
}

}  // namespace

// ---- the gradient of log probabilities and entropies ----
//   dx_j = (g ([j = id] - p_j) - gH p_j (log p_j + H)) / T
// With e_j = exp(-d_j) = S p_j this is e_j (A + B d_j), A = -(g + gH (H - log S)) / (S T),
// B = gH / (S T); the given token's own element uses 1 - p = -expm1(log p).
template <typename T, int W>
__global__ __launch_bounds__(256, 6) void logprob_grad_kernel(LogprobGradArgs a, int slices, int64_t slice) {
  constexpr int R = 256 / W, N = kPiece<T>;
  const int lane = threadIdx.x % W;
  const float c = a.inv_t * kLog2e;
  const int64_t jobs = a.n * slices;
  for (int64_t job = (int64_t)blockIdx.x * R + threadIdx.x / W; job < jobs; job += (int64_t)gridDim.x * R) {
    const int64_t row = slices == 1 ? job : job / slices;
    const int64_t c0 = (job - row * slices) * slice;
    const int cols = (int)(a.V - c0 < slice ? a.V - c0 : slice);
    const T *x = (const T *)a.x + row * a.V + c0;
    T *dx = (T *)a.dx + row * a.V + c0;
    const float m = a.stats[2 * row], log_s = a.stats[2 * row + 1];
    int64_t id = a.ids ? a.ids[row] : -1;
    if (id < 0 || id >= a.V) id = -1;
    const float g = a.dlogprob && id >= 0 ? a.dlogprob[row] : 0.f;
    const float gh = a.dentropy ? a.dentropy[row] : 0.f;
    // no weight, or no token to put it on: zeros, whatever the logits are
    if ((g == 0.f && gh == 0.f) || (m == -INFINITY && !(log_s != log_s))) {
      zero_row<T, W>(dx, cols, lane);
      continue;
    }
    const float h = gh != 0.f ? a.entropy[row] : 0.f;
    const float k = expf(-log_s) * a.inv_t;
    const float A = -(g + gh * (h - log_s)) * k, B = gh * kLn2 * k;
    // the given token's own element is this lane's to write again; it is read before (dx may be x)
    const int64_t at_id = id - c0;
    const bool mine = id >= 0 && at_id >= 0 && at_id < cols && (int)(at_id / N) % W == lane;
    const float x_id = mine ? load_f32(x, at_id) : 0.f;
    map_row<T, W>(x, dx, cols, lane, [&](float v) {
      const float d = fminf((m - v) * c, kFar);
      return exp2_neg(d) * (A + B * d);
    });
    if (mine) {
      const float lp = log_prob(x_id, m, log_s, a.inv_t), p = expf(lp);
      store_f32(dx, at_id, (-g * expm1f(lp) - (p > 0.f ? gh * p * (lp + h) : 0.f)) * a.inv_t);
    }
  }
}

template <typename T>
static hipError_t logprobs_grad(const LogprobGradArgs &a, hipStream_t s) {
  constexpr int N = kPiece<T>;
  // a workgroup a row; of few rows several, of four pieces a thread at least (65,536 fp32, one
  // row 2.8 us, 8.5 in one; 128 rows 11.9 and 14.1, 400 rows 33.0 and 32.6)
  int64_t slices = 1;
  if (a.n < 1024) {
    slices = ceil_div(2048, a.n);
    const int64_t most = ceil_div(a.V, 256 * kPieces * N);
    if (slices > most) slices = most;
  }
  const int64_t slice = round_up(ceil_div(a.V, slices), 8);
  slices = ceil_div(a.V, slice);
  const auto grid = [&](int rows) {
    const int64_t groups = ceil_div(a.n * slices, rows);
    return dim3((unsigned)(groups < kMaxGroups ? groups : kMaxGroups));
  };
  // Threads of a row, four pieces each: 512 bf16 columns of 586,000 rows 201 us with 16
  // threads, 251 with 32; 1,024 of 293,000 199 with 32, 224 with 16, 246 with 64; 4,096 of 73,000 218 with
  // 64, 234 with a workgroup, which takes 200 for 8,192 of 36,600 where a wave takes 225.
  const int64_t bytes = (int64_t)a.V * sizeof(T);
  if (slices == 1 && bytes <= 1024)
    logprob_grad_kernel<T, 16><<<grid(16), 256, 0, s>>>(a, 1, slice);
  else if (slices == 1 && bytes <= 2048)
    logprob_grad_kernel<T, 32><<<grid(8), 256, 0, s>>>(a, 1, slice);
  else if (slices == 1 && (bytes <= 4096 || (bytes <= 8192 && a.n >= 2048)))
    logprob_grad_kernel<T, 64><<<grid(4), 256, 0, s>>>(a, 1, slice);
  else
    logprob_grad_kernel<T, 256><<<grid(1), 256, 0, s>>>(a, (int)slices, slice);
  return hipGetLastError();
}

hipError_t launch_logprobs_grad(const LogprobGradArgs &a, bool x_bf16, hipStream_t s) {
  if (a.n == 0) return hipSuccess;
  return x_bf16 ? logprobs_grad<uint16_t>(a, s) : logprobs_grad<float>(a, s);
}

// ---- distillation ----
// The teacher gives k tokens of each row and values t.  Without tail, q is the
// softmax of t / T over them; with tail, q = exp(t), and all other tokens are one
// outcome more: q_T = 1 - sum q beside p_T, the sum of their p.
//   loss = sum q_e (log q_e - log p_e) (+ q_T (log q_T - log p_T))
//   dx_j = (p_j - q_j) / T;   with tail, of the others: p_j (1 - q_T / p_T) / T
// (without tail, q_j = 0 for the others.)  A repeated ID counts where it comes
// first; a row without a valid ID has no loss and no gradient.
//
// One thread an entry; q and the loss are computed in 64 bits (a few numbers a
// row).  p_T is added up over the others themselves, whose places a map of bits in
// LDS tells apart, not as 1 - sum p, which would lose a small p_T.
//
// Bound by memory where rows are long (4096 x 65,536 bf16 with tail 125 to 129 us, 4.2 TB/s,
// without 108; its gradient 204 behind the loss, 5.4, and 231 where gradients follow one another and
// wait for each other's writes), and by what is done once a row, in 64 bits, where they are short (1,171,875 x 256 with 64 entries 2.1 ms).

namespace {

constexpr int kSegment = 1 << 18;  // columns that the map holds at once: 32 KB
// What the teacher's entries may leave where no other token has any weight: fp32 logarithms
// are off by 2^-24 of themselves, the teacher's own softmax by a few times that.
constexpr double kNoRest = 0x1p-16;
// The others have no weight where log p_T is below that of fp32's smallest number, 2^-149: they are
// masked, by -inf or by a large negative value alike (whose logarithm times a rounding's rest would
// be the whole loss: 2^-26 times the type's lowest value is 5e30).
constexpr double kNoWeight = -149 * 0.69314718055994530942;

struct Entry {
  int id;       // -1: does not count
  double q, logq;
};
// The row's entry of this thread; the row's W threads call it together.
template <int W>
__device__ Entry entry_of(const DistillArgs &a, int64_t row, int lane, int *ids, double *red, bool count_bad) {
  int id = -1;
  double t = 0.0;
  if (lane < a.k) {
    id = a.ids[row * a.k + lane];
    if (id < 0 || id >= a.V) {
      if (id != -1 && a.bad && count_bad) atomicAdd(a.bad, 1u);
      id = -1;
    }
    t = (double)a.teacher[row * a.k + lane];
  }
  if (W > 64) __syncthreads();
  if (lane < a.k) ids[lane] = id;
  if (W > 64)
    __syncthreads();
  else
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  if (id >= 0) {
    bool again = false;
    for (int j = 0; j < lane; ++j) again |= ids[j] == id;
    if (again) id = -1;
  }
  Entry e = {id, 0.0, 0.0};
  if (a.tail) {
    e.logq = t;
  } else {
    t *= (double)a.inv_t;
    // NaN is not lost: it returns in the sum
    float top = all_max<W>(id >= 0 ? (float)t : -INFINITY, (float *)red);
    if (top == -INFINITY) top = 0.f;
    const double z = all_sum<W>(id >= 0 ? exp(t - (double)top) : 0.0, red);
    if (z == 0.0) e.id = -1;  // all of them masked: the teacher says nothing
    e.logq = t - (double)top - log(z);
  }
  if (e.id >= 0) e.q = exp(e.logq);
  return e;
}

template <int W>
__device__ __forceinline__ void row_barrier() {
  if (W > 64)
    __syncthreads();
  else
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
}

}  // namespace

template <typename T, int W, bool TAIL>
__global__ __launch_bounds__(256, 4) void distill_kernel(DistillArgs a, int words) {
  constexpr int R = 256 / W;
  extern __shared__ uint32_t maps[];  // [R][words]
  __shared__ double red64[R][16];
  __shared__ int ids[R][W];
  const int lane = threadIdx.x % W, sub = threadIdx.x / W;
  uint32_t *map = maps + sub * words;
  double *red = red64[sub];
  const float c = a.inv_t * kLog2e;
  for (int64_t row = (int64_t)blockIdx.x * R + sub; row < a.n; row += (int64_t)gridDim.x * R) {
    const T *x = (const T *)a.x + row * a.V;
    const Entry en = entry_of<W>(a, row, lane, ids[sub], red, true);
    const float xe = en.id >= 0 ? load_f32(x, en.id) : -INFINITY;
    Sums s = {-INFINITY, 0.f, 0.f};
    if constexpr (TAIL) {
      for (int64_t c0 = 0; c0 < a.V; c0 += kSegment) {
        const int cols = (int)(a.V - c0 < kSegment ? a.V - c0 : kSegment);
        row_barrier<W>();
        for (int i = lane; i < words; i += W) map[i] = 0;
        row_barrier<W>();
        if (en.id >= c0 && en.id < c0 + cols) atomicOr(map + ((en.id - (int)c0) >> 5), 1u << (en.id & 31));
        row_barrier<W>();
        stream_row<T, W, false, true, false>(x + c0, cols, lane, c, (const uint8_t *)map, s);
      }
    } else {
      stream_row<T, W, false, false, false>(x, a.V, lane, c, nullptr, s);
    }
    const Sums others = join_threads<W, false>(s, c, (float *)red);  // without tail: all tokens
    // log S out of the sum without one of its largest terms, in 64 bits: where student and teacher
    // are all but certain, the loss is the difference of such small numbers.
    const double inv_t = (double)a.inv_t;
    float m = others.m;
    double rest_s, log_s;
    bool empty;
    if constexpr (TAIL) {
      m = fmaxf(m, all_max<W>(xe, (float *)red));
      const int owner = all_min<W>(xe == m && m > -INFINITY ? lane : W, (int *)red);
      double t = 0.0;
      if (lane != owner && (xe > -INFINITY || xe != xe)) t = exp(((double)xe - (double)m) * inv_t);
      rest_s = all_sum<W>(t, red);
      if (!(others.t == 0.f)) rest_s += (double)others.t * exp(((double)others.m - (double)m) * inv_t);
      empty = owner == W && rest_s == 0.0;
      log_s = owner < W ? log1p(rest_s) : log(rest_s);
      if (m == INFINITY) log_s = NAN;
    } else {
      const float rest = rest_of<T, W>(x, a.V, lane, c, s, others, (float *)red);
      empty = others.t == 0.f;
      log_s = log1p((double)rest);
    }
    double term = 0.0;
    if (en.id >= 0 && en.q != 0.0) {  // NaN goes on
      const double log_p = ((double)xe - (double)m) * inv_t - log_s;
      term = en.q * (en.logq - log_p);
    }
    const double any = all_sum<W>(en.id >= 0 ? 1.0 : 0.0, red);
    double loss = all_sum<W>(term, red);
    const double sum_q = TAIL ? all_sum<W>(en.q, red) : 1.0;
    if (lane == 0) {
      // of the others: dx_j T = exp((x_j - from) / T) factor
      float from = m;
      double factor = exp(-log_s);
      if (TAIL) {
        double rest = 1.0 - sum_q;
        if (rest < 0.0) rest = 0.0;
        // by the others' own largest value: p_T may be too small for fp32
        const double down = ((double)others.m - (double)m) * inv_t - log_s;
        const double log_left = others.t == 0.f ? -INFINITY : down + log((double)others.t);
        if (rest <= kNoRest && log_left < kNoWeight) {
          factor = 0.0;
        } else if (others.t == 0.f) {
          if (rest > kNoRest) loss = INFINITY;
          factor = 0.0;
        } else {
          if (rest != 0.0) loss += rest * (log(rest) - log_left);
          from = others.m;
          factor = exp(down) - rest / (double)others.t;
        }
      }
      const bool masked = m == -INFINITY && empty;  // no token to put weight on
      const bool none = any == 0.0;
      a.loss[row] = none ? 0.f : masked ? INFINITY : (float)loss;
      float *st = a.stats + 4 * row;
      st[0] = none ? -INFINITY : m;  // -inf, 0: the gradient is zero
      st[1] = none || masked ? 0.f : (float)log_s;
      st[2] = from;
      st[3] = (float)factor;
    }
  }
}

template <typename T, int W>
__global__ __launch_bounds__(256, 4) void distill_grad_kernel(DistillArgs a) {
  constexpr int R = 256 / W;
  __shared__ double red64[R][16];
  __shared__ int ids[R][W];
  const int lane = threadIdx.x % W, sub = threadIdx.x / W;
  const float c = a.inv_t * kLog2e;
  for (int64_t row = (int64_t)blockIdx.x * R + sub; row < a.n; row += (int64_t)gridDim.x * R) {
    const T *x = (const T *)a.x + row * a.V;
    T *dx = (T *)a.dx + row * a.V;
    const float *st = a.stats + 4 * row;
    const float m = st[0], log_s = st[1], g = a.dloss[row] * a.inv_t;
    if (g == 0.f || (m == -INFINITY && log_s == 0.f)) {  // the same for the row's threads
      zero_row<T, W>(dx, a.V, lane);
      continue;
    }
    const Entry en = entry_of<W>(a, row, lane, ids[sub], red64[sub], false);
    // read before anything is written: dx may be x
    const float xe = en.id >= 0 ? load_f32(x, en.id) : 0.f;
    row_barrier<W>();
    const float from = st[2], A = g * st[3];
    map_row<T, W>(x, dx, a.V, lane, [&](float v) { return A * exp2_neg((from - v) * c); });
    row_barrier<W>();
    if (en.id >= 0) {
      const double p = exp(((double)xe - (double)m) * (double)a.inv_t - (double)log_s);
      store_f32(dx, en.id, g * (float)(p - en.q));
    }
  }
}

template <typename T, int W>
static void start_distill(const DistillArgs &a, bool grad, hipStream_t s) {
  constexpr int R = 256 / W;
  const int64_t groups = ceil_div(a.n, R);
  const dim3 grid((unsigned)(groups < kMaxGroups ? groups : kMaxGroups));
  if (grad) {
    distill_grad_kernel<T, W><<<grid, 256, 0, s>>>(a);
  } else if (a.tail) {
    const int words = (int)ceil_div(a.V < kSegment ? a.V : kSegment, 32) + 1;
    distill_kernel<T, W, true><<<grid, 256, (size_t)R * words * 4, s>>>(a, words);
  } else {
    distill_kernel<T, W, false><<<grid, 256, 0, s>>>(a, 0);
  }
}

template <typename T>
static hipError_t distill(const DistillArgs &a, bool grad, hipStream_t s) {
  // At least as many threads as the teacher has entries.  What is done once a row a wave does
  // for itself, the four of a workgroup together for one row: 16,384 x 2049 bf16 40 us with a wave
  // a row and 136, 16,384 x 32,000 200 and 288; the gradient, with less of it, of 16,384 x 2049 37
  // and 80, of 8192 columns 136 and 128.
  static_assert(kMaxTeacher <= 256, "a thread each");
  if (a.k <= 64 && (a.V <= 2048 || (a.V * sizeof(T) <= (grad ? 12288 : 65536) && a.n >= 2048)))
    start_distill<T, 64>(a, grad, s);
  else
    start_distill<T, 256>(a, grad, s);
  return hipGetLastError();
}

hipError_t launch_distill(const DistillArgs &a, bool x_bf16, hipStream_t s) {
  if (a.n == 0) return hipSuccess;
  return x_bf16 ? distill<uint16_t>(a, false, s) : distill<float>(a, false, s);
}
hipError_t launch_distill_grad(const DistillArgs &a, bool x_bf16, hipStream_t s) {
  if (a.n == 0) return hipSuccess;
  return x_bf16 ? distill<uint16_t>(a, true, s) : distill<float>(a, true, s);
}

}  // namespace rvq
