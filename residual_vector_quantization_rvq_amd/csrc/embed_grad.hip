// embed_grad.hip -- gradient of the unified token embedding (embed.hip).
//
//   dlevel[l][k] = sum of dout[t] over visual tokens t with ids[t][l] == k
//   dtext[v]     = sum of dout[t] over text tokens t with ids[t][0] == v
//
// No float atomics: every destination row is summed in token order, so the
// result depends on the inputs alone.
//
// embed_index_kernel lists, for each destination row, the tokens that add to
// it.  A workgroup owns kRange consecutive rows of one table and reads that
// table's column of the IDs twice: once to count (its rows, and the IDs below
// them, which is where its part of the table's list begins), once to place.
// Every wave has a piece of the tokens and a counter per row, so the lists
// come out in token order.
//
// embed_sum_kernel sums each row's tokens.  The list is also cut in segments
// of equal length: a row with more tokens than a segment (a hot codeword, a
// padding token) is summed segment by segment, and embed_join_kernel adds
// the pieces in order.
#include "learn.h"

namespace rvq {

namespace {

constexpr int kRange = 128;        // destination rows of one index workgroup
constexpr int kIndexThreads = 1024;
constexpr int kIndexWaves = kIndexThreads / 64;
constexpr int kThreads = 256;
constexpr int kMaxGroups = 1 << 20;

// Length of a segment of the list.  A row of at most this many tokens is
// summed in one go.
int64_t segment_length(int64_t positions) {
  const int64_t h = round_up(ceil_div(positions, 4096), 64);
  return h < 256 ? 256 : h;
}

// Which tables' gradients are wanted, and where their lists lie: T positions
// for each level, then T for the text table.
struct Tables {
  int L, K;        // L = 0: no level gradients
  int64_t V;       // 0: no text gradient
  int64_t T;
  int64_t rows, positions, seg, segments;
};

Tables tables_of(int64_t T, int L, int K, int64_t V) {
  Tables t;
  t.L = L;
  t.K = K;
  t.V = V;
  t.T = T;
  t.rows = (int64_t)L * K + V;
  t.positions = (L + (V > 0 ? 1 : 0)) * T;
  t.seg = segment_length(t.positions);
  // a row has at most T tokens: none is long if T is not
  t.segments = T > t.seg ? ceil_div(t.positions, t.seg) : 0;
  return t;
}

}  // namespace

__global__ __launch_bounds__(kIndexThreads) void embed_index_kernel(EmbedGradArgs a, Tables tb) {
  __shared__ int cnt[kIndexWaves][kRange];
  __shared__ int below_sum, total;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // this workgroup's rows [r0, r1) of its table
  const int per_level = (int)ceil_div(tb.K, kRange);
  const bool text = (int64_t)blockIdx.x >= (int64_t)tb.L * per_level;
  const int l = text ? 0 : blockIdx.x / per_level;
  const int range = text ? (int)(blockIdx.x - (int64_t)tb.L * per_level) : blockIdx.x % per_level;
  const int64_t limit = text ? tb.V : tb.K;
  const int64_t r0 = (int64_t)range * kRange;
  const int64_t r1 = r0 + kRange < limit ? r0 + kRange : limit;
  const int64_t region = text ? tb.L * tb.T : l * tb.T;
  const int64_t row0 = (text ? (int64_t)tb.L * tb.K : (int64_t)l * tb.K) + r0;

  for (int i = threadIdx.x; i < kIndexWaves * kRange; i += kIndexThreads) (&cnt[0][0])[i] = 0;
  if (threadIdx.x == 0) below_sum = 0;
  __syncthreads();

  const int64_t piece = round_up(ceil_div(tb.T, kIndexWaves), 64);
  const int64_t t0 = wave * piece < tb.T ? wave * piece : tb.T;
  const int64_t t1 = t0 + piece < tb.T ? t0 + piece : tb.T;
  // the token's ID in this table, or -1 (a token of the other kind)
  const auto id_of = [&](int64_t t, bool &mine) {
    mine = (a.is_visual == nullptr || a.is_visual[t] != 0) != text;
    return a.ids[t * a.L + l];
  };

  int below = 0, bad = 0;
  for (int64_t t = t0 + lane; t < t1; t += 64) {
    bool mine;
    const int id = id_of(t, mine);
    if (!mine) continue;
    if (id < 0 || id >= limit) {
      ++bad;
    } else if (id < r0) {
      ++below;
    } else if (id < r1) {
      atomicAdd(&cnt[wave][id - (int)r0], 1);
    }
  }
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) {
    below += __shfl_xor(below, off, 64);
    bad += __shfl_xor(bad, off, 64);
  }
  if (lane == 0) {
    if (below) atomicAdd(&below_sum, below);
    if (bad && range == 0 && a.bad) atomicAdd(a.bad, (uint32_t)bad);
  }
  __syncthreads();

  // a row's tokens: its waves' in turn; the rows one after the other
  if (wave == 0) {
    int mine[kRange / 64], sum = 0;
#pragma unroll
    for (int j = 0; j < kRange / 64; ++j) {
      int c = 0;
      for (int w = 0; w < kIndexWaves; ++w) {
        const int v = cnt[w][lane * (kRange / 64) + j];
        cnt[w][lane * (kRange / 64) + j] = c;
        c += v;
      }
      mine[j] = c;
      sum += c;
    }
    int incl = sum;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const int v = __shfl_up(incl, off, 64);
      if (lane >= off) incl += v;
    }
    int at = (int)region + below_sum + incl - sum;
#pragma unroll
    for (int j = 0; j < kRange / 64; ++j) {
      const int r = lane * (kRange / 64) + j;
      for (int w = 0; w < kIndexWaves; ++w) cnt[w][r] += at;
      if (r0 + r < r1) {
        a.start[row0 + r] = at;
        a.count[row0 + r] = mine[j];
      }
      at += mine[j];
    }
    if (lane == 63) total = at;
  }
  __syncthreads();
  // the table's last workgroup marks the positions that no token has
  if (r1 == limit)
    for (int64_t i = total + (int64_t)threadIdx.x; i < region + tb.T; i += kIndexThreads) a.row[i] = -1;

  for (int64_t tw = t0; tw < t1; tw += 64) {
    const int64_t t = tw + lane;
    bool mine = false;
    int id = -1;
    if (t < t1) id = id_of(t, mine);
    const bool hit = mine && id >= r0 && id < r1;
    if (__ballot(hit) == 0) continue;
    const int r = hit ? id - (int)r0 : 0;
    // lanes of the same row
    unsigned long long same = __ballot(hit);
#pragma unroll
    for (int b = 0; (1 << b) < kRange; ++b) {
      const unsigned long long m = __ballot((r >> b) & 1);
      same &= ((r >> b) & 1) ? m : ~m;
    }
    const int first = hit ? __ffsll((long long)same) - 1 : lane;
    int at = 0;
    if (hit && lane == first) at = atomicAdd(&cnt[wave][r], __popcll(same));
    at = __shfl(at, first, 64);
    if (hit) {
      at += __popcll(same & ((1ull << lane) - 1));
      a.token[at] = (int)t;
      a.row[at] = (int)(row0 + r);
    }
  }
}

namespace {

// sum of list entries [e0, e1) in column c
template <typename T>
__device__ __forceinline__ float sum_entries(const EmbedGradArgs &a, int64_t e0, int64_t e1, int c) {
  float s = 0.f;
  for (int64_t e = e0; e < e1; ++e) s += load_f32((const T *)a.dout, (int64_t)a.token[e] * a.D + c);
  return s;
}

template <typename G>
__device__ __forceinline__ G *row_of(const EmbedGradArgs &a, const Tables &tb, int64_t row) {
  const int64_t levels = (int64_t)tb.L * tb.K;
  return row < levels ? (G *)a.dlevel + row * a.D : (G *)a.dtext + (row - levels) * a.D;
}

}  // namespace

// Workgroups [0, row_groups) take rows; the others a segment each, whose
// first and last row may be long ones: their sums go to part[2 s] (the row
// that holds the segment's first position) and part[2 s + 1] (the row that
// begins inside it).
template <typename T, typename G>
__global__ __launch_bounds__(kThreads) void embed_sum_kernel(EmbedGradArgs a, Tables tb,
                                                             int row_groups) {
  if ((int)blockIdx.x < row_groups) {
    for (int64_t row = blockIdx.x; row < tb.rows; row += row_groups) {
      const int64_t n = a.count[row], e0 = a.start[row];
      if ((tb.segments && n > tb.seg) || (a.accumulate && n == 0)) continue;
      G *o = row_of<G>(a, tb, row);
      for (int c = threadIdx.x; c < a.D; c += kThreads) {
        float s = sum_entries<T>(a, e0, e0 + n, c);
        if (a.accumulate) s += load_f32(o, c);
        store_f32(o, c, s);
      }
    }
    return;
  }
  const int64_t s = blockIdx.x - row_groups;
  const int64_t p0 = s * tb.seg, p1 = p0 + tb.seg < tb.positions ? p0 + tb.seg : tb.positions;
  const int ra = a.row[p0], rb = a.row[p1 - 1];
  if (ra >= 0 && a.count[ra] > tb.seg) {
    const int64_t end = (int64_t)a.start[ra] + a.count[ra];
    for (int c = threadIdx.x; c < a.D; c += kThreads)
      a.part[2 * s * a.D + c] = sum_entries<T>(a, p0, end < p1 ? end : p1, c);
  }
  if (rb >= 0 && rb != ra && a.count[rb] > tb.seg) {
    for (int c = threadIdx.x; c < a.D; c += kThreads)
      a.part[(2 * s + 1) * a.D + c] = sum_entries<T>(a, a.start[rb], p1, c);
  }
}

// The long row that begins in segment s, if there is one: its pieces in order.
template <typename G>
__global__ __launch_bounds__(kThreads) void embed_join_kernel(EmbedGradArgs a, Tables tb) {
  const int64_t s = blockIdx.x;
  const int64_t p0 = s * tb.seg, p1 = p0 + tb.seg < tb.positions ? p0 + tb.seg : tb.positions;
  const int row = a.row[p1 - 1];
  if (row < 0 || a.count[row] <= tb.seg || a.start[row] < p0) return;
  const int64_t end = (int64_t)a.start[row] + a.count[row];
  const int64_t first = a.start[row] == p0 ? 2 * s : 2 * s + 1;
  G *o = row_of<G>(a, tb, row);
  for (int c = threadIdx.x; c < a.D; c += kThreads) {
    float v = a.part[first * a.D + c];
    for (int64_t q = s + 1; q * tb.seg < end; ++q) v += a.part[2 * q * a.D + c];
    if (a.accumulate) v += load_f32(o, c);
    store_f32(o, c, v);
  }
}

EmbedGradLayout embed_grad_layout(int64_t T, int L, int K, int64_t V, int D) {
  const Tables tb = tables_of(T, L, K, V);
  EmbedGradLayout w;
  w.start = 0;
  w.count = w.start + al256((size_t)tb.rows * 4);
  w.token = w.count + al256((size_t)tb.rows * 4);
  w.row = w.token + al256((size_t)tb.positions * 4);
  w.part = w.row + al256((size_t)tb.positions * 4);
  w.total = w.part + al256((size_t)tb.segments * 2 * D * sizeof(float));
  if (w.total == 0) w.total = 256;
  return w;
}

template <typename T, typename G>
static hipError_t launch_sums(const EmbedGradArgs &a, const Tables &tb, hipStream_t s) {
  const int row_groups = (int)(tb.rows < kMaxGroups ? tb.rows : kMaxGroups);
  embed_sum_kernel<T, G><<<dim3((unsigned)(row_groups + tb.segments)), kThreads, 0, s>>>(a, tb, row_groups);
  if (tb.segments) embed_join_kernel<G><<<dim3((unsigned)tb.segments), kThreads, 0, s>>>(a, tb);
  return hipGetLastError();
}

hipError_t launch_embed_grad(const EmbedGradArgs &a, bool x_bf16, bool g_bf16, hipStream_t s) {
  const Tables tb = tables_of(a.T, a.dlevel ? a.L : 0, a.K, a.dtext ? a.V : 0);
  if (tb.rows == 0) return hipSuccess;
  const int64_t units = (int64_t)tb.L * ceil_div(tb.K, kRange) + ceil_div(tb.V, kRange);
  embed_index_kernel<<<dim3((unsigned)units), kIndexThreads, 0, s>>>(a, tb);
  if (x_bf16)
    return g_bf16 ? launch_sums<uint16_t, uint16_t>(a, tb, s) : launch_sums<uint16_t, float>(a, tb, s);
  return g_bf16 ? launch_sums<float, uint16_t>(a, tb, s) : launch_sums<float, float>(a, tb, s);
}

}  // namespace rvq
