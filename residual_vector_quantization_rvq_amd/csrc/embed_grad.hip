// embed_grad.hip -- gradient of the unified token embedding (embed.hip).
//
//   dlevel[l][k] = sum of dout[t] over visual tokens t with ids[t][l] == k
//   dtext[v]     = sum of dout[t] over text tokens t with ids[t][0] == v
//
// No float atomics: every destination row is summed in token order (a long
// row in pieces, added in order), so the result depends on the inputs alone.
//
// embed_index_kernel lists, for each destination row, the tokens that add to
// it.  A workgroup owns kRange consecutive rows of one table and reads that
// table's column of the IDs twice: once to count (its rows, and the IDs below
// them, which is where its part of the table's list begins), once to place.
// Every wave has a piece of the tokens and a counter per row, so the lists
// come out in token order.  One launch and no scan over workgroups; its work
// grows with (rows / kRange) x T, a few per cent of the sums'.
//
// embed_sum_kernel sums each row's tokens.  Each table's part of the list is also
// cut in segments of equal length: a row with more tokens than a segment (a hot
// codeword, a padding token) is summed segment by segment, and embed_join_kernel
// adds the pieces in order.  Where a row is cut depends on its table's IDs alone,
// whichever other tables are asked for.
//
// What bounds it: every row of the tables is written once, and a visual
// token's row of dout is read once for each of its L levels.  Those reads miss
// the L2 (a row is back L levels later) and share the fabric with the writes.
// 39,731 tokens of 4096 bf16, 131,072 rows of fp32: 2.15 GB written and 2.29
// GB read in 681 us, 6.5 TB/s; dout read once would leave 370 us.  Tried and
// slower there: slabs of 64 to 512 bytes, one an XCD, that its L2 can hold
// (1.1 to 1.4 ms: eight to 32 lanes a row are bound by their control, and the
// stream of results evicts the slab).  Kernels of that call: by-table IDs 5
// us, index 29 us, sums 681 us, join 10 us.
#include "learn.h"

namespace rvq {

namespace {

constexpr int kRange = 512;        // destination rows of one index workgroup
constexpr int kBatch = 8;          // loads in flight: ID batches of a wave, rows of a sum
constexpr int kFlight = 4;         // rows of dout in flight while as many are added
constexpr int kShort = 256;        // tokens; see segment_length
// Columns of dout taken together: what the 256 MB Infinity Cache keeps beside
// the streams (39,731 x 4096 bf16, 325 MB: 776 us in one panel, 753 in panels
// of 160 MB, 747 of 100 MB, 749 of 60 MB).
constexpr int64_t kPanelBytes = (int64_t)100 << 20;
// Above it the IDs are laid out by table first, a launch of 4 to 5 us.  Index, and
// layout with index: 2,049 tokens of 8 levels 9.2 and 11.5 us, 3,000 11.4 and 11.5,
// 4,096 12.5 and 12.1; of 16 levels 2,049 15.3 and 14.7, 5,003 25.5 and 20.4.
constexpr int kKeysAbove = 3072;
// An index workgroup has sixteen waves, or four: where there are more than the
// 512 workgroups of sixteen that the device holds and up to kFewTokens tokens
// (514 workgroups: 4,096 tokens 14.7 us with sixteen waves and 13.1 with four, 5,003
// 16.0 and 15.3, 7,000 17.4 and 18.4; 256 workgroups: 39,731 tokens 29 and 71), and
// for the shortest sequences (256 tokens 6.2 and 5.8 us, 512 6.4 and 6.5).
constexpr int kFewTokens = 6144;
constexpr int kVeryFewTokens = 384;
// Up to so many of a wave's 64 IDs in the workgroup's rows are told apart one by
// one (about 8 instructions each), more of them bit by bit (80).  All bit by bit:
// 39,731 tokens of 8 levels of 8,192, four of 64 IDs, 37.6 us and not 29.2; all one
// by one: 600 tokens of levels of 256, all of them, 12.6 us and not 6.8.
constexpr int kFewHits = 12;
constexpr int kNone = INT32_MIN;   // not an ID of this table
constexpr int kThreads = 256;
constexpr int kMaxGroups = 1 << 22;

// Length of a segment of the list.  A row of at most this many tokens is
// summed by one wave in one go, at about 0.2 us a token (160 tokens of a row of
// 2324: 54 us with segments of 256, 26 us of 64); sequences of up to kShort
// tokens are spared the third launch.  About 2048 segments at most, as each is
// looked at whether or not a long row is in it.  By the IDs' shape, and not by the
// tables that are asked for: a row's sum is cut the same way for all of them.
int64_t segment_length(int64_t T, int L) {
  if (T <= kShort) return kShort;
  const int64_t h = round_up(ceil_div(T * (L + 1), 2048), 64);
  return h < 64 ? 64 : h;
}

// an ID of this table, kNone among them only as any other out-of-range ID
__device__ __forceinline__ int id_or_bad(int id) { return id == kNone ? -1 : id; }

// Which tables' gradients are wanted, and where their lists lie: T positions
// for each level, then T for the text table.
struct Tables {
  int L, K;        // L = 0: no level gradients
  int64_t V;       // 0: no text gradient
  int64_t T;
  int64_t rows, positions;
  int seg, parts, segments;  // segments: parts of each table, or none at all
  uint32_t per_parts;        // 2^32 / parts, rounded up
  bool keys;       // the IDs are laid out by table first
};

// L levels' tables and the text table of IDs of L_ids levels
Tables tables_of(int64_t T, int L_ids, int L, int K, int64_t V) {
  Tables t;
  t.L = L;
  t.K = K;
  t.V = V;
  t.T = T;
  t.rows = (int64_t)L * K + V;
  const int tables = L + (V > 0 ? 1 : 0);
  t.positions = tables * T;
  t.seg = (int)segment_length(T, L_ids);
  t.parts = (int)ceil_div(T, t.seg);
  // a row has at most T tokens: none is long if T is not
  t.segments = T > t.seg ? tables * t.parts : 0;
  t.per_parts = t.segments ? (uint32_t)ceil_div((int64_t)1 << 32, t.parts) : 0;
  // the layout is a launch of its own, which short sequences do not win back
  t.keys = T > kKeysAbove;
  return t;
}

}  // namespace

// The IDs by table: keys[l][t] is token t's ID in table l (L: the text table),
// kNone where the token is of the other kind.  The index workgroups read a
// table's IDs many times over; out of ids [T][L] each such load would touch L
// times the lines.
__global__ __launch_bounds__(kThreads) void embed_keys_kernel(EmbedGradArgs a, Tables tb) {
  const int64_t t = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (t >= tb.T) return;
  const bool visual = a.is_visual == nullptr || a.is_visual[t] != 0;
  const int32_t *id = a.ids + t * a.L;
  for (int l = 0; l < tb.L; ++l) a.keys[l * tb.T + t] = visual ? id_or_bad(id[l]) : kNone;
  if (tb.V > 0) a.keys[tb.L * tb.T + t] = visual ? kNone : id_or_bad(id[0]);
}

template <int NW>  // waves of a workgroup
__global__ __launch_bounds__(NW * 64) void embed_index_kernel(EmbedGradArgs a, Tables tb) {
  constexpr int kIndexWaves = NW, kIndexThreads = NW * 64;
  __shared__ int cnt[kIndexWaves][kRange];
  __shared__ int sums[kRange / 64];
  __shared__ int below_sum;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // this workgroup's rows [r0, r1) of its table
  const int per_level = (int)ceil_div(tb.K, kRange);
  const bool text = (int64_t)blockIdx.x >= (int64_t)tb.L * per_level;
  const int l = text ? 0 : blockIdx.x / per_level;
  const int range = text ? (int)(blockIdx.x - (int64_t)tb.L * per_level) : blockIdx.x % per_level;
  const int limit = (int)(text ? tb.V : tb.K);
  const int r0 = range * kRange;
  const int r1 = r0 + kRange < limit ? r0 + kRange : limit;
  const int64_t region = text ? tb.L * tb.T : l * tb.T;
  const int64_t row0 = (text ? (int64_t)tb.L * tb.K : (int64_t)l * tb.K) + r0;

  for (int i = threadIdx.x; i < kIndexWaves * kRange; i += kIndexThreads) (&cnt[0][0])[i] = 0;
  if (threadIdx.x == 0) below_sum = 0;
  __syncthreads();

  // 32-bit token numbers and byte offsets (T (L + 1) <= 2^30, checked on the
  // host): the loops below are bound by their instructions
  const int T = (int)tb.T;
  const int piece = (int)round_up(ceil_div(tb.T, kIndexWaves), 64);
  const int t0 = wave * piece < T ? wave * piece : T;
  const int t1 = t0 + piece < T ? t0 + piece : T;
  const uint32_t u0 = (uint32_t)r0, rows = (uint32_t)(r1 - r0);
  const int32_t *keys = a.keys + region;
  // IDs of kBatch x 64 tokens in this table; kNone for a token of the other kind
  int id[kBatch];
  const auto load_ids = [&](int tw) {
    if (tb.keys && tw + kBatch * 64 <= t1) {
#pragma unroll
      for (int u = 0; u < kBatch; ++u) id[u] = keys[(uint32_t)(tw + u * 64 + lane)];
    } else if (tb.keys) {
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int t = tw + u * 64 + lane;
        id[u] = t < t1 ? keys[(uint32_t)t] : kNone;
      }
    } else {
      bool mine[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int t = tw + u * 64 + lane;
        id[u] = t < t1 ? a.ids[(uint32_t)t * (uint32_t)a.L + (uint32_t)l] : 0;
        mine[u] = t < t1 && (a.is_visual == nullptr || a.is_visual[t] != 0) != text;
      }
#pragma unroll
      for (int u = 0; u < kBatch; ++u) id[u] = mine[u] ? id_or_bad(id[u]) : kNone;
    }
  };

  int below = 0, bad = 0;
  for (int tw = t0; tw < t1; tw += kBatch * 64) {
    load_ids(tw);
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      below += (uint32_t)id[u] < u0;
      const uint32_t k = (uint32_t)id[u] - u0;
      if (k < rows) atomicAdd(&cnt[wave][k], 1);
    }
    if (range == 0) {
#pragma unroll
      for (int u = 0; u < kBatch; ++u) bad += (uint32_t)id[u] >= (uint32_t)limit && id[u] != kNone;
    }
  }
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) {
    below += __shfl_xor(below, off, 64);
    bad += __shfl_xor(bad, off, 64);
  }
  if (lane == 0) {
    if (below) atomicAdd(&below_sum, below);
    if (bad && a.bad) atomicAdd(a.bad, (uint32_t)bad);
  }
  __syncthreads();

  // RP rows a thread: a row's waves' tokens in turn, the rows one after the other
  constexpr int RP = kRange / kIndexThreads > 1 ? kRange / kIndexThreads : 1;
  const int r = threadIdx.x * RP;
  int mine[RP], all = 0, incl = 0;
  if (r < kRange) {
#pragma unroll
    for (int j = 0; j < RP; ++j) {
      mine[j] = 0;
#pragma unroll
      for (int w = 0; w < kIndexWaves; ++w) mine[j] += cnt[w][r + j];
      all += mine[j];
    }
    incl = all;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const int v = __shfl_up(incl, off, 64);
      if (lane >= off) incl += v;
    }
    if (lane == 63) sums[wave] = incl;
  }
  __syncthreads();
  constexpr int kSums = kRange / RP / 64;
  int total = (int)region + below_sum;
#pragma unroll
  for (int w = 0; w < kSums; ++w) total += sums[w];
  if (r < kRange) {
    int at = (int)region + below_sum + incl - all;
    for (int w = 0; w < wave; ++w) at += sums[w];
#pragma unroll
    for (int j = 0; j < RP; ++j) {
      if (r0 + r + j < r1) {
        a.place[row0 + r + j] = make_int2(at, mine[j]);
      }
#pragma unroll
      for (int w = 0; w < kIndexWaves; ++w) {
        const int c = cnt[w][r + j];
        cnt[w][r + j] = at;
        at += c;
      }
    }
  }
  __syncthreads();
  // the table's last workgroup marks the positions that no token has
  if (r1 == limit)
    for (int64_t i = total + (int64_t)threadIdx.x; i < region + tb.T; i += kIndexThreads) a.row[i] = -1;

  for (int tw = t0; tw < t1; tw += kBatch * 64) {
    load_ids(tw);
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const uint32_t k = (uint32_t)id[u] - u0;
      const bool hit = k < rows;
      const unsigned long long hits = __ballot(hit);
      if (hits == 0) continue;
      unsigned long long same = 0;  // lanes of the same row
      if (__popcll(hits) <= kFewHits) {  // row by row
        for (unsigned long long rest = hits; rest;) {
          const uint32_t of = (uint32_t)__builtin_amdgcn_readlane((int)k, __ffsll((long long)rest) - 1);
          const unsigned long long m = __ballot(k == of);  // of is below rows: a hit
          if (k == of) same = m;
          rest &= ~m;
        }
      } else {  // bit by bit
        same = hits;
#pragma unroll
        for (int b = 0; (1 << b) < kRange; ++b) {
          const unsigned long long m = __ballot((k >> b) & 1);
          same &= ((k >> b) & 1) ? m : ~m;
        }
      }
      const int first = hit ? __ffsll((long long)same) - 1 : lane;
      int at = 0;
      if (hit && lane == first) at = atomicAdd(&cnt[wave][k], __popcll(same));
      at = __shfl(at, first, 64);
      if (hit) {
        at += __popcll(same & ((1ull << lane) - 1));
        a.token[at] = tw + u * 64 + lane;
        a.row[at] = (int)row0 + (int)k;
      }
    }
  }
}

namespace {

// A lane's 16 bytes of a slab of W lanes: where they are read, and which of
// their elements are the lane's to write.  Where the gradients are wider than
// dout, the lane has 8 bytes in either half of the slab, so that its stores of
// 16 bytes still join into whole lines (fp32 rows out of bf16 stored 32 bytes
// a lane went out at half the rate).  A row that ends inside a part is read
// from the part's length before its end on, so that every load is whole; rows
// narrower than a part (TINY) are read by elements.
template <typename T, typename G, int W, bool TINY>
struct Piece {
  static constexpr int N = kPiece<T>, H = sizeof(G) > sizeof(T) ? 2 : 1, M = N / H;
  int at[H];                  // first element read
  int8_t first[H], last[H];   // elements [first, last) of the part are written

  __device__ __forceinline__ Piece(int slab, int lane, int D) {
#pragma unroll
    for (int h = 0; h < H; ++h) {
      const int c = slab * W * N + (h * W + lane) * M, left = D - c;
      const int from = TINY || left >= M ? c : D - M;
      at[h] = left > 0 ? from : 0;
      first[h] = (int8_t)(left > 0 ? c - from : 0);
      last[h] = (int8_t)(left <= 0 ? 0 : TINY && left < M ? left : M);
    }
  }
  __device__ __forceinline__ u32x4 load(const T *row) const {
    u32x4 q = {0, 0, 0, 0};
    if constexpr (TINY) {
#pragma unroll
      for (int h = 0; h < H; ++h)
        for (int j = 0; j < last[h]; ++j) {
          if constexpr (sizeof(T) == 4)
            q[j] = __float_as_uint(row[at[h] + j]);
          else
            q[(h * M + j) / 2] |= (uint32_t)row[at[h] + j] << (16 * (j & 1));
        }
    } else if constexpr (H == 1) {
      q = load16((const T *)((const char *)row + (uint32_t)at[0] * (uint32_t)sizeof(T)));
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const u32x2 w = *(const u32x2_at2 *)((const char *)row + (uint32_t)at[h] * (uint32_t)sizeof(T));
        q[2 * h] = w[0];
        q[2 * h + 1] = w[1];
      }
    }
    return q;
  }
  template <typename O>
  __device__ __forceinline__ void store(O *row, const float (&s)[N], bool accumulate) const {
#pragma unroll
    for (int h = 0; h < H; ++h) {
      O *o = row + at[h];
      float v[M];
#pragma unroll
      for (int j = 0; j < M; ++j) v[j] = s[h * M + j];
      if (first[h] == 0 && last[h] == M) {
        if (accumulate) {
          float w[M];
          load_n<M>(o, M, w);
#pragma unroll
          for (int j = 0; j < M; ++j) v[j] += w[j];
        }
        stream_n<M>(o, v);
      } else {
#pragma unroll
        for (int j = 0; j < M; ++j)
          if (j >= first[h] && j < last[h]) store_f32(o, j, accumulate ? v[j] + load_f32(o, j) : v[j]);
      }
    }
  }
};

// positions [p0, p1) of segment s, of which there are too few for the rounding of
// per_parts to matter (segments x parts < 2^32)
__device__ __forceinline__ void segment_at(const Tables &tb, int s, int &p0, int &p1) {
  const int table = (int)__umulhi((uint32_t)s, tb.per_parts), from = (s - table * tb.parts) * tb.seg;
  const int T = (int)tb.T, begin = table * T;
  p0 = begin + from;
  p1 = begin + (from + tb.seg < T ? from + tb.seg : T);
}

template <typename G>
__device__ __forceinline__ G *row_of(const EmbedGradArgs &a, const Tables &tb, int64_t row) {
  const int64_t levels = (int64_t)tb.L * tb.K;
  return row < levels ? (G *)a.dlevel + row * a.D : (G *)a.dtext + (row - levels) * a.D;
}

}  // namespace

// W lanes sum W x N columns (a slab) of R consecutive rows of one table,
// R <= W.  Their tokens follow one another in the list, so the wave runs
// through the list: kFlight rows of dout are loaded while the kFlight before
// them are added, and a row is stored when its last token has been.  Lane j
// holds row j's place in the list and the tokens of W positions, so that the
// only loads that are waited for are those of dout.
// The first 2 x segments units are pieces of long rows: of a segment, the row
// that holds its first position (part[2 s]), and the row that begins inside
// it (part[2 s + 1]).
template <typename T, typename G, int W, bool TINY>
__global__ __launch_bounds__(kThreads) void embed_sum_kernel(EmbedGradArgs a, Tables tb, int R,
                                                             int slabs, int panel) {
  constexpr int N = kPiece<T>;
  const int lane = threadIdx.x % W;
  // lane j's value, j the same for the W lanes
  const auto from = [](int v, int j) {
    if constexpr (W == 64)
      return __builtin_amdgcn_readlane(v, j);
    else
      return __shfl(v, j, W);
  };
  const int level_groups = (int)ceil_div(tb.K, R);
  const int64_t groups = (int64_t)tb.L * level_groups + ceil_div(tb.V, R);
  const int64_t units = 2 * tb.segments + groups;
  int64_t v = (int64_t)blockIdx.x * (kThreads / W) + threadIdx.x / W;
  if constexpr (W == 64)  // the same for the wave
    v = (int64_t)blockIdx.x * (kThreads / W) + __builtin_amdgcn_readfirstlane(threadIdx.x / W);
  for (; v < units * slabs; v += (int64_t)gridDim.x * (kThreads / W)) {
    // panel by panel of the slabs; in a panel a row group's slabs in turn
    const int64_t at = v / (units * panel) * panel;
    const int wide = slabs - at < panel ? (int)(slabs - at) : panel;
    const int64_t u = (v - at * units) / wide;
    const int slab = (int)(at + (v - at * units) - u * wide);
    const Piece<T, G, W, TINY> piece(slab, lane, a.D);
    float s[N];
    int counts = 0, starts = 0, rows = 1;
    G *o = nullptr;         // the row that is being summed
    float *part = nullptr;  // instead of it: a long row's piece
    if (u < 2 * tb.segments) {
      int p0, p1;
      segment_at(tb, (int)(u >> 1), p0, p1);
      const int ra = a.row[p0], row = u & 1 ? a.row[p1 - 1] : ra;
      if (row < 0 || (u & 1 && row == ra) || a.place[row].y <= tb.seg) continue;
      const int b = a.place[row].x, e = b + a.place[row].y;
      starts = b > p0 ? b : p0;
      counts = (e < p1 ? e : p1) - starts;
      part = a.part + u * a.D;
    } else {
      // rows row0 .. row0 + rows - 1, of one table
      const int64_t g = u - 2 * tb.segments;
      const bool text = g >= (int64_t)tb.L * level_groups;
      const int l = text ? tb.L : (int)(g / level_groups);
      const int64_t r0 = (text ? g - (int64_t)tb.L * level_groups : g - (int64_t)l * level_groups) * R;
      const int64_t limit = text ? tb.V : tb.K;
      rows = (int)(limit - r0 < R ? limit - r0 : R);
      const int64_t row0 = (int64_t)l * tb.K + r0;
      if (lane < rows) {
        const int2 at = a.place[row0 + lane];
        starts = at.x;
        counts = at.y;
      }
      o = row_of<G>(a, tb, row0);
    }
    const auto store = [&](int n) {
      if (part)
        piece.store(part, s, false);
      else if (!(a.accumulate && n == 0))
        piece.store(o, s, a.accumulate);
      o += a.D;
#pragma unroll
      for (int j = 0; j < N; ++j) s[j] = 0.f;
    };
#pragma unroll
    for (int j = 0; j < N; ++j) s[j] = 0.f;

    for (int i = 0; i < rows;) {
      // rows [i, k) are short; k is a long row, which is not this wave's, or the end
      int k = i;
      if (tb.segments)
        while (k < rows && from(counts, k) <= tb.seg) ++k;
      else
        k = rows;
      int e = 0, e1 = 0;
      if (k > i) {
        e = from(starts, i);
        e1 = from(starts, k - 1) + from(counts, k - 1);
      }
      int n = k > i ? from(counts, i) : 0, end = e + n;   // row i's
      int w0 = e, tokens = 0, next = 0;                   // positions [w0, w0 + W), and the W after them
      if (e < e1) {
        tokens = e + lane < e1 ? a.token[e + lane] : 0;
        next = e + W + lane < e1 ? a.token[e + W + lane] : 0;
      }
      u32x4 raw[2][kFlight];
      const auto load = [&](int p, u32x4(&q)[kFlight]) {  // positions p .. p + kFlight - 1 below e1
        if (p - w0 >= W) {                                // kFlight divides W and p - w0
          w0 += W;
          tokens = next;
          next = w0 + W + lane < e1 ? a.token[w0 + W + lane] : 0;
        }
#pragma unroll
        for (int j = 0; j < kFlight; ++j)
          if (p + j < e1)
            q[j] = piece.load((const T *)a.dout + (int64_t)from(tokens, p + j - w0) * a.D);
      };
      const auto add = [&](int p, const u32x4(&q)[kFlight]) {
#pragma unroll
        for (int j = 0; j < kFlight; ++j)
          if (p + j < e1) {
            while (p + j >= end) {  // the rows that end here
              store(n);
              n = from(counts, ++i);
              end += n;
            }
            float f[N];
            unpack(q[j], f);
#pragma unroll
            for (int m = 0; m < N; ++m) s[m] += f[m];
          }
      };
      if (e < e1) load(e, raw[0]);
      for (; e < e1; e += 2 * kFlight) {
        load(e + kFlight, raw[1]);
        add(e, raw[0]);
        load(e + 2 * kFlight, raw[0]);
        add(e + kFlight, raw[1]);
      }
      for (; i < k; ++i) {
        store(n);
        n = i + 1 < k ? from(counts, i + 1) : 0;
      }
      if (k < rows) o += a.D;
      i = k + 1;
    }
  }
}

// The long row that begins in segment s, if there is one: its pieces in order.
template <typename G>
__global__ __launch_bounds__(kThreads) void embed_join_kernel(EmbedGradArgs a, Tables tb) {
  const int64_t s = blockIdx.x;
  int p0, p1;
  segment_at(tb, (int)s, p0, p1);
  const int row = a.row[p1 - 1];
  if (row < 0 || a.place[row].y <= tb.seg || a.place[row].x < p0) return;
  const int end = a.place[row].x + a.place[row].y;
  const int64_t first = a.place[row].x == p0 ? 2 * s : 2 * s + 1;
  G *o = row_of<G>(a, tb, row);
  const int c = blockIdx.y * kThreads + threadIdx.x;
  if (c >= a.D) return;
  float v = a.part[first * a.D + c];
  int64_t q = s + 1;  // the segments of the row's table
  for (p1 = p0 + tb.seg; p1 < end; p1 += tb.seg, ++q) v += a.part[2 * q * a.D + c];
  if (a.accumulate) v += load_f32(o, c);
  store_f32(o, c, v);
}

EmbedGradLayout embed_grad_layout(int64_t T, int L_ids, int L, int K, int64_t V, int D) {
  const Tables tb = tables_of(T, L_ids, L, K, V);
  EmbedGradLayout w;
  w.place = 0;
  w.token = w.place + al256((size_t)tb.rows * sizeof(int2));
  w.row = w.token + al256((size_t)tb.positions * 4);
  w.part = w.row + al256((size_t)tb.positions * 4);
  w.keys = w.part + al256((size_t)tb.segments * 2 * D * sizeof(float));
  w.total = w.keys + al256(tb.keys ? (size_t)tb.positions * 4 : 0);
  if (w.total == 0) w.total = 256;
  return w;
}

template <typename T, typename G>
static hipError_t launch_sums(const EmbedGradArgs &a, const Tables &tb, hipStream_t s) {
  const int64_t pieces = ceil_div(a.D, kPiece<T>);
  // Rows a wave takes in turn: four to pay for looking its list up, where that
  // leaves 8192 waves (75 k rows of 384 bf16, all but 16 without a token: 24 us,
  // one row each 51 us), more of them only beyond 65536 x 4 waves' worth, so that
  // the last round of waves is short (263 k rows of 1280 in three slabs: 12 rows
  // 165 us, 24 rows 193, 48 rows 212).
#define RVQ_SUM(W, TINY)                                                                        \
  do {                                                                                      \
    const int64_t slabs = ceil_div(pieces, W);                                              \
    const int64_t panels = ceil_div(a.T * a.D * (int64_t)sizeof(T), kPanelBytes);           \
    const int64_t panel = panels > 1 ? ceil_div(slabs, panels) : slabs;                     \
    const int64_t waves = tb.rows * slabs / (64 / W), few = waves / 8192;                   \
    int64_t R = waves / 65536;                                                              \
    if (R < 4) R = few < 4 ? few : 4;                                                       \
    R = R < 1 ? 1 : R > W ? W : R;                                                          \
    const int64_t units = 2 * tb.segments + tb.L * ceil_div(tb.K, R) + ceil_div(tb.V, R);   \
    const int64_t groups = ceil_div(units * slabs, kThreads / W);                           \
    embed_sum_kernel<T, G, W, TINY><<<dim3((unsigned)(groups < kMaxGroups ? groups : kMaxGroups)), \
                                kThreads, 0, s>>>(a, tb, (int)R, (int)slabs, (int)panel);   \
  } while (0)
  if (a.D < kPiece<T>) RVQ_SUM(8, true); else if (pieces <= 8) RVQ_SUM(8, false);
  else if (pieces <= 16) RVQ_SUM(16, false); else if (pieces <= 32) RVQ_SUM(32, false);
  else RVQ_SUM(64, false);
#undef RVQ_SUM
  if (tb.segments) 
    embed_join_kernel<G><<<dim3((unsigned)tb.segments, (unsigned)ceil_div(a.D, kThreads)), kThreads, 0, s>>>(a, tb);
  return hipGetLastError();
}

hipError_t launch_embed_grad(const EmbedGradArgs &a, bool x_bf16, bool g_bf16, hipStream_t s) {
  const Tables tb = tables_of(a.T, a.L, a.dlevel ? a.L : 0, a.K, a.dtext ? a.V : 0);
  if (tb.rows == 0) return hipSuccess;
  const int64_t units = (int64_t)tb.L * ceil_div(tb.K, kRange) + ceil_div(tb.V, kRange);
  if (tb.keys) embed_keys_kernel<<<dim3((unsigned)ceil_div(a.T, kThreads)), kThreads, 0, s>>>(a, tb);
  if (a.T <= kVeryFewTokens || (a.T <= kFewTokens && units > 512))
    embed_index_kernel<4><<<dim3((unsigned)units), 256, 0, s>>>(a, tb);
  else
    embed_index_kernel<16><<<dim3((unsigned)units), 1024, 0, s>>>(a, tb);
  if (x_bf16)
    return g_bf16 ? launch_sums<uint16_t, uint16_t>(a, tb, s) : launch_sums<uint16_t, float>(a, tb, s);
  return g_bf16 ? launch_sums<float, uint16_t>(a, tb, s) : launch_sums<float, float>(a, tb, s);
}

}  // namespace rvq
