// What the attention kernels share: tiles of packed sequences, masks, the rows
// done again one by one, and the plan of the dk, dv kernels.
#pragma once

#include "attn_row.h"
#include "attn_tile.h"

namespace staple {

constexpr int kWaves = 4;   // of a workgroup, unless said otherwise
constexpr int kF32RowsLog2 = 5, kBf16RowsLog2 = 7;   // queries (keys) of a workgroup's tile: 32 in fp32, 128 in bf16

// A tile of 2^rows_log2 consecutive rows of one sequence.  Sequence b owns the
// slots floor(cu[b] / rows) + b onwards, at least as many as it has tiles, so a
// grid of total / rows + n_seqs slots holds every sequence and a workgroup
// finds its own by a search of cu alone.
struct TileOf {
  int64_t seq, first;   // first: the tile's first row within the sequence; seq -1: none
};
__device__ __forceinline__ TileOf tile_of_slot(const int32_t* cu, int64_t n_seqs, int rows_log2, int64_t slot) {
  int64_t lo = 0, hi = n_seqs;   // slots of lo start at or before `slot`, those of hi after
  while (hi - lo > 1) {
    const int64_t mid = (lo + hi) >> 1;
    if ((cu[mid] >> rows_log2) + mid <= slot) lo = mid;
    else hi = mid;
  }
  const int64_t tile = slot - ((cu[lo] >> rows_log2) + lo);
  return TileOf{tile < 0 ? -1 : lo, tile << rows_log2};
}
// The same of one slot by a whole wave, which looks at 64 sequences at once.
__device__ __forceinline__ TileOf tile_of_slot_wave(const int32_t* cu, int n_seqs, int rows_log2, int slot) {
  const int lane = threadIdx.x & 63;
  int lo = 0, n = n_seqs, start;   // the last of [lo, lo + n) that starts at or before `slot`
  do {
    const int stride = (n + 63) >> 6;
    const int at = lane * stride, mid = lo + min(at, n - 1);
    start = (cu[mid] >> rows_log2) + mid;
    // lane 0's counts as before
    const uint64_t before = __ballot(at < n && start <= slot) | 1;
    const int last = 63 - __builtin_clzll(before);
    start = __shfl(start, last);
    lo += last * stride;
    n = min(stride, n - last * stride);
  } while (n > 1);
  lo = __builtin_amdgcn_readfirstlane(lo);
  const int tile = slot - __builtin_amdgcn_readfirstlane(start);
  return TileOf{tile < 0 ? -1 : lo, static_cast<int64_t>(tile) << rows_log2};
}
inline int64_t tile_slots(int64_t total, int64_t n_seqs, int rows_log2) { return (total >> rows_log2) + n_seqs; }

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ int wave_id() { return uniform(threadIdx.x >> 6); }

// One sequence and head, and the workgroup's tile of its queries or keys.
struct Segment {
  int64_t q0, k0;          // first rows
  int nq, nk, past;        // lengths, and the position of query 0
  int first;               // the tile's first query (key)
  // False where there is no such tile.  find_lane: any slot a lane; find: one
  // slot for the whole workgroup, kept in scalar registers.
  __device__ __forceinline__ bool find_lane(const AttnView& a, const int32_t* cu, int rows_log2, int64_t slot, int* err) {
    return take(a, cu, tile_of_slot(cu, a.n_seqs, rows_log2, slot), err);
  }
  __device__ __forceinline__ bool take(const AttnView& a, const int32_t* cu, TileOf tile, int* err) {
    if (tile.seq < 0) return false;
    int64_t q1, k1;
    seq_rows(a.cu_q, tile.seq, a.total_q, &q0, &q1, err);
    seq_rows(a.cu_k, tile.seq, a.total_k, &k0, &k1, err);
    if (tile.first >= (cu == a.cu_q ? q1 - q0 : k1 - k0)) return false;
    nq = static_cast<int>(q1 - q0);
    nk = static_cast<int>(k1 - k0);
    past = nk - nq;
    first = static_cast<int>(tile.first);
    return true;
  }
  __device__ __forceinline__ bool find(const AttnView& a, const int32_t* cu, int rows_log2, int slot, int* err) {
    if (!take(a, cu, tile_of_slot_wave(cu, static_cast<int>(a.n_seqs), rows_log2, slot), err)) return false;
    nq = uniform(nq);
    nk = uniform(nk);
    past = nk - nq;
    first = uniform(first);
    q0 = uniform(static_cast<int>(q0));
    k0 = uniform(static_cast<int>(k0));
    return true;
  }
};

// ---------------------------------------------------------------------- masks
// Applied with selects (a few integer compares an element), never by branching
// on one element of a result.

// Which keys of a block the lane's query (at position p) sees: key j = 8 (r /
// 4) + r % 4 (+ 4 for the upper half-wave) of the block at `key` is seen when
// j <= hi and (j >= lo or j < sink).
struct SeenKeys {
  int hi, lo, sink;
  __device__ __forceinline__ SeenKeys(const AttnView& a, int p, bool in, int key) {
    const int at = key + 4 * static_cast<int>((threadIdx.x & 63) >> 5);
    hi = in ? p - at : -1;
    lo = a.window > 0 ? p - a.window + 1 - at : -kMaxTokens;
    sink = a.sinks - at;
  }
  __device__ __forceinline__ bool operator()(int r) const {
    const int j = 8 * (r >> 2) + (r & 3);
    return (j <= hi) & ((j >= lo) | (j < sink));
  }
};
// Which queries of a block (the first is number i0 of the sequence) see the
// lane's key.
struct SeenBy {
  int lo, hi;
  __device__ __forceinline__ SeenBy(const AttnView& a, const Segment& s, int key, bool in, int i0) {
    const int at = i0 + 4 * static_cast<int>((threadIdx.x & 63) >> 5);
    lo = key - s.past - at;
    int end = s.nq;
    if (a.window > 0 && key >= a.sinks) end = min(end, key - s.past + a.window);
    hi = in ? end - at : -1;
  }
  __device__ __forceinline__ bool operator()(int r) const {
    const int j = 8 * (r >> 2) + (r & 3);
    return (j >= lo) & (j < hi);
  }
};

// True where a value is NaN or infinite.
__device__ __forceinline__ bool not_finite(float x) { return !(fabsf(x) < INFINITY); }

// Blocks of a part of a tile's keys, at least.  256 queries after 2000 keys, 8
// heads of 64, take 31 us in parts of 8; 37 of 4, 33 of 16; 8 x 16 queries
// after 600 keys 33; 33, 40.
constexpr int kMinShare = 8;

// The 32-key blocks that some query at a position in [p_min, p_max] sees: those
// of the sinks, then the window's; and which of them every query of the wave's
// range sees whole.
struct KeyBlocks {
  int n_sink, lo, n;
  int nk, skip = 0;
  int whole_sink, whole_lo, whole_n;
  __device__ __forceinline__ KeyBlocks(const AttnView& a, int n_keys, int p_min, int p_max) : nk(n_keys) {
    lo = (a.window > 0 ? max(p_min - a.window + 1, 0) : 0) / 32;
    n_sink = p_max < 0 ? 0 : (min(a.sinks, lo * 32) + 31) / 32;
    n = p_max < 0 ? 0 : n_sink + p_max / 32 + 1 - lo;
    whole_sink = whole_n = 0;
  }
  // The wave's own queries: positions [p_min, p_max], all 32 of them there.
  __device__ __forceinline__ void set_wave(const AttnView& a, int p_min, int p_max, bool full) {
    const int end = full ? max(p_min + 1, 0) / 32 : 0;               // blocks that end at or before p_min
    const int from = a.window > 0 ? (max(p_max - a.window + 1, 0) + 31) / 32 : 0;
    // numbered as first() numbers them; the sinks' whole blocks come first
    whole_sink = min(min(a.sinks / 32, n_sink), end);
    whole_lo = n_sink + max(from - lo, 0);
    whole_n = max(n_sink + end - lo - whole_lo, 0);
  }
  __device__ __forceinline__ bool whole(int b) const {
    return b < whole_sink || static_cast<unsigned>(b - whole_lo) < static_cast<unsigned>(whole_n);
  }
  // Keeps share `part` of at most `parts`, of kMinShare blocks at least; returns
  // how many there are.
  __device__ __forceinline__ int share(int parts, int part) {
    const int chunk = max((n + parts - 1) / parts, kMinShare);
    const int shares = max((n + chunk - 1) / chunk, 1);
    skip = min(part * chunk, n);
    n = min(chunk, n - skip);
    n_sink -= skip;
    whole_sink = min(whole_sink - skip, n);
    whole_lo -= skip;
    whole_n = max(min(whole_n, n - whole_lo), 0);
    return shares;
  }
  // First key of block b; blocks past the last lie past the keys.
  __device__ __forceinline__ int first(int b) const { return b < n ? (b < n_sink ? b + skip : lo + b - n_sink) * 32 : nk; }
};

// The wave's 32 queries, one a column.
struct QueryCols : Segment {
  int head, hk;
  int wq, row, p;             // the wave's first query; the lane's, and its position
  bool in;
  int tile_rows;
  // group_of_wave: which 32 queries of the workgroup's tile the wave has.
  __device__ __forceinline__ bool find(const AttnView& a, int rows_log2, int64_t n_slots, int id, int group_of_wave, int* err) {
    // the last tiles of a sequence see the most keys: they start first
    const int back = id / static_cast<int>(a.n_heads);
    if (!Segment::find(a, a.cu_q, rows_log2, static_cast<int>(n_slots) - 1 - back, err)) return false;
    tile_rows = 1 << rows_log2;
    head = uniform(id - back * static_cast<int>(a.n_heads));
    hk = uniform(head / static_cast<int>(a.group));
    wq = first + 32 * group_of_wave;
    row = wq + (threadIdx.x & 31);
    in = row < nq;
    p = past + row;
    return true;
  }
  __device__ __forceinline__ KeyBlocks blocks(const AttnView& a) const {
    KeyBlocks b(a, nk, past + first, past + min(first + tile_rows, nq) - 1);
    b.set_wave(a, past + wq, past + wq + 31, wq + 31 < nq);
    return b;
  }
};

// One side of the scores takes the scale's sign: scores in powers of two are
// then score_factor() times the products, and as that is positive the largest
// product has the largest score and a hidden one can be -inf before scaling.
template <typename T>
__device__ __forceinline__ u32x4_t signed_frag(const AttnView& a, u32x4_t v) {
  if (a.scale < 0.0f) v = flip_sign<T>(v);
  return a.scale == 0.0f ? u32x4_t{0, 0, 0, 0} : v;
}
__device__ __forceinline__ float score_factor(const AttnView& a) {
  return a.scale == 0.0f ? 1.0f : fabsf(a.scale) * kLog2e;
}
template <typename T, int DP>
__device__ __forceinline__ float load_queries(const AttnView& a, const QueryCols& w, u32x4_t* qf) {
#pragma unroll
  for (int s = 0; s < Tile<T, DP>::kSteps; ++s)
    qf[s] = signed_frag<T>(a, load_frag<T>(a.q, w.q0 + w.row, w.head, a.head_dim, s, w.in));
  return score_factor(a);
}

// ------------------------------------------------------------------- forward
// One query row, by a whole wave (row t of q, at position p of the sequence
// whose keys start at row k0).
template <typename T>
__device__ __forceinline__ void attn_fwd_row(const AttnView& a, int64_t t, int64_t h, int64_t p, int64_t k0) {
  const int64_t hk = h / a.group;
  int64_t sink_end, lo;
  visible_keys(p, a.window, a.sinks, &sink_end, &lo);
  const Row2 q = load_row<T>(a.q, t, h, a.head_dim);
  RowSoftmax sm;
  for (int64_t j = 0; j <= p; ++j) {
    if (j == sink_end) j = lo;
    if (j > p) break;
    const Row2 k = load_row<T>(a.k, k0 + j, hk, a.head_dim);
    sm.add(dot(q, k) * a.scale, load_row<T>(a.v, k0 + j, hk, a.head_dim));
  }
  store_row<T>(a.o, t, h, a.head_dim, sm.value());
}

// Running softmax of the lane's column: the sums stay relative to `top`, the
// largest score of the first block that held one, until a score passes it by 8.
// Then it rises by an integer: the exponentials stay below 2^9, far from fp32's
// range, lanes exchange maxima only then, and what has been summed is scaled by
// a power of two, exactly.  A query that sees one key has the weight 1, which a
// rounding to bf16 leaves as it is: its o is that key's value.
struct ColumnSoftmax {
  float top = -INFINITY, sum = 0.0f;   // sum: this half-wave's keys
  // s: the block's products, c times which are the scores.  True where `keep`
  // has to scale the sums.
  __device__ __forceinline__ bool raise(const f32x16_t& s, float c, float* keep) {
    float m = s[0];
#pragma unroll
    for (int r = 1; r < 16; ++r) m = fmaxf(m, s[r]);
    m *= c;
    if (!__any((m > top + 8.0f) | ((top == -INFINITY) & (m > top)))) return false;
    m = fmaxf(m, other_half(m));
    const bool first = top == -INFINITY;
    const float up = fmaxf(ceilf(m - top), 0.0f);
    *keep = first ? 0.0f : __builtin_amdgcn_exp2f(-up);
    top = first ? m : top + up;
    sum *= *keep;
    return true;
  }
  __device__ __forceinline__ float base() const { return top == -INFINITY ? 0.0f : top; }
};

// -inf for the hidden keys of the block at `key`.
__device__ __forceinline__ void mask_keys(const AttnView& a, const QueryCols& w, int key, f32x16_t& s) {
  const SeenKeys seen(a, w.p, w.in, key);
#pragma unroll
  for (int r = 0; r < 16; ++r) s[r] = seen(r) ? s[r] : -INFINITY;
}

// A NaN or an infinity in a result may have come from a row that the query does
// not see (its zero weight times it): such queries are done again key by key,
// a thousand times slower than the products.  A training step that has gone to
// NaN must not pay that in every row, so a NaN that the query's own row explains
// (its statistics, or the value at its own position, which it always sees) is
// left as it is.  4 x 1024 tokens, 8 heads on 2 of 128, with NaN in one element
// of every row of q, k, v or d_o take 44 + 123 us, as without; 21 + 156 ms with
// every such row done again.

// The columns that some lane marks, one a bit.
__device__ __forceinline__ uint32_t columns(bool bad) {
  const uint64_t b = __ballot(bad);
  return static_cast<uint32_t>(b) | static_cast<uint32_t>(b >> 32);
}
// What the n waves first, first + step, ... have marked; their results are
// stored by then.
__device__ __forceinline__ uint32_t join_marks(uint32_t mine, int first, int step, int n) {
  __shared__ uint32_t marks[8];
  if ((threadIdx.x & 63) == 0) marks[wave_id()] = mine;
  __syncthreads();
  uint32_t all = 0;
  for (int u = 0; u < n; ++u) all |= marks[first + u * step];
  return uniform(all);
}
// Does every n-th marked column again, from the turn-th on.
template <typename RowFn>
__device__ __forceinline__ void redo(uint32_t marked, int turn, int n, RowFn row) {
  for (int i = 0; marked; ++i, marked &= marked - 1)
    if (i % n == turn) row(__builtin_ctz(marked));
}

// Elements e .. e + 3 of a head's row.
template <typename T>
__device__ __forceinline__ f32x4_t load4(const HeadsView& t, int64_t row, int64_t head, int e) {
  const T* p = reinterpret_cast<const T*>(t.data) + row * t.row_stride + head * t.head_stride;
  return f32x4_t{Elem<T>::load(p, e), Elem<T>::load(p, e + 1), Elem<T>::load(p, e + 2), Elem<T>::load(p, e + 3)};
}
__device__ __forceinline__ bool is_nan(float x) { return x != x; }

// Whether every element of x (32 dims of the lane's query, as store_column has
// them) that is not finite is a NaN where the value at the query's own position
// is one.
template <typename T>
__device__ __forceinline__ bool own_value_explains(const AttnView& a, const QueryCols& w, int d, const f32x16_t& x) {
  bool fine = true;
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    const int e = d * 32 + 8 * g + 4 * static_cast<int>((threadIdx.x & 63) >> 5);
    if (e >= a.head_dim) continue;
    const f32x4_t v = load4<T>(a.v, w.k0 + w.p, w.hk, e);
#pragma unroll
    for (int i = 0; i < 4; ++i) fine &= !not_finite(x[4 * g + i]) | (is_nan(x[4 * g + i]) & is_nan(v[i]));
  }
  return fine;
}

// A tile's keys in parts, where there are too few tiles to occupy the GPU: each
// part is a workgroup of the forward (dq) and leaves its sums, the forward's
// relative to its own reference, and attn_join_kernel adds them in part order.
// Calls of bf16 and dim 128 measured in parts, and with a workgroup a tile:
//   16 queries after 14000 keys, 16 heads on 4: 57 us; 388 us
//   512 queries after 8000 keys, 16 heads on 4: 74 us; 178 us
//   2048 queries, 4 heads: 41 us; 56 us
//   8 sequences of 16 queries after 600 keys, 4 heads: 33 us; 36 us
//   backward of 4096 queries, 1 head: 90 us; 192 us
//   backward of 2048 queries, 4 heads: 95 us; 138 us
struct KeyParts {
  int n;         // at most so many of a tile
  f32x4_t* o;    // [tiles][heads][parts][32s of queries][32s of dims][4][64]: sums as they lie in a wave
  float* rows;   // [tiles][heads][parts][32s of queries][2][32]: reference and sum
  // unit: a part's number times the tile's 32s of queries, plus one of these
  __device__ __forceinline__ void put_rows(int64_t unit, float top, float sum) const {
    const int lane = threadIdx.x & 63;
    if (lane < 32) {
      rows[unit * 64 + lane] = top;
      rows[unit * 64 + 32 + lane] = sum;
    }
  }
  template <int kDT>
  __device__ __forceinline__ void put(int64_t unit, int d, const f32x16_t& x) const {
    f32x4_t* to = o + (unit * kDT + d) * 256 + (threadIdx.x & 63);
#pragma unroll
    for (int g = 0; g < 4; ++g) to[g * 64] = f32x4_t{x[4 * g], x[4 * g + 1], x[4 * g + 2], x[4 * g + 3]};
  }
};

// What a sum relative to `top` is worth relative to `all`, the largest.
__device__ __forceinline__ float rebase(float top, float sum, float all) {
  return top == -INFINITY && sum == 0.0f ? 0.0f : __builtin_amdgcn_exp2f(top - all);
}

// The end of 32 queries' forward, by the waves that have some of their dims
// each (every kWaves-th 32, kOut at most); `total`: the sum of the weights.
template <typename T, int DP, int kOut>
__device__ __forceinline__ void finish_dims(const AttnView& a, const QueryCols& w, int n_waves, float top, float total,
                                            const f32x16_t (&out)[kOut]) {
  const float inv = total == 0.0f ? 0.0f : 1.0f / total;
  bool bad = false;
#pragma unroll
  for (int i = 0; i < kOut; ++i) {
    const int d = i * n_waves + wave_id();
    if (d >= Tile<T, DP>::kDT) continue;
#pragma unroll
    for (int r = 0; r < 16; ++r) bad |= not_finite(out[i][r]);
    store_column<T>(a.o, w.q0 + w.row, w.head, a.head_dim, d, out[i], inv, w.in);
  }
  bad = bad && w.in && !is_nan(total);   // a NaN among the weights makes the row NaN
  if (bad && w.p >= 0) {
    bad = false;
#pragma unroll
    for (int i = 0; i < kOut; ++i) {
      const int d = i * n_waves + wave_id();
      if (d < Tile<T, DP>::kDT) bad |= !own_value_explains<T>(a, w, d, out[i]);
    }
  }
  if (wave_id() == 0 && w.in && (threadIdx.x & 63) < 32)
    a.lse[(w.q0 + w.row) * a.n_heads + w.head] = (top + __builtin_amdgcn_logf(total)) * kLn2;
  redo(join_marks(columns(bad), 0, 1, n_waves), wave_id(), n_waves,
       [&](int i) { attn_fwd_row<T>(a, w.q0 + w.wq + i, w.head, w.past + w.wq + i, w.k0); });
}

// ------------------------------------------------------------------ backward
// One query's row of dq, by a whole wave.  A NaN in its statistics makes the
// whole row NaN, if the query sees a key.
template <typename T>
__device__ __forceinline__ void attn_dq_row(const AttnView& a, int64_t t, int64_t h, int64_t p, int64_t k0) {
  const int64_t hk = h / a.group;
  int64_t sink_end, lo;
  visible_keys(p, a.window, a.sinks, &sink_end, &lo);
  const Row2 q = load_row<T>(a.q, t, h, a.head_dim), d_o = load_row<T>(a.d_o, t, h, a.head_dim);
  const float dl = dot(d_o, load_row<T>(a.o, t, h, a.head_dim)), lse = a.lse[t * a.n_heads + h];
  if (p >= 0 && (is_nan(dl) || is_nan(lse))) return store_row<T>(a.dq, t, h, a.head_dim, Row2{{NAN, NAN}});
  Row2 dq{{0.0f, 0.0f}};
  for (int64_t j = 0; j <= p; ++j) {
    if (j == sink_end) j = lo;
    if (j > p) break;
    const Row2 k = load_row<T>(a.k, k0 + j, hk, a.head_dim);
    const float pr = __expf(dot(q, k) * a.scale - lse);
    const float ds = pr * (dot(d_o, load_row<T>(a.v, k0 + j, hk, a.head_dim)) - dl);
    dq.x[0] += ds * k.x[0];
    dq.x[1] += ds * k.x[1];
  }
  dq.x[0] *= a.scale;
  dq.x[1] *= a.scale;
  store_row<T>(a.dq, t, h, a.head_dim, dq);
}

// The end of 32 queries' dq; see finish_dims.
template <typename T, int DP, int kOut>
__device__ __forceinline__ void finish_dq_dims(const AttnView& a, const QueryCols& w, int n_waves, const f32x16_t (&out)[kOut]) {
  bool bad = false;
#pragma unroll
  for (int i = 0; i < kOut; ++i) {
    const int d = i * n_waves + wave_id();
    if (d >= Tile<T, DP>::kDT) continue;
#pragma unroll
    for (int r = 0; r < 16; ++r) bad |= not_finite(out[i][r]);
    store_column<T>(a.dq, w.q0 + w.row, w.head, a.head_dim, d, out[i], a.scale, w.in);
  }
  redo(join_marks(columns(bad && w.in), 0, 1, n_waves), wave_id(), n_waves,
       [&](int i) { attn_dq_row<T>(a, w.q0 + w.wq + i, w.head, w.past + w.wq + i, w.k0); });
}

// 32 queries of a tile in parts a workgroup, 32 dims a wave.  kGrad: dq, whose
// parts need no weights.
template <typename T, int DP, bool kGrad>
__global__ __launch_bounds__(2 * DP) void attn_join_kernel(AttnView a, int rows_log2, int64_t n_slots, KeyParts parts, int* err) {
  constexpr int kDT = Tile<T, DP>::kDT;
  const int groups = 1 << (rows_log2 - 5), lane = threadIdx.x & 63;
  const int tile = static_cast<int>(blockIdx.x) / groups, group = static_cast<int>(blockIdx.x) - tile * groups;
  QueryCols w;
  if (!w.find(a, rows_log2, n_slots, tile, group, err) || w.wq >= w.nq) return;
  const int n = w.blocks(a).share(parts.n, 0);
  if (n == 1) return;   // stored already
  const int64_t unit = static_cast<int64_t>(tile) * parts.n * groups + group;
  const float* const tops = parts.rows + unit * 64 + (lane & 31);
  const f32x4_t* const from = parts.o + (unit * kDT + wave_id()) * 256 + lane;
  // a batch of parts at a time: what it costs is waiting for their loads
  constexpr int kBatch = 8;
  float top = -INFINITY, total = 0.0f;
  f32x16_t out[1] = {};
  for (int u0 = 0; u0 < n; u0 += kBatch) {
    float t[kBatch], sum[kBatch];
    f32x4_t v[kBatch][4];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int64_t u = static_cast<int64_t>(min(u0 + i, n - 1)) * groups;
      if constexpr (!kGrad) {
        t[i] = tops[u * 64];
        sum[i] = tops[u * 64 + 32];
      }
#pragma unroll
      for (int g = 0; g < 4; ++g) v[i][g] = from[u * kDT * 256 + g * 64];
    }
    if constexpr (!kGrad) {
      float all = top;
#pragma unroll
      for (int i = 0; i < kBatch; ++i) all = fmaxf(all, t[i]);
      const float keep = rebase(top, total, all);
      top = all;
      total *= keep;
      out[0] *= keep;
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      // past the last part: that one again, times zero
      float f = u0 + i < n ? 1.0f : 0.0f;
      if constexpr (!kGrad) {
        f *= rebase(t[i], sum[i], top);
        total += sum[i] * f;
      }
#pragma unroll
      for (int g = 0; g < 4; ++g)
#pragma unroll
        for (int e = 0; e < 4; ++e) out[0][4 * g + e] += v[i][g][e] * f;
    }
  }
  if constexpr (kGrad) finish_dq_dims<T, DP, 1>(a, w, kDT, out);
  else finish_dims<T, DP, 1>(a, w, kDT, top, total, out);
}

// One key's rows of dk and dv, by a whole wave.
template <typename T>
__device__ __forceinline__ void attn_dkv_row(const AttnView& a, const float* delta, int j, int hk, const Segment& s) {
  const Row2 k = load_row<T>(a.k, s.k0 + j, hk, a.head_dim), v = load_row<T>(a.v, s.k0 + j, hk, a.head_dim);
  Row2 dk{{0.0f, 0.0f}}, dv{{0.0f, 0.0f}};
  const int i0 = max(j - s.past, 0);
  const int i1 = a.window > 0 && j >= a.sinks ? min(j - s.past + a.window, s.nq) : s.nq;
  for (int64_t g = 0; g < a.group; ++g) {
    const int64_t h = static_cast<int64_t>(hk) * a.group + g;
    for (int64_t i = i0; i < i1; ++i) {
      const Row2 q = load_row<T>(a.q, s.q0 + i, h, a.head_dim);
      const Row2 d_o = load_row<T>(a.d_o, s.q0 + i, h, a.head_dim);
      const float pr = __expf(dot(q, k) * a.scale - a.lse[(s.q0 + i) * a.n_heads + h]);
      const float ds = pr * (dot(d_o, v) - delta[h * a.total_q + s.q0 + i]);
      dk.x[0] += ds * q.x[0];
      dk.x[1] += ds * q.x[1];
      dv.x[0] += pr * d_o.x[0];
      dv.x[1] += pr * d_o.x[1];
    }
  }
  dk.x[0] *= a.scale;
  dk.x[1] *= a.scale;
  store_row<T>(a.dk, s.k0 + j, hk, a.head_dim, dk);
  store_row<T>(a.dv, s.k0 + j, hk, a.head_dim, dv);
}

// What the backward needs of the forward: lse in powers of two (0 where no key
// is seen) and delta = sum d_o o, both [n_heads][total_q].
struct RowStats {
  float* lse2;
  float* delta;
};

// The 32-query blocks that see some key of a workgroup's tile: `per_head` of
// them, from block b_lo, for each head of the group.
struct QueryBlocks {
  int b_lo, per_head;
  __device__ __forceinline__ QueryBlocks(const AttnView& a, const Segment& w, int tile_rows) {
    const int last_key = min(w.first + tile_rows, w.nk) - 1;
    const int lo = max(w.first - w.past, 0);
    const int hi = a.window > 0 && w.first >= a.sinks ? min(last_key - w.past + a.window, w.nq) : w.nq;
    b_lo = lo / 32;
    per_head = hi > lo ? (hi + 31) / 32 - b_lo : 0;
  }
};

// How dk and dv are worked off.  Key tiles see very different numbers of
// queries (the first of a causal sequence all of them, a window's only its
// own, the sinks' all again), and a shared key-value head those of every head
// of its group.  A tile with more blocks than `chunk` is split into parts of
// equal size, whose fp32 sums go to the workspace and are added in part order
// by attn_dkv_join_kernel; and the items (tiles and parts) start in the order
// of their size, the largest first.  Written by one workgroup of the dq kernel,
// which runs before.
//
// Joined by the part that arrives last, every part pays a flush of its L2 to
// the device: the backward of 2048 queries of 4 heads took 153 us so and takes
// 95 with a kernel of its own, 4096 of one head 141 and 90.
struct __align__(16) DkvRecord {
  int32_t part, parts;          // of a tile's: which, and how many
  int32_t sums;                 // the tile's first partial result, where there are several parts
  int32_t q0, k0, nq, nk, first;   // its Segment
};
struct DkvPlan {
  int32_t* head;      // [0] items, [1] split tiles
  int32_t* blocks;    // [slots] blocks of the slot's tile
  DkvRecord* tiles;   // [slots]
  int32_t* split;     // [max_parts] slots of the split tiles
  DkvRecord* items;   // [slots + max_parts], one load for a workgroup to know its work
  f32x4_t* sums;      // [max_parts][n_kv_heads][32s of keys][dk, dv, 32s of dims][4][64]: as they lie in a wave
  int64_t n_slots;
  int max_parts;
  int target;         // parts per head to aim for
  int rows_log2;      // keys of a tile
};
// Blocks of a part, at least.  The backward of 2048 queries of 4 heads takes 95
// us; 108 with 8, 107 with 32.
constexpr int kMinChunk = 16;
constexpr int kBuckets = 64;

__device__ __forceinline__ int64_t group_sum(int64_t v, int64_t* lds) {
#pragma unroll
  for (int d = 32; d > 0; d /= 2) v += __shfl_xor(v, d);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  int64_t all = 0;
#pragma unroll
  for (int i = 0; i < kWaves; ++i) all += lds[i];
  return all;
}

__device__ __forceinline__ void plan_dkv(const AttnView& a, const DkvPlan& plan, int* err) {
  __shared__ int64_t sums[kWaves];
  __shared__ int count[kBuckets], start[kBuckets], n_parts, n_split;
  constexpr int kThreads = 64 * kWaves;
  const int n_slots = static_cast<int>(plan.n_slots);
  int64_t mine = 0;
  for (int s = threadIdx.x; s < n_slots; s += kThreads) {
    Segment w;
    int n = -1;   // no tile
    if (w.find_lane(a, a.cu_k, plan.rows_log2, s, err)) {
      n = QueryBlocks(a, w, 1 << plan.rows_log2).per_head * a.group;
      plan.tiles[s] = DkvRecord{0, 1, 0, static_cast<int>(w.q0), static_cast<int>(w.k0), w.nq, w.nk, w.first};
    }
    plan.blocks[s] = n;
    mine += max(n, 0);
  }
  const int64_t total = group_sum(mine, sums);
  const int64_t share = (total + plan.target - 1) / plan.target;
  const int chunk = static_cast<int>(share < kMinChunk ? kMinChunk : share);
  if (threadIdx.x < kBuckets) count[threadIdx.x] = 0;
  if (threadIdx.x == 0) n_parts = n_split = 0;
  __syncthreads();
  // an item has at most `chunk` blocks; bucket 0 holds the largest
  auto bucket = [&](int size) { return kBuckets - 1 - static_cast<int>(static_cast<int64_t>(size) * (kBuckets - 1) / chunk); };
  for (int s = threadIdx.x; s < n_slots; s += kThreads) {
    const int n = plan.blocks[s];
    if (n < 0) continue;
    const int parts = max((n + chunk - 1) / chunk, 1);
    if (parts > 1) {
      plan.tiles[s].parts = parts;
      plan.tiles[s].sums = atomicAdd(&n_parts, parts);
      plan.split[atomicAdd(&n_split, 1)] = s;
    }
    atomicAdd(&count[bucket((n + parts - 1) / parts)], parts);
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    int at = 0;
    for (int b = 0; b < kBuckets; ++b) {
      start[b] = at;
      at += count[b];
    }
    plan.head[0] = at;
    plan.head[1] = n_split;
  }
  __syncthreads();
  for (int s = threadIdx.x; s < n_slots; s += kThreads) {
    const int n = plan.blocks[s];
    if (n < 0) continue;
    DkvRecord r = plan.tiles[s];   // this thread wrote it
    int at = atomicAdd(&start[bucket((n + r.parts - 1) / r.parts)], r.parts);
    for (; r.part < r.parts; ++r.part, ++at) plan.items[at] = r;
  }
}

// dk and dv: one key a column; the queries that see them (of every head of the
// group) go through LDS.  An item is a key tile or a part of one.
struct DkvItem : Segment {
  int part, parts, sums, hk;
  int64_t h0;              // the head of the item's first block
  int n, ln;               // its blocks, and the first one's number within its head
  int b_lo, per_head;      // see QueryBlocks
  int wkey, key;           // the wave's first key; the lane's
  bool in;
  int whole_lo, whole_n;   // of a head's blocks, those whose every query sees all of the wave's keys
  int seen_lo, seen_hi;    // and those of which some query sees some of them: [seen_lo, seen_hi)
  // False where there is no such item; `group`: which 32 keys of the tile the wave has.
  __device__ __forceinline__ bool find(const AttnView& a, const DkvPlan& plan, int group_of_wave) {
    const int item = uniform(static_cast<int>(blockIdx.x) / a.n_kv_heads);
    const DkvRecord r = plan.items[item];
    if (item >= plan.head[0]) return false;
    hk = static_cast<int>(blockIdx.x) - item * a.n_kv_heads;
    take(r);
    wkey = first + 32 * group_of_wave;
    key = wkey + (threadIdx.x & 31);
    in = key < nk;
    const QueryBlocks blocks(a, *this, 1 << plan.rows_log2);
    b_lo = blocks.b_lo;
    per_head = blocks.per_head;
    const int all = per_head * a.group, chunk = uniform((all + parts - 1) / parts);
    const int from_block = min(part * chunk, all);
    n = min(chunk, all - from_block);
    const int skip = uniform(per_head > 0 ? from_block / per_head : 0);
    h0 = static_cast<int64_t>(hk) * a.group + skip;
    ln = from_block - skip * per_head;
    const bool sink = wkey < a.sinks, all_sinks = wkey + 31 < a.sinks;
    const int from = (max(wkey + 31 - past, 0) + 31) / 32;
    const int to = (a.window > 0 && !all_sinks ? min(max(wkey - past + a.window, 0), nq) : nq) / 32;
    whole_lo = from - b_lo;
    whole_n = wkey + 31 < nk ? max(to - from, 0) : 0;
    const int end = a.window > 0 && !sink ? min(max(wkey + 31 - past + a.window, 0), nq) : nq;
    seen_lo = max(wkey - past, 0) / 32 - b_lo;
    seen_hi = wkey < nk ? (end + 31) / 32 - b_lo : 0;
    return true;
  }
  __device__ __forceinline__ void take(const DkvRecord& r) {
    part = uniform(r.part);
    parts = uniform(r.parts);
    sums = uniform(r.sums);
    q0 = uniform(r.q0);
    k0 = uniform(r.k0);
    nq = uniform(r.nq);
    nk = uniform(r.nk);
    past = nk - nq;
    first = uniform(r.first);
  }
  __device__ __forceinline__ bool whole(int b) const {
    return static_cast<unsigned>(b - whole_lo) < static_cast<unsigned>(whole_n);
  }
};

// Where a part's sums of 32 keys lie, for the lane: kTiles results of a wave.
template <int kTiles>
__device__ __forceinline__ f32x4_t* part_sums(const DkvPlan& plan, int64_t part, int hk, int n_kv_heads, int group) {
  return plan.sums + ((((part * n_kv_heads + hk) << (plan.rows_log2 - 5)) + group) * kTiles) * 256 + (threadIdx.x & 63);
}
__device__ __forceinline__ void put_sums(f32x4_t* to, int tile, const f32x16_t& x) {
#pragma unroll
  for (int g = 0; g < 4; ++g) to[(tile * 4 + g) * 64] = f32x4_t{x[4 * g], x[4 * g + 1], x[4 * g + 2], x[4 * g + 3]};
}

// Keys whose gradients came out not finite: a query that does not see the key
// may have brought it (zero times its rows), so they are done again query by
// query, unless the query at the key's own position explains it; see the
// forward.  first, step, n: the waves that have these 32 keys; turn: which of
// them this one is.
template <typename T>
__device__ __forceinline__ void redo_keys(const AttnView& a, const RowStats& stats, const DkvItem& w, bool bad, int first, int step,
                                          int n, int turn) {
  redo(join_marks(columns(bad && w.in), first, step, n), turn, n,
       [&](int i) { attn_dkv_row<T>(a, stats.delta, w.wkey + i, w.hk, w); });
}
// Whether every element of x (32 dims of the lane's key's dk, or its dv) that is
// not finite is a NaN that the query at the key's position brings: a NaN in its
// statistics makes the whole row NaN (delta: of dk alone), one in its d_o that
// element of dv.
template <typename T>
__device__ __forceinline__ bool own_query_explains(const AttnView& a, const RowStats& stats, const DkvItem& w, bool value, int d,
                                                   const f32x16_t& x) {
  const int i = w.key - w.past;
  if (!w.in || i < 0) return false;
  uint32_t nan = 0;   // a bit an element
  for (int g = 0; g < a.group; ++g) {
    const int64_t h = static_cast<int64_t>(w.hk) * a.group + g, at = h * a.total_q + w.q0 + i;
    if (is_nan(stats.lse2[at]) || (!value && is_nan(stats.delta[at]))) nan = 0xffff;
    if (!value || nan == 0xffff) continue;
#pragma unroll
    for (int y = 0; y < 4; ++y) {
      const int e = d * 32 + 8 * y + 4 * static_cast<int>((threadIdx.x & 63) >> 5);
      if (e >= a.head_dim) continue;
      const f32x4_t v = load4<T>(a.d_o, w.q0 + i, h, e);
#pragma unroll
      for (int j = 0; j < 4; ++j) nan |= is_nan(v[j]) ? 1u << (4 * y + j) : 0u;
    }
  }
  bool fine = true;
#pragma unroll
  for (int r = 0; r < 16; ++r) fine &= !not_finite(x[r]) | (is_nan(x[r]) & ((nan >> r & 1) != 0));
  return fine;
}
// Whether x holds something not finite that a key's row has to be done again for.
template <typename T>
__device__ __forceinline__ bool has_unexplained(const AttnView& a, const RowStats& stats, const DkvItem& w, bool value, int d,
                                                const f32x16_t& x) {
  bool bad = false;
#pragma unroll
  for (int r = 0; r < 16; ++r) bad |= not_finite(x[r]);
  return bad && !own_query_explains<T>(a, stats, w, value, d, x);
}

// 32 keys of a split tile a workgroup, 32 dims of dk or dv a wave.
template <typename T, int DP>
__global__ __launch_bounds__(4 * DP) void attn_dkv_join_kernel(AttnView a, RowStats stats, DkvPlan plan) {
  constexpr int kDT = Tile<T, DP>::kDT, kTiles = 2 * kDT, kBatch = 8;
  const int groups = 1 << (plan.rows_log2 - 5);
  const int id = static_cast<int>(blockIdx.x) / groups, group = static_cast<int>(blockIdx.x) - id * groups;
  const int split = id / a.n_kv_heads;
  if (split >= plan.head[1]) return;
  DkvItem w;
  w.take(plan.tiles[uniform(plan.split[split])]);
  w.hk = id - split * a.n_kv_heads;
  w.wkey = w.first + 32 * group;
  w.key = w.wkey + (threadIdx.x & 31);
  w.in = w.key < w.nk;
  if (w.wkey >= w.nk) return;
  const int tile = wave_id();
  f32x16_t x = {};
  for (int u0 = 0; u0 < w.parts; u0 += kBatch) {
    f32x4_t v[kBatch][4];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const f32x4_t* from = part_sums<kTiles>(plan, w.sums + min(u0 + i, w.parts - 1), w.hk, a.n_kv_heads, group);
#pragma unroll
      for (int g = 0; g < 4; ++g) v[i][g] = from[(tile * 4 + g) * 64];
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const float f = u0 + i < w.parts ? 1.0f : 0.0f;   // past the last part: that one again, times zero
#pragma unroll
      for (int g = 0; g < 4; ++g)
#pragma unroll
        for (int e = 0; e < 4; ++e) x[4 * g + e] += v[i][g][e] * f;
    }
  }
  const bool value = tile >= kDT;
  const int d = value ? tile - kDT : tile;
  store_column<T>(value ? a.dv : a.dk, w.k0 + w.key, w.hk, a.head_dim, d, x, value ? 1.0f : a.scale, w.in);
  redo_keys<T>(a, stats, w, has_unexplained<T>(a, stats, w, value, d, x), 0, 1, kTiles, tile);
}

// ------------------------------------------------------------------- launches
// Raises a kernel's limit of dynamic LDS past the 64 KB that a launch gets
// unasked (once a kernel), then launches it.
template <auto kKernel, int kLds, int kThreads = 64 * kWaves, typename... Args>
inline hipError_t launch_lds(int64_t wgs, hipStream_t s, Args... args) {
  if (wgs == 0) return hipSuccess;
  static const hipError_t attr =
      hipFuncSetAttribute(reinterpret_cast<const void*>(kKernel), hipFuncAttributeMaxDynamicSharedMemorySize, kLds);
  if (attr != hipSuccess) return attr;
  kKernel<<<static_cast<unsigned>(wgs), kThreads, kLds, s>>>(args...);
  return hipGetLastError();
}

// How many parts a tile's keys are split into: as many as make two workgroups a
// CU, if there are keys for them.  The lengths are on the device; the longest
// sequence is taken to have up to four times the mean.
inline int key_parts(const AttnView& a, int rows_log2) {
  const int64_t wgs = tile_slots(a.total_q, a.n_seqs, rows_log2) * a.n_heads;
  if (wgs == 0) return 1;
  int64_t keys = a.n_seqs > 4 ? 4 * (a.total_k / a.n_seqs) : a.total_k;
  const int64_t window = a.window + (int64_t(1) << rows_log2) + a.sinks;
  if (a.window > 0 && window < keys) keys = window;
  int64_t parts = 2 * device_cus() / wgs;
  if (parts > keys / (32 * kMinShare)) parts = keys / (32 * kMinShare);
  return parts < 2 ? 1 : static_cast<int>(parts);
}
inline KeyParts take_parts(const AttnView& a, int rows_log2, Workspace& w) {
  KeyParts p{key_parts(a, rows_log2), nullptr, nullptr};
  if (p.n == 1) return p;
  const size_t units = static_cast<size_t>(tile_slots(a.total_q, a.n_seqs, rows_log2) * a.n_heads * p.n) << (rows_log2 - 5);
  p.o = w.take<f32x4_t>(units * (a.head_dim <= 64 ? 64 : 128) * 32 * sizeof(float));
  p.rows = w.take<float>(units * 64 * sizeof(float));
  return p;
}
template <typename T, int DP, bool kGrad>
inline hipError_t launch_join(const AttnView& a, int rows_log2, int64_t n_slots, const KeyParts& parts, hipStream_t s, int* err) {
  if (parts.n == 1) return hipSuccess;
  attn_join_kernel<T, DP, kGrad>
      <<<static_cast<unsigned>((n_slots * a.n_heads) << (rows_log2 - 5)), 2 * DP, 0, s>>>(a, rows_log2, n_slots, parts, err);
  return hipGetLastError();
}

// Whether a head's rows may span 2^31 bytes.
inline bool spans_buffer(const HeadsView& t, int64_t rows, int elem_bytes) {
  return t.row_stride >= (int64_t(1) << 31) / elem_bytes / (rows + 256);
}

// The backward's workspace: the row statistics, the plan, and the sums of split
// tiles of queries and keys.
struct BwdSpace {
  RowStats stats;
  DkvPlan plan;
  KeyParts parts;   // of dq
  size_t bytes;
};

template <typename T, int DP>
inline hipError_t launch_dkv_join(const AttnView& a, const BwdSpace& b, hipStream_t s) {
  const int64_t tiles = b.plan.max_parts / 2;   // split ones have two parts or more
  if (tiles == 0) return hipSuccess;
  attn_dkv_join_kernel<T, DP>
      <<<static_cast<unsigned>((tiles * a.n_kv_heads) << (b.plan.rows_log2 - 5)), 4 * DP, 0, s>>>(a, b.stats, b.plan);
  return hipGetLastError();
}

// kernels of fp32 (attn_f32.hip)
hipError_t launch_attn_fwd_f32(const AttnView& a, void* ws, hipStream_t s, int* err);
hipError_t launch_attn_bwd_f32(const AttnView& a, const BwdSpace& b, hipStream_t s, int* err);

}  // namespace staple
