// Attention over packed sequences with a causal mask, a sliding window and
// sinks: forward and backward.
//
// A workgroup is four waves of 32 queries (or, for dk and dv, keys), one a
// column of the products of attn_tile.h; the rows they meet come through LDS,
// 32 at a time, in rings of slots filled a few blocks ahead.  All three bf16
// kernels are bound by what a wave can issue: matrix products, exponentials
// and LDS reads together.  So they spread one block's vector work between the
// products of other blocks, and keep their loop free of address and mask work:
// positions are 32-bit, a head's rows are one buffer, and only blocks at the
// edge of what is seen apply a mask.
#include <type_traits>

#include "attn_row.h"
#include "attn_tile.h"

namespace staple {

constexpr int kWaves = 4;
constexpr int kTileRows = 32 * kWaves;   // queries (keys) of a workgroup

// A tile of kTileRows consecutive rows of one sequence.  Sequence b owns the
// slots floor(cu[b] / kTileRows) + b onwards, at least as many as it has
// tiles, so a grid of total / kTileRows + n_seqs slots holds every sequence
// and a workgroup finds its own by a search of cu alone.
struct TileOf {
  int64_t seq, first;   // first: the tile's first row within the sequence; seq -1: none
};
__device__ __forceinline__ TileOf tile_of_slot(const int32_t* cu, int64_t n_seqs, int64_t slot) {
  int64_t lo = 0, hi = n_seqs;   // slots of lo start at or before `slot`, those of hi after
  while (hi - lo > 1) {
    const int64_t mid = (lo + hi) >> 1;
    if (cu[mid] / kTileRows + mid <= slot) lo = mid;
    else hi = mid;
  }
  const int64_t tile = slot - (cu[lo] / kTileRows + lo);
  return TileOf{tile < 0 ? -1 : lo, tile * kTileRows};
}
static int64_t slots(int64_t total, int64_t n_seqs) { return total / kTileRows + n_seqs; }

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ int wave_id() { return uniform(threadIdx.x >> 6); }

// One sequence and head, and the workgroup's tile of its queries or keys.
struct Segment {
  int64_t q0, k0;          // first rows
  int nq, nk, past;        // lengths, and the position of query 0
  int first;               // the tile's first query (key)
  // False where there is no such tile.  find_lane: any slot a lane; find: one
  // slot for the whole workgroup, kept in scalar registers.
  __device__ __forceinline__ bool find_lane(const AttnView& a, const int32_t* cu, int64_t slot, int* err) {
    const TileOf tile = tile_of_slot(cu, a.n_seqs, slot);
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
  __device__ __forceinline__ bool find(const AttnView& a, const int32_t* cu, int64_t slot, int* err) {
    if (!find_lane(a, cu, slot, err)) return false;
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

// The 32-key blocks that some query at a position in [p_min, p_max] sees: those
// of the sinks, then the window's; and which of them every query of the wave's
// range sees whole.
struct KeyBlocks {
  int n_sink, lo, n;
  int nk;
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
  // First key of block b; blocks past the last lie past the keys.
  __device__ __forceinline__ int first(int b) const { return b < n ? (b < n_sink ? b : lo + b - n_sink) * 32 : nk; }
};

// The wave's 32 queries, one a column.
struct QueryCols : Segment {
  int head, hk;
  int wq, row, p;             // the wave's first query; the lane's, and its position
  bool in;
  __device__ __forceinline__ bool find(const AttnView& a, int64_t n_slots, int64_t id, int* err) {
    // the last tiles of a sequence see the most keys: they start first
    if (!Segment::find(a, a.cu_q, n_slots - 1 - id / a.n_heads, err)) return false;
    head = uniform(static_cast<int>(id % a.n_heads));
    hk = uniform(head / a.group);
    wq = first + 32 * wave_id();
    row = wq + (threadIdx.x & 31);
    in = row < nq;
    p = past + row;
    return true;
  }
  __device__ __forceinline__ KeyBlocks blocks(const AttnView& a) const {
    KeyBlocks b(a, nk, past + first, past + min(first + kTileRows, nq) - 1);
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

// Running softmax of the lane's column: the sums stay relative to `top`, an
// earlier maximum rounded up to an integer, until a score passes it by 8: the
// exponentials stay below 2^9, far from fp32's range, lanes exchange maxima
// only then, and what has been summed is scaled by a power of two, exactly.
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
    const float t = fmaxf(top, ceilf(fmaxf(m, other_half(m))));
    *keep = top == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(top - t);
    top = t;
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

// o / sum and lse of the wave's columns.  A NaN or an infinity may have come
// from a value row that the query does not see (its zero weight times it):
// such rows are done again key by key.
template <typename T, int DP>
__device__ __forceinline__ void finish_fwd(const AttnView& a, const QueryCols& w, const ColumnSoftmax& sm, f32x16_t* o) {
  const int half = (threadIdx.x & 63) >> 5;
  const float sum = sm.sum + other_half(sm.sum);
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
  bool bad = false;
#pragma unroll
  for (int d = 0; d < Tile<T, DP>::kDT; ++d) {
#pragma unroll
    for (int r = 0; r < 16; ++r) bad |= not_finite(o[d][r]);
    store_column<T>(a.o, w.q0 + w.row, w.head, a.head_dim, d, o[d], inv, w.in);
  }
  if (w.in && half == 0)
    a.lse[(w.q0 + w.row) * a.n_heads + w.head] = (sm.top + __builtin_amdgcn_logf(sum)) * kLn2;
  uint64_t again = __ballot(bad && w.in);
  again = (again | (again >> 32)) & 0xffffffffull;
  while (again) {
    const int i = __builtin_ctzll(again);
    again &= again - 1;
    attn_fwd_row<T>(a, w.q0 + w.wq + i, w.head, w.past + w.wq + i, w.k0);
  }
}

// fp32: one block after the other.
template <int DP, bool kWide>
__global__ __launch_bounds__(64 * kWaves, 1) void attn_fwd_f32_kernel(AttnView a, int64_t n_slots, int* err) {
  using T = float;
  using TL = Tile<T, DP>;
  constexpr int kBlock = 32 * TL::kRow;
  extern __shared__ __align__(1024) char smem[];
  lds_char* const lds = (lds_char*)smem;               // [2][K, V]
  check_offsets(a, err);
  QueryCols w;
  if (!w.find(a, n_slots, blockIdx.x, err)) return;
  const KeyBlocks keys = w.blocks(a);
  u32x4_t qf[TL::kSteps];
  const float c = load_queries<T, DP>(a, w, qf);
  TileLoader<T, DP, 32, kWaves, kWide> kl, vl;
  kl.init(a.k, w.k0, w.nk, w.hk, a.head_dim, wave_id());
  vl.init(a.v, w.k0, w.nk, w.hk, a.head_dim, wave_id());
  f32x16_t o[TL::kDT] = {};
  ColumnSoftmax sm;
  kl.load(keys.first(0), lds);
  vl.load(keys.first(0), lds + kBlock);
  for (int b = 0; b < keys.n; ++b) {
    wait_vmcnt<0>();
    lds_barrier();
    const lds_char* kt = lds + (b & 1) * 2 * kBlock;
    const lds_char* vt = kt + kBlock;
    lds_char* next = lds + ((b + 1) & 1) * 2 * kBlock;
    kl.load(keys.first(b + 1), next);
    vl.load(keys.first(b + 1), next + kBlock);
    f32x16_t s = {};
#pragma unroll
    for (int st = 0; st < TL::kSteps; ++st) s = mma16(TL::row_frag(kt, 0, st), qf[st], s, T{});
    if (!keys.whole(b)) mask_keys(a, w, keys.first(b), s);
    float keep;
    if (sm.raise(s, c, &keep)) {
#pragma unroll
      for (int d = 0; d < TL::kDT; ++d) o[d] *= keep;
    }
    const float base = sm.base();
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      s[r] = __builtin_amdgcn_exp2f(fmaf(s[r], c, -base));
      sm.sum += s[r];
    }
    Column<T> pc;
    pc.set(s);
#pragma unroll
    for (int d = 0; d < TL::kDT; ++d) o[d] = mma_transposed<DP>(vt, 0, d, pc, o[d]);
  }
  wait_vmcnt<0>();   // no load into LDS outlives the workgroup
  finish_fwd<T, DP>(a, w, sm, o);
}

// bf16.  A block (32 keys x 32 queries at DP 128) is 16 MFMAs, 512 cycles, and
// 16 exponentials a lane, nearly as many cycles of vector work.  So the wave
// runs three blocks at a time: between the exponentials of block b stand the
// score products of block b + 1 and the value products of block b - 1.  The
// workgroup meets every second block: a stage loads two blocks of K and of V
// while the two before are worked on.
template <int DP>
struct FwdShape {
  static constexpr int kBlock = 32 * Tile<bf16_t, DP>::kRow;
  static constexpr int kLds = 8 * kBlock;   // rings of four K blocks and four V blocks
};
template <int DP, bool kWide>
__global__ __launch_bounds__(64 * kWaves, 2) void attn_fwd_bf16_kernel(AttnView a, int64_t n_slots, int* err) {
  using T = bf16_t;
  using TL = Tile<T, DP>;
  constexpr int kBlock = FwdShape<DP>::kBlock;
  extern __shared__ __align__(1024) char smem[];
  lds_char* const kring = (lds_char*)smem;
  lds_char* const vring = kring + 4 * kBlock;
  check_offsets(a, err);
  QueryCols w;
  if (!w.find(a, n_slots, blockIdx.x, err)) return;
  const KeyBlocks keys = w.blocks(a);
  f32x16_t o[TL::kDT] = {};
  ColumnSoftmax sm;
  if (keys.n > 0) {
    TileLoader<T, DP, 32, kWaves, kWide> kl, vl;
    kl.init(a.k, w.k0, w.nk, w.hk, a.head_dim, wave_id());
    vl.init(a.v, w.k0, w.nk, w.hk, a.head_dim, wave_id());
#pragma unroll
    for (int b = 0; b < 4; ++b) kl.load(keys.first(b), kring + b * kBlock);
#pragma unroll
    for (int b = 0; b < 2; ++b) vl.load(keys.first(b), vring + b * kBlock);
    u32x4_t qf[TL::kSteps];
    const float c = load_queries<T, DP>(a, w, qf);
    wait_vmcnt<0>();
    lds_barrier();
    f32x16_t s0 = {}, s1;
    Column<T> p0, p1;
    RowReader<T, DP> rows(kring);
    ColumnReader<DP> cols(vring);
#pragma unroll
    for (int st = 0; st < TL::kSteps; ++st) s0 = mma16(rows.read(st, 0), qf[st], s0, T{});

    // Step b: exponentials of s (block b) into p, scores of block b + 1 into
    // next, values of block b - 1 with the weights prev; `at` bytes past the
    // readers' places.
    auto step = [&](auto is_first, auto place, int b, f32x16_t& s, f32x16_t& next, Column<T>& prev, Column<T>& p) {
      constexpr bool kFirst = decltype(is_first)::value;
      constexpr int at = decltype(place)::value;
      if (!keys.whole(b)) mask_keys(a, w, keys.first(b), s);
      float keep;
      if (sm.raise(s, c, &keep)) {
        if constexpr (!kFirst) {
#pragma unroll
          for (int d = 0; d < TL::kDT; ++d) o[d] *= keep;
          prev.scale(keep);
        }
      }
      const float base = sm.base();
      constexpr int kPairs = TL::kSteps;   // one score MFMA and one value MFMA each
      static_assert(kPairs == 2 * TL::kDT, "as many of either kind");
      u32x4_t kf[2], vf[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        kf[i] = rows.read(i, at);
        if constexpr (!kFirst) vf[i] = cols.read(i & 1, i >> 1, at);
      }
      float even = 0.0f;
      auto element = [&](int r) {
        const float e = __builtin_amdgcn_exp2f(fmaf(s[r], c, -base));
        sm.sum += e;
        if (r & 1) {
          uint32_t pair = pack_bf16x2(even, e);
          pin(pair);
          p.v[r >> 3][(r >> 1) & 3] = pair;
        }
        even = e;
      };
      constexpr int kPer = 8 / kPairs;   // elements after each MFMA
#pragma unroll
      for (int i = 0; i < kPairs; ++i) {
        __builtin_amdgcn_sched_barrier(0);
        next = mma16(kf[i & 1], qf[i], i == 0 ? f32x16_t{} : next, T{});
        if (i + 2 < kPairs) kf[i & 1] = rows.read(i + 2, at);
#pragma unroll
        for (int e = 0; e < kPer; ++e) element(2 * kPer * i + e);
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (!kFirst) {
          o[i >> 1] = mma16(vf[i & 1], prev.v[i & 1], o[i >> 1], T{});
          if (i + 2 < kPairs) vf[i & 1] = cols.read(i & 1, (i + 2) >> 1, at);
        }
#pragma unroll
        for (int e = 0; e < kPer; ++e) element(2 * kPer * i + kPer + e);
      }
      __builtin_amdgcn_sched_barrier(0);
    };
    // an odd number of steps, the last one's keys all hidden where it is one
    // more than there are blocks: the pair's registers change roles in place
    const int n = keys.n | 1;
    using Low = std::integral_constant<int, 0>;
    using High = std::integral_constant<int, kBlock>;
    step(std::true_type{}, High{}, 0, s0, s1, p1, p0);
    // a stage's blocks b - 1 and b lie in one half of the V ring, b + 1 and b +
    // 2 in the other half of K's
    int half = 0;
    rows.move(2 * kBlock);
    for (int b = 1; b < n; b += 2) {
      const int other = 2 * kBlock - half;
      wait_vmcnt<0>();   // the last stage's loads
      lds_barrier();
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        kl.load(keys.first(b + 3 + i), kring + half + i * kBlock);
        vl.load(keys.first(b + 1 + i), vring + other + i * kBlock);
      }
      step(std::false_type{}, Low{}, b, s1, s0, p0, p1);
      step(std::false_type{}, High{}, b + 1, s0, s1, p1, p0);
      rows.move(half - other);
      cols.move(other - half);
      half = other;
    }
    // the last block's values
    wait_vmcnt<0>();
    lds_barrier();
#pragma unroll
    for (int d = 0; d < TL::kDT; ++d)
#pragma unroll
      for (int x = 0; x < 2; ++x) o[d] = mma16(cols.read(x, d, 0), p0.v[x], o[d], T{});
  }
  finish_fwd<T, DP>(a, w, sm, o);
}

// ------------------------------------------------------------------ backward
// One query's row of dq, by a whole wave.
template <typename T>
__device__ __forceinline__ void attn_dq_row(const AttnView& a, int64_t t, int64_t h, int64_t p, int64_t k0) {
  const int64_t hk = h / a.group;
  int64_t sink_end, lo;
  visible_keys(p, a.window, a.sinks, &sink_end, &lo);
  const Row2 q = load_row<T>(a.q, t, h, a.head_dim), d_o = load_row<T>(a.d_o, t, h, a.head_dim);
  const float dl = dot(d_o, load_row<T>(a.o, t, h, a.head_dim)), lse = a.lse[t * a.n_heads + h];
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
  __device__ __forceinline__ QueryBlocks(const AttnView& a, const Segment& w) {
    const int last_key = min(w.first + kTileRows, w.nk) - 1;
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
// by the last of them to finish; and the items (tiles and parts) start in the
// order of their size, the largest first.  Written by one workgroup of the dq
// kernel, which runs before.
struct DkvPlan {
  int32_t* head;      // [0] items
  int32_t* blocks;    // [slots] blocks of the slot's tile
  int32_t* parts;     // [slots] its parts
  int32_t* first;     // [slots] its first partial result, where there are several parts
  int32_t* split;     // [slots] its number among the split tiles
  int32_t* items;     // [slots + max_parts][2] slot, part
  int32_t* done;      // [max_parts][n_kv_heads] parts of a split tile that have finished
  float* sums;        // [max_parts][n_kv_heads] dk and dv sums of a part
  int64_t n_slots;
  int target;         // parts per head to aim for
};
constexpr int kMinChunk = 16;   // blocks: a part's sums cost about as much traffic as two blocks
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

__device__ void plan_dkv(const AttnView& a, const DkvPlan& plan, int* err) {
  __shared__ int64_t sums[kWaves];
  __shared__ int count[kBuckets], start[kBuckets], n_parts, n_split;
  constexpr int kThreads = 64 * kWaves;
  const int n_slots = static_cast<int>(plan.n_slots);
  int64_t mine = 0;
  for (int s = threadIdx.x; s < n_slots; s += kThreads) {
    Segment w;
    int n = -1;   // no tile
    if (w.find_lane(a, a.cu_k, s, err)) n = QueryBlocks(a, w).per_head * a.group;
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
    plan.parts[s] = parts;
    if (parts > 1) {
      plan.first[s] = atomicAdd(&n_parts, parts);
      plan.split[s] = atomicAdd(&n_split, 1);
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
  }
  __syncthreads();
  for (int s = threadIdx.x; s < n_slots; s += kThreads) {
    const int n = plan.blocks[s];
    if (n < 0) continue;
    const int parts = plan.parts[s];
    int at = atomicAdd(&start[bucket((n + parts - 1) / parts)], parts);
    for (int p = 0; p < parts; ++p, ++at) {
      plan.items[2 * at] = s;
      plan.items[2 * at + 1] = p;
    }
  }
  for (int i = threadIdx.x; i < n_split * a.n_kv_heads; i += kThreads) plan.done[i] = 0;
}

// dq, and the row statistics for the other kernel.  In bf16 a block is 16
// MFMAs for the scores and their gradients, then 16 elements of vector work
// with the 8 MFMAs of the block before in between.
template <typename T, int DP>
struct DqShape {
  static constexpr int kAhead = 2;
  static constexpr int kKSlots = kAhead + 2, kVSlots = kAhead + 1;
  static constexpr int kBlock = 32 * Tile<T, DP>::kRow;
  static constexpr int kLds = (kKSlots + kVSlots) * kBlock;
};
template <typename T, int DP, bool kWide>
__global__ __launch_bounds__(64 * kWaves, sizeof(T) == 2 ? 2 : 1) void attn_dq_kernel(AttnView a, int64_t n_slots, RowStats stats,
                                                                                      DkvPlan plan, int* err) {
  using TL = Tile<T, DP>;
  using Shape = DqShape<T, DP>;
  using Loader = TileLoader<T, DP, 32, kWaves, kWide>;
  constexpr int kAhead = Shape::kAhead, kBlock = Shape::kBlock;
  constexpr int kFew = 8;   // blocks: see below
  extern __shared__ __align__(1024) char smem[];
  lds_char* const kring = (lds_char*)smem;
  lds_char* const vring = kring + Shape::kKSlots * kBlock;
  check_offsets(a, err);
  QueryCols w;
  if (blockIdx.x == 0) {
    plan_dkv(a, plan, err);
    return;
  }
  if (!w.find(a, n_slots, static_cast<int64_t>(blockIdx.x) - 1, err)) return;
  const KeyBlocks keys = w.blocks(a);
  const int half = (threadIdx.x & 63) >> 5;
  Loader kl, vl;
  kl.init(a.k, w.k0, w.nk, w.hk, a.head_dim, wave_id());
  vl.init(a.v, w.k0, w.nk, w.hk, a.head_dim, wave_id());
  // ring places of the blocks to read, and to load next
  int kr = 0, vr = 0, kn = kAhead * kBlock, vn = kAhead * kBlock;
  auto bump = [](int& at, int slots) { at = at + kBlock == slots * kBlock ? 0 : at + kBlock; };
  u32x4_t qf[TL::kSteps], dof[TL::kSteps];
  float delta = 0.0f;
#pragma unroll
  for (int s = 0; s < TL::kSteps; ++s) {
    dof[s] = load_frag<T>(a.d_o, w.q0 + w.row, w.head, a.head_dim, s, w.in);
    delta += dot_frag(dof[s], load_frag<T>(a.o, w.q0 + w.row, w.head, a.head_dim, s, w.in), T{});
  }
  delta += other_half(delta);
  const float lse = w.in ? a.lse[(w.q0 + w.row) * a.n_heads + w.head] : 0.0f;
  const float lse2 = lse == -INFINITY ? 0.0f : lse * kLog2e;
  const float c = load_queries<T, DP>(a, w, qf);
  if constexpr (sizeof(T) == 2) {
    // delta from the rounded o is off by sum d_o (o's rounding), which counts
    // where o is large: where few keys share a query's weight.  A workgroup of
    // few blocks therefore meets them once before, for delta + sum P (dP -
    // delta), exact as sum P = 1.
    if (keys.n <= kFew) {
      float more = 0.0f;
      for (int b = 0; b < keys.n; ++b) {
        kl.load(keys.first(b), kring);
        vl.load(keys.first(b), vring);
        wait_vmcnt<0>();
        lds_barrier();
        f32x16_t s = {}, dp = {};
#pragma unroll
        for (int st = 0; st < TL::kSteps; ++st) {
          s = mma16(TL::row_frag(kring, 0, st), qf[st], s, T{});
          dp = mma16(TL::row_frag(vring, 0, st), dof[st], dp, T{});
        }
        const SeenKeys seen(a, w.p, w.in, keys.first(b));
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const float g = __builtin_amdgcn_exp2f(fmaf(s[r], c, -lse2)) * (dp[r] - delta);
          more += seen(r) ? g : 0.0f;
        }
        lds_barrier();   // the block has been read
      }
      delta += more + other_half(more);
    }
  }
  if (w.in && half == 0) {
    stats.lse2[w.head * a.total_q + w.q0 + w.row] = lse2;
    stats.delta[w.head * a.total_q + w.q0 + w.row] = delta;
  }
#pragma unroll
  for (int b = 0; b < kAhead; ++b) {
    kl.load(keys.first(b), kring + b * kBlock);
    vl.load(keys.first(b), vring + b * kBlock);
  }
  f32x16_t dq[TL::kDT] = {};
  Column<T> prev;
  const lds_char* kprev = kring;
  auto step = [&](auto is_first, int b) {
    constexpr bool kFirst = decltype(is_first)::value;
    // the loads of one step may be under way; the first step also waits for
    // the columns' own
    wait_vmcnt<kFirst ? 0 : (kAhead - 1) * 2 * Loader::kPer>();
    lds_barrier();
    kl.load(keys.first(b + kAhead), kring + kn);
    vl.load(keys.first(b + kAhead), vring + vn);
    bump(kn, Shape::kKSlots);
    bump(vn, Shape::kVSlots);
    const lds_char* kt = kring + kr;
    const lds_char* vt = vring + vr;
    bump(kr, Shape::kKSlots);
    bump(vr, Shape::kVSlots);
    f32x16_t s = {}, dp = {};
#pragma unroll
    for (int st = 0; st < TL::kSteps; ++st) {
      s = mma16(TL::row_frag(kt, 0, st), qf[st], s, T{});
      dp = mma16(TL::row_frag(vt, 0, st), dof[st], dp, T{});
    }
    const bool whole = keys.whole(b);
    const SeenKeys seen(a, w.p, w.in, keys.first(b));
    if constexpr (sizeof(T) == 2) {
      if (!whole) {
        // hidden pairs: probability and gradient zero, whatever the products are
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          s[r] = seen(r) ? s[r] : -INFINITY;
          dp[r] = seen(r) ? dp[r] : delta;
        }
      }
      Column<T> ds;
      float even = 0.0f;
      constexpr int kMfma = 2 * TL::kDT;   // of the block before
      u32x4_t kf[2];
      if constexpr (!kFirst) {
#pragma unroll
        for (int i = 0; i < 2; ++i) kf[i] = column_frag<DP>(kprev, 0, i & 1, i >> 1);
      }
#pragma unroll
      for (int i = 0; i < kMfma; ++i) {
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (!kFirst) {
          dq[i >> 1] = mma16(kf[i & 1], prev.v[i & 1], dq[i >> 1], T{});
          if (i + 2 < kMfma) kf[i & 1] = column_frag<DP>(kprev, 0, i & 1, (i + 2) >> 1);
        }
#pragma unroll
        for (int e = 0; e < 16 / kMfma; ++e) {
          const int r = i * (16 / kMfma) + e;
          const float g = __builtin_amdgcn_exp2f(fmaf(s[r], c, -lse2)) * (dp[r] - delta);
          if (r & 1) {
            uint32_t pair = pack_bf16x2(even, g);
            pin(pair);
            ds.v[r >> 3][(r >> 1) & 3] = pair;
          }
          even = g;
        }
      }
      __builtin_amdgcn_sched_barrier(0);
      prev = ds;
      kprev = kt;
    } else {
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const float g = __builtin_amdgcn_exp2f(fmaf(s[r], c, -lse2)) * (dp[r] - delta);
        s[r] = (whole | seen(r)) ? g : 0.0f;
      }
      prev.set(s);
#pragma unroll
      for (int d = 0; d < TL::kDT; ++d) dq[d] = mma_transposed<DP>(kt, 0, d, prev, dq[d]);
    }
  };
  if (keys.n > 0) {
    step(std::true_type{}, 0);
    for (int b = 1; b < keys.n; ++b) step(std::false_type{}, b);
    if constexpr (sizeof(T) == 2) {
#pragma unroll
      for (int d = 0; d < TL::kDT; ++d) dq[d] = mma_transposed<DP>(kprev, 0, d, prev, dq[d]);
    }
  }
  wait_vmcnt<0>();   // no load into LDS outlives the workgroup
  bool bad = false;
#pragma unroll
  for (int d = 0; d < TL::kDT; ++d) {
#pragma unroll
    for (int r = 0; r < 16; ++r) bad |= not_finite(dq[d][r]);
    store_column<T>(a.dq, w.q0 + w.row, w.head, a.head_dim, d, dq[d], a.scale, w.in);
  }
  // a hidden key's rows may have brought it (zero times them): see the forward
  uint64_t again = __ballot(bad && w.in);
  again = (again | (again >> 32)) & 0xffffffffull;
  while (again) {
    const int i = __builtin_ctzll(again);
    again &= again - 1;
    attn_dq_row<T>(a, w.q0 + w.wq + i, w.head, w.past + w.wq + i, w.k0);
  }
}

// dk and dv: one key a column; the queries that see them (of every head of the
// group) go through LDS.  An item is a key tile or a part of one.
struct DkvItem : Segment {
  int slot, part, parts, hk;
  int64_t h0;              // the head of the item's first block
  int n, ln;               // its blocks, and the first one's number within its head
  int b_lo, per_head;      // see QueryBlocks
  int wkey, key;           // the wave's first key; the lane's
  bool in;
  int whole_lo, whole_n;   // of a head's blocks, those whose every query sees all of the wave's keys
  int seen_lo, seen_hi;    // and those of which some query sees some of them: [seen_lo, seen_hi)
  // False where there is no such item; `group`: which 32 keys of the tile the wave has.
  __device__ __forceinline__ bool find(const AttnView& a, const DkvPlan& plan, int group_of_wave, int* err) {
    const int item = uniform(static_cast<int>(blockIdx.x) / a.n_kv_heads);
    if (item >= plan.head[0]) return false;
    hk = static_cast<int>(blockIdx.x) - item * a.n_kv_heads;
    slot = uniform(plan.items[2 * item]);
    part = uniform(plan.items[2 * item + 1]);
    parts = uniform(plan.parts[slot]);
    if (!Segment::find(a, a.cu_k, slot, err)) return false;
    wkey = first + 32 * group_of_wave;
    key = wkey + (threadIdx.x & 31);
    in = key < nk;
    const QueryBlocks blocks(a, *this);
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
  __device__ __forceinline__ bool whole(int b) const {
    return static_cast<unsigned>(b - whole_lo) < static_cast<unsigned>(whole_n);
  }
};

// A split tile's part: its fp32 sums to the workspace, as they lie in the
// registers of the workgroup's kThreads threads (x: kX results a thread); true
// in the part that arrives last, with all parts' sums added in part order.
template <int kThreads, int kX>
__device__ __forceinline__ bool join_parts(const DkvPlan& plan, const DkvItem& w, int n_kv_heads, f32x16_t* x) {
  constexpr int kFloats = kThreads * 16 * kX;
  auto sums_of = [&](int p) {
    return reinterpret_cast<f32x4_t*>(plan.sums + (static_cast<int64_t>(plan.first[w.slot] + p) * n_kv_heads + w.hk) * kFloats) +
           threadIdx.x;
  };
  f32x4_t* mine = sums_of(w.part);
#pragma unroll
  for (int d = 0; d < kX; ++d)
#pragma unroll
    for (int g = 0; g < 4; ++g)
      mine[(d * 4 + g) * kThreads] = f32x4_t{x[d][4 * g], x[d][4 * g + 1], x[d][4 * g + 2], x[d][4 * g + 3]};
  __shared__ int arrived;
  __threadfence();   // the sums are visible to the device before the count
  __syncthreads();
  if (threadIdx.x == 0)
    arrived = __hip_atomic_fetch_add(&plan.done[plan.split[w.slot] * n_kv_heads + w.hk], 1, __ATOMIC_ACQ_REL,
                                     __HIP_MEMORY_SCOPE_AGENT);
  __syncthreads();
  if (arrived != w.parts - 1) return false;
  __threadfence();
#pragma unroll
  for (int d = 0; d < kX; ++d) x[d] = f32x16_t{};
  for (int p = 0; p < w.parts; ++p) {
    const f32x4_t* from = sums_of(p);
#pragma unroll
    for (int d = 0; d < kX; ++d)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const f32x4_t v = from[(d * 4 + g) * kThreads];
#pragma unroll
        for (int e = 0; e < 4; ++e) x[d][4 * g + e] += v[e];
      }
  }
  return true;
}

// Keys whose gradients came out not finite: a query that does not see the key
// may have brought it (zero times its rows), so they are done again query by
// query; see the forward.
template <typename T>
__device__ __forceinline__ void redo_keys(const AttnView& a, const RowStats& stats, const DkvItem& w, bool bad) {
  uint64_t again = __ballot(bad && w.in);
  again = (again | (again >> 32)) & 0xffffffffull;
  while (again) {
    const int i = __builtin_ctzll(again);
    again &= again - 1;
    attn_dkv_row<T>(a, stats.delta, w.wkey + i, w.hk, w);
  }
}

// A ring slot holds a block's Q and dO, then lse2 and delta (256 bytes each,
// half of it used).
template <typename T, int DP>
struct DkvShape {
  static constexpr int kBlock = 32 * Tile<T, DP>::kRow;
  static constexpr int kStage = 2 * kBlock + 512;
};

// fp32: one block after the other.
template <int DP, bool kWide>
__global__ __launch_bounds__(64 * kWaves, 1) void attn_dkv_f32_kernel(AttnView a, RowStats stats, DkvPlan plan, int* err) {
  using T = float;
  using TL = Tile<T, DP>;
  constexpr int kBlock = DkvShape<T, DP>::kBlock, kStage = DkvShape<T, DP>::kStage;
  extern __shared__ __align__(1024) char smem[];
  lds_char* const ring = (lds_char*)smem;
  DkvItem w;
  if (!w.find(a, plan, wave_id(), err)) return;
  const int lane = threadIdx.x & 63;
  TileLoader<T, DP, 32, kWaves, kWide> ql, dl;
  ql.init(a.q, w.q0, w.nq, w.h0, a.head_dim, wave_id());
  dl.init(a.d_o, w.q0, w.nq, w.h0, a.head_dim, wave_id());
  const int sw = wave_id();
  const float* stat = (sw & 1 ? stats.delta : stats.lse2) + w.h0 * a.total_q + w.q0;
  int left = w.n, ln = w.ln, bn = w.ln;   // to load; at hand
  auto load = [&](lds_char* slot) {
    const int i0 = left > 0 ? (w.b_lo + ln) * 32 : w.nq;   // past the last block: zeros
    ql.load(i0, slot);
    dl.load(i0, slot + kBlock);
    if (sw < 2) dma4(stat + min(i0 + lane, w.nq - 1), static_cast<lds_void*>(slot + 2 * kBlock + 256 * sw));
    --left;
    if (++ln == w.per_head) {
      ln = 0;
      ql.next_head(a.q);
      dl.next_head(a.d_o);
      if (left > 0) stat += a.total_q;
    }
  };
  f32x16_t x[2 * TL::kDT] = {};   // dk, then dv
  const float c = score_factor(a);
  if (w.n > 0) {
    u32x4_t kf[TL::kSteps], vf[TL::kSteps];
#pragma unroll
    for (int s = 0; s < TL::kSteps; ++s) {
      kf[s] = signed_frag<T>(a, load_frag<T>(a.k, w.k0 + w.key, w.hk, a.head_dim, s, w.in));
      vf[s] = load_frag<T>(a.v, w.k0 + w.key, w.hk, a.head_dim, s, w.in);
    }
    load(ring);
    for (int b = 0; b < w.n; ++b) {
      wait_vmcnt<0>();
      lds_barrier();
      const lds_char* qt = ring + (b & 1) * kStage;
      const lds_char* dt = qt + kBlock;
      load(ring + ((b + 1) & 1) * kStage);
      f32x16_t s = {}, g = {};
#pragma unroll
      for (int st = 0; st < TL::kSteps; ++st) {
        s = mma16(TL::row_frag(qt, 0, st), kf[st], s, T{});
        g = mma16(TL::row_frag(dt, 0, st), vf[st], g, T{});
      }
      const lds_char* st = qt + 2 * kBlock + 16 * (lane >> 5);
      const bool every = w.whole(bn);
      const SeenBy seen(a, w, w.key, w.in, (w.b_lo + bn) * 32);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const f32x4_t l4 = *reinterpret_cast<const lds_f32x4*>(st + 32 * q);
        const f32x4_t d4 = *reinterpret_cast<const lds_f32x4*>(st + 256 + 32 * q);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int r = 4 * q + e;
          const bool yes = every | seen(r);
          const float pr = __builtin_amdgcn_exp2f(fmaf(s[r], c, -l4[e]));
          g[r] = yes ? pr * (g[r] - d4[e]) : 0.0f;
          s[r] = yes ? pr : 0.0f;
        }
      }
      Column<T> pc, ds;
      pc.set(s);
      ds.set(g);
#pragma unroll
      for (int d = 0; d < TL::kDT; ++d) {
        x[d] = mma_transposed<DP>(qt, 0, d, ds, x[d]);
        x[TL::kDT + d] = mma_transposed<DP>(dt, 0, d, pc, x[TL::kDT + d]);
      }
      if (++bn == w.per_head) bn = 0;
    }
    wait_vmcnt<0>();   // no load into LDS outlives the workgroup
  }
  if (w.parts > 1 && !join_parts<64 * kWaves, 2 * TL::kDT>(plan, w, a.n_kv_heads, x)) return;
  bool bad = false;
#pragma unroll
  for (int d = 0; d < TL::kDT; ++d) {
#pragma unroll
    for (int r = 0; r < 16; ++r) bad |= not_finite(x[d][r]) || not_finite(x[TL::kDT + d][r]);
    store_column<T>(a.dk, w.k0 + w.key, w.hk, a.head_dim, d, x[d], a.scale, w.in);
    store_column<T>(a.dv, w.k0 + w.key, w.hk, a.head_dim, d, x[TL::kDT + d], 1.0f, w.in);
  }
  redo_keys<T>(a, stats, w, bad);
}

// bf16.  dk and dv of 32 keys take 2 DP registers a lane, too many beside the
// operands for two waves a SIMD.  So two waves share 32 keys: of a stage of
// two query blocks each forms the probabilities and score gradients of one,
// they trade them through LDS, and each adds both to its half of head_dim.
// Between the elements of a stage stand the gradient products of the stage
// before.
constexpr int kDkvWaves = 8;
template <int DP>
struct DkvPair {
  static constexpr int kStage = DkvShape<bf16_t, DP>::kStage;
  static constexpr int kTrade = 4 * 2 * 4 * 1024;              // [keys / 32][block][P, P, dS, dS][lane]
  static constexpr int kLds = 6 * kStage + kTrade;             // three pairs of slots: before, at hand, loading
};
template <int DP, bool kWide>
__global__ __launch_bounds__(64 * kDkvWaves, 2) void attn_dkv_bf16_kernel(AttnView a, RowStats stats, DkvPlan plan, int* err) {
  using T = bf16_t;
  using TL = Tile<T, DP>;
  using Shape = DkvPair<DP>;
  constexpr int kBlock = DkvShape<T, DP>::kBlock, kStage = Shape::kStage, kPair = 2 * kStage;
  constexpr int kHalf = TL::kDT / 2;   // 32-element blocks of head_dim a wave
  extern __shared__ __align__(1024) char smem[];
  lds_char* const ring = (lds_char*)smem;
  const int keys_of = wave_id() & 3, side = wave_id() >> 2;
  DkvItem w;
  if (!w.find(a, plan, keys_of, err)) return;
  const int lane = threadIdx.x & 63;
  lds_char* const trade = ring + 6 * kStage + keys_of * (2 * 4 * 1024) + lane * 16;

  // waves 0-3 load Q and lse2, waves 4-7 dO and delta
  TileLoader<T, DP, 32, 4, kWide> loader;
  const HeadsView& source = side ? a.d_o : a.q;
  loader.init(source, w.q0, w.nq, w.h0, a.head_dim, keys_of);
  const float* stat = (side ? stats.delta : stats.lse2) + w.h0 * a.total_q + w.q0;
  int left = w.n, ln = w.ln;
  auto load = [&](lds_char* slot) {
    const int i0 = left > 0 ? (w.b_lo + ln) * 32 : w.nq;   // past the last block: zeros
    loader.load(i0, slot + side * kBlock);
    if (keys_of == 0) dma4(stat + min(i0 + lane, w.nq - 1), static_cast<lds_void*>(slot + 2 * kBlock + 256 * side));
    --left;
    if (++ln == w.per_head) {
      ln = 0;
      loader.next_head(source);
      if (left > 0) stat += a.total_q;
    }
  };
  f32x16_t x[2 * kHalf] = {};   // dk, then dv
  const float c = score_factor(a);
  if (w.n > 0) {
    load(ring);
    load(ring + kStage);
    u32x4_t kf[TL::kSteps], vf[TL::kSteps];
#pragma unroll
    for (int s = 0; s < TL::kSteps; ++s) {
      kf[s] = signed_frag<T>(a, load_frag<T>(a.k, w.k0 + w.key, w.hk, a.head_dim, s, w.in));
      vf[s] = load_frag<T>(a.v, w.k0 + w.key, w.hk, a.head_dim, s, w.in);
    }
    RowReader<T, DP> rows(ring + side * kStage);                   // this wave's block of the stage
    ColumnReader<DP, kHalf> cols(ring, side * kHalf);              // its half of head_dim, of the stage before
    const lds_char* stat_at = ring + side * kStage + 2 * kBlock + 16 * (lane >> 5);
    int bn = w.ln + side;   // the wave's block, within its head
    while (bn >= w.per_head) bn -= w.per_head;

    // product m of the stage before: block, result, rows and elements
    constexpr int kProducts = 2 * 2 * 2 * kHalf;   // blocks x (dk, dv) x row halves x element blocks
    struct Product {
      int block, which, t, d;
    };
    auto product = [](int m) { return Product{m / (4 * kHalf), m / (2 * kHalf) & 1, m & 1, (m >> 1) % kHalf}; };
    auto read_a = [&](int m) {
      const Product q = product(m);
      return cols.read(q.t, q.d, q.block * kStage + q.which * kBlock);
    };
    auto read_b = [&](int m) {   // dk takes the score gradients, dv the probabilities
      const Product q = product(m);
      return *reinterpret_cast<const lds_u32x4*>(trade + q.block * 4096 + ((q.which ? 0 : 2) + q.t) * 1024);
    };

    // pair_seen: whether the blocks of the stage before hold anything for these keys
    auto stage = [&](auto is_first, int j, bool pair_seen) {
      constexpr bool kFirst = decltype(is_first)::value;
      wait_vmcnt<0>();   // this stage's blocks
      lds_barrier();     // and the trade of the stage before
      lds_char* const next = ring + (j + 1) % 3 * kPair;
      load(next);
      load(next + kStage);
      Column<T> p, e;
      const bool mine = 2 * j + side < w.n && bn >= w.seen_lo && bn < w.seen_hi;
      if (mine || pair_seen) {
        f32x16_t s = {}, g = {};
#pragma unroll
        for (int st = 0; st < TL::kSteps; ++st) {
          s = mma16(rows.read(st, 0), kf[st], s, T{});
          g = mma16(rows.read(st, kBlock), vf[st], g, T{});
        }
        f32x4_t l4[4], d4[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          l4[q] = *reinterpret_cast<const lds_f32x4*>(stat_at + 32 * q);
          d4[q] = *reinterpret_cast<const lds_f32x4*>(stat_at + 256 + 32 * q);
        }
        if (!(mine && w.whole(bn))) {
          // hidden pairs: probability and gradient zero, whatever the products
          // and the query's statistics are
          const SeenBy seen(a, w, w.key, mine && w.in, (w.b_lo + bn) * 32);
#pragma unroll
          for (int r = 0; r < 16; ++r) {
            const bool yes = seen(r);
            s[r] = yes ? s[r] : -INFINITY;
            l4[r >> 2][r & 3] = yes ? l4[r >> 2][r & 3] : 0.0f;
            g[r] = yes ? g[r] : 0.0f;
            d4[r >> 2][r & 3] = yes ? d4[r >> 2][r & 3] : 0.0f;
          }
        }
        float pe = 0.0f, ee = 0.0f;
        auto element = [&](int r) {
          const float pr = __builtin_amdgcn_exp2f(fmaf(s[r], c, -l4[r >> 2][r & 3]));
          const float ds = pr * (g[r] - d4[r >> 2][r & 3]);
          if (r & 1) {
            uint32_t px = pack_bf16x2(pe, pr), ex = pack_bf16x2(ee, ds);
            pin(px);
            pin(ex);
            p.v[r >> 3][(r >> 1) & 3] = px;
            e.v[r >> 3][(r >> 1) & 3] = ex;
          }
          pe = pr;
          ee = ds;
        };
        constexpr int kAhead = 2;   // operands in flight
        u32x4_t af[kAhead], bf[kAhead];
        if constexpr (!kFirst) {
#pragma unroll
          for (int m = 0; m < kAhead; ++m) {
            af[m] = read_a(m);
            bf[m] = read_b(m);
          }
        }
#pragma unroll
        for (int m = 0; m < kProducts; ++m) {
          __builtin_amdgcn_sched_barrier(0);
          if constexpr (!kFirst) {
            const Product q = product(m);
            x[q.which * kHalf + q.d] = mma16(af[m % kAhead], bf[m % kAhead], x[q.which * kHalf + q.d], T{});
            if (m + kAhead < kProducts) {
              af[m % kAhead] = read_a(m + kAhead);
              bf[m % kAhead] = read_b(m + kAhead);
            }
          }
#pragma unroll
          for (int r = 0; r < 16 / kProducts; ++r) element(m * (16 / kProducts) + r);
        }
        __builtin_amdgcn_sched_barrier(0);
      } else {
        p.v[0] = p.v[1] = e.v[0] = e.v[1] = u32x4_t{0, 0, 0, 0};
      }
      lds_barrier();   // both waves have read the trade of the stage before
      lds_char* const mine_at = trade + side * 4096;
      *reinterpret_cast<lds_u32x4*>(mine_at) = p.v[0];
      *reinterpret_cast<lds_u32x4*>(mine_at + 1024) = p.v[1];
      *reinterpret_cast<lds_u32x4*>(mine_at + 2048) = e.v[0];
      *reinterpret_cast<lds_u32x4*>(mine_at + 3072) = e.v[1];
      const int by = (j + 1) % 3 == 0 ? -2 * kPair : kPair;
      rows.move(by);
      stat_at += by;
      if constexpr (!kFirst) cols.move(j % 3 == 0 ? -2 * kPair : kPair);
    };
    // whether some query of either block of stage j sees some of the keys
    auto seen_pair = [&](int j) {
      int first = bn - side;
      if (first < 0) first += w.per_head;
      const int second = first + 1 == w.per_head ? 0 : first + 1;
      return (first >= w.seen_lo && first < w.seen_hi) || (2 * j + 1 < w.n && second >= w.seen_lo && second < w.seen_hi);
    };
    auto next_blocks = [&]() {
      bn += 2;
      while (bn >= w.per_head) bn -= w.per_head;
    };
    const int n_stages = (w.n + 1) / 2;
    bool before = seen_pair(0);
    stage(std::true_type{}, 0, false);
    next_blocks();
    for (int j = 1; j < n_stages; ++j) {
      const bool here = seen_pair(j);
      stage(std::false_type{}, j, before);
      before = here;
      next_blocks();
    }
    wait_vmcnt<0>();   // no load into LDS outlives the workgroup
    lds_barrier();
    if (before) {
#pragma unroll
      for (int m = 0; m < kProducts; ++m) {
        const Product q = product(m);
        x[q.which * kHalf + q.d] = mma16(read_a(m), read_b(m), x[q.which * kHalf + q.d], T{});
      }
    }
  }
  if (w.parts > 1 && !join_parts<64 * kDkvWaves, 2 * kHalf>(plan, w, a.n_kv_heads, x)) return;
  bool bad = false;
#pragma unroll
  for (int d = 0; d < kHalf; ++d) {
#pragma unroll
    for (int r = 0; r < 16; ++r) bad |= not_finite(x[d][r]) || not_finite(x[kHalf + d][r]);
    store_column<T>(a.dk, w.k0 + w.key, w.hk, a.head_dim, side * kHalf + d, x[d], a.scale, w.in);
    store_column<T>(a.dv, w.k0 + w.key, w.hk, a.head_dim, side * kHalf + d, x[kHalf + d], 1.0f, w.in);
  }
  __syncthreads();   // a row done again is stored after both its halves
  redo_keys<T>(a, stats, w, bad);
}

// ------------------------------------------------------------------- launches
// Raises a kernel's limit of dynamic LDS past the 64 KB that a launch gets
// unasked (once a kernel), then launches it.
template <auto kKernel, int kLds, int kThreads = 64 * kWaves, typename... Args>
static hipError_t launch_lds(int64_t wgs, hipStream_t s, Args... args) {
  if (wgs == 0) return hipSuccess;
  static const hipError_t attr =
      hipFuncSetAttribute(reinterpret_cast<const void*>(kKernel), hipFuncAttributeMaxDynamicSharedMemorySize, kLds);
  if (attr != hipSuccess) return attr;
  kKernel<<<static_cast<unsigned>(wgs), kThreads, kLds, s>>>(args...);
  return hipGetLastError();
}

// Whether a head's rows may span 2^31 bytes.
static bool wide(const HeadsView& t, int64_t rows, int elem_bytes) {
  return t.row_stride >= (int64_t(1) << 31) / elem_bytes / (rows + 2 * kTileRows);
}

template <bool kWide>
static hipError_t fwd_launch(const AttnView& a, int dtype, hipStream_t s, int* err) {
  const int64_t n = slots(a.total_q, a.n_seqs), wgs = n * a.n_heads;
  if (dtype == STAPLE_BF16) {
    if (a.head_dim <= 64) return launch_lds<attn_fwd_bf16_kernel<64, kWide>, FwdShape<64>::kLds>(wgs, s, a, n, err);
    return launch_lds<attn_fwd_bf16_kernel<128, kWide>, FwdShape<128>::kLds>(wgs, s, a, n, err);
  }
  if (a.head_dim <= 64) return launch_lds<attn_fwd_f32_kernel<64, kWide>, 4 * 32 * 256>(wgs, s, a, n, err);
  return launch_lds<attn_fwd_f32_kernel<128, kWide>, 4 * 32 * 512>(wgs, s, a, n, err);
}

hipError_t launch_attn_fwd(const AttnView& a, int dtype, hipStream_t s, int* err) {
  const int es = dtype == STAPLE_BF16 ? 2 : 4;
  return wide(a.k, a.total_k, es) || wide(a.v, a.total_k, es) ? fwd_launch<true>(a, dtype, s, err)
                                                              : fwd_launch<false>(a, dtype, s, err);
}

// The backward's workspace: the row statistics, the plan, and the sums of
// split tiles.  A split tile has more than `chunk` blocks, so that all of them
// together have at most 2 total / chunk <= 2 target parts, and no more than
// two for every kMinChunk blocks.
struct BwdSpace {
  RowStats stats;
  DkvPlan plan;
  int max_parts;
  size_t bytes;
};
static BwdSpace bwd_space(const AttnView& a, int dtype, void* ws) {
  BwdSpace b{};
  const int dp = a.head_dim <= 64 ? 64 : 128;
  const int64_t n = slots(a.total_k, a.n_seqs);
  b.plan.n_slots = n;
  b.plan.target = (2 * device_cus() + a.n_kv_heads - 1) / a.n_kv_heads;   // two parts a CU
  const int64_t blocks = (a.total_q / 32 + a.n_seqs) * a.group * n;       // more than there are
  const int64_t most = 2 * (blocks / kMinChunk) + 2;
  b.max_parts = static_cast<int>(most < 2 * b.plan.target ? most : 2 * b.plan.target);
  Workspace w(ws, ~size_t(0));
  const size_t rows = static_cast<size_t>(a.total_q) * a.n_heads * sizeof(float);
  const size_t ints = static_cast<size_t>(n) * sizeof(int32_t);
  b.stats.lse2 = w.take<float>(rows);
  b.stats.delta = w.take<float>(rows);
  b.plan.head = w.take<int32_t>(sizeof(int32_t));
  b.plan.blocks = w.take<int32_t>(ints);
  b.plan.parts = w.take<int32_t>(ints);
  b.plan.first = w.take<int32_t>(ints);
  b.plan.split = w.take<int32_t>(ints);
  b.plan.items = w.take<int32_t>(2 * (ints + b.max_parts * sizeof(int32_t)));
  b.plan.done = w.take<int32_t>(static_cast<size_t>(b.max_parts) * a.n_kv_heads * sizeof(int32_t));
  const size_t sums = static_cast<size_t>(kWaves) * 2 * 64 * 16 * (dp / 32) * sizeof(float);
  b.plan.sums = w.take<float>(static_cast<size_t>(b.max_parts) * a.n_kv_heads * sums);
  b.bytes = w.used;
  return b;
}
size_t attn_bwd_workspace_bytes(const AttnView& a, int dtype) { return bwd_space(a, dtype, nullptr).bytes; }

template <typename T, int DP, bool kWide>
static hipError_t bwd_launch(const AttnView& a, int dtype, void* ws, hipStream_t s, int* err) {
  const BwdSpace b = bwd_space(a, dtype, ws);
  const int64_t nq = slots(a.total_q, a.n_seqs);
  // one workgroup more than there are query tiles: it makes the plan
  hipError_t e = launch_lds<attn_dq_kernel<T, DP, kWide>, DqShape<T, DP>::kLds>(nq * a.n_heads + 1, s, a, nq, b.stats, b.plan, err);
  if (e != hipSuccess) return e;
  const int64_t items = (b.plan.n_slots + b.max_parts) * a.n_kv_heads;   // at most
  if constexpr (sizeof(T) == 2)
    return launch_lds<attn_dkv_bf16_kernel<DP, kWide>, DkvPair<DP>::kLds, 64 * kDkvWaves>(items, s, a, b.stats, b.plan, err);
  else
    return launch_lds<attn_dkv_f32_kernel<DP, kWide>, 2 * DkvShape<T, DP>::kStage>(items, s, a, b.stats, b.plan, err);
}

template <bool kWide>
static hipError_t bwd_launch(const AttnView& a, int dtype, void* ws, hipStream_t s, int* err) {
  if (dtype == STAPLE_BF16)
    return a.head_dim <= 64 ? bwd_launch<bf16_t, 64, kWide>(a, dtype, ws, s, err) : bwd_launch<bf16_t, 128, kWide>(a, dtype, ws, s, err);
  return a.head_dim <= 64 ? bwd_launch<float, 64, kWide>(a, dtype, ws, s, err) : bwd_launch<float, 128, kWide>(a, dtype, ws, s, err);
}

hipError_t launch_attn_bwd(const AttnView& a, int dtype, void* ws, hipStream_t s, int* err) {
  const int es = dtype == STAPLE_BF16 ? 2 : 4;
  const bool far = wide(a.q, a.total_q, es) || wide(a.d_o, a.total_q, es) || wide(a.k, a.total_k, es) || wide(a.v, a.total_k, es);
  return far ? bwd_launch<true>(a, dtype, ws, s, err) : bwd_launch<false>(a, dtype, ws, s, err);
}

}  // namespace staple
