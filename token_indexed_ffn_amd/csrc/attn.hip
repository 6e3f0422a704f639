// Attention over packed sequences with a causal mask, a sliding window and
// sinks: forward and backward.
#include "attn_row.h"
#include "attn_tile.h"

namespace staple {

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

// ------------------------------------------------------------------- forward
// A tile of `rows` consecutive rows of one sequence and one head.  Sequence b
// owns the slots floor(cu[b] / rows) + b onwards, at least as many as it has
// tiles, so a grid of total / rows + n_seqs slots holds every sequence and a
// workgroup finds its own by a search of cu alone.
struct TileOf {
  int64_t seq, first;   // first: the tile's first row within the sequence; seq -1: none
};
__device__ __forceinline__ TileOf tile_of_slot(const int32_t* cu, int64_t n_seqs, int rows, int64_t slot) {
  int64_t lo = 0, hi = n_seqs;   // slots of lo start at or before `slot`, those of hi after
  while (hi - lo > 1) {
    const int64_t mid = (lo + hi) >> 1;
    if (cu[mid] / rows + mid <= slot) lo = mid;
    else hi = mid;
  }
  const int64_t tile = slot - (cu[lo] / rows + lo);
  return TileOf{tile < 0 ? -1 : lo, tile * rows};
}
static int64_t slots(int64_t total, int64_t n_seqs, int rows) { return total / rows + n_seqs; }

// Workgroup id -> (slot, head).  Consecutive ids run on different XCDs, each
// with its own L2.
struct Work {
  int64_t slot;
  int head;
};
__device__ __forceinline__ Work work_of(int64_t n_slots, int heads) {
  const int64_t id = blockIdx.x;
  return Work{n_slots - 1 - id / heads, static_cast<int>(id % heads)};
}

// The key tiles of `rows` keys that some query at a position in [p_min, p_max]
// sees: those of the sinks, then the window's.
struct KeyTiles {
  int64_t n_sink, lo, n;
  int rows;
  __device__ __forceinline__ KeyTiles(const AttnView& a, int64_t p_min, int64_t p_max, int rows_)
      : rows(rows_) {
    lo = (a.window > 0 && p_min >= a.window ? p_min - a.window + 1 : 0) / rows;
    const int64_t sink_keys = a.sinks < lo * rows ? a.sinks : lo * rows;
    n_sink = p_max < 0 ? 0 : (sink_keys + rows - 1) / rows;
    n = p_max < 0 ? 0 : n_sink + p_max / rows + 1 - lo;
  }
  __device__ __forceinline__ int64_t first(int64_t it) const { return (it < n_sink ? it : lo + it - n_sink) * rows; }
};
// Whether no query at a position in [p_min, p_max] sees a key in [key, key +
// n), or every one sees them all.
__device__ __forceinline__ bool none_visible(const AttnView& a, int64_t p_min, int64_t p_max, int64_t key, int n) {
  return key > p_max || (a.window > 0 && key + n - 1 <= p_min - a.window && key >= a.sinks);
}
__device__ __forceinline__ bool all_visible(const AttnView& a, int64_t p_min, int64_t p_max, int64_t key, int n) {
  return key + n - 1 <= p_min && (a.window == 0 || key > p_max - a.window || key + n <= a.sinks);
}
// Masks are applied with selects (a few integer compares an element), never by
// branching on one element of a result.
// Which rows of a key block the lane's query (at position p) sees: row j =
// 8 (r / 4) + r % 4 (+ 4 for the upper half-wave) of the tile that starts at
// `key` is seen when j <= hi and (j >= lo or j < sink).
struct SeenKeys {
  int hi, lo, sink;
  __device__ __forceinline__ SeenKeys(const AttnView& a, int64_t p, bool in, int64_t key) {
    const int64_t at = key + 4 * ((threadIdx.x & 63) >> 5);
    hi = in ? clamp_rel(p - at) : -(1 << 20);
    lo = a.window > 0 ? clamp_rel(p - a.window + 1 - at) : -(1 << 20);
    sink = clamp_rel(a.sinks - at);
  }
  __device__ __forceinline__ bool operator()(int j) const { return (j <= hi) & ((j >= lo) | (j < sink)); }
};

// Which queries of a 32-query block (the first at position p0, number i0 of
// nq) see the lane's key: query j = 8 (r / 4) + r % 4 (+ 4 for the upper
// half-wave) does when lo <= j < hi.
struct SeenBy {
  int lo, hi;
  __device__ __forceinline__ SeenBy(const AttnView& a, int64_t key, bool in, int64_t p0, int64_t i0, int64_t nq) {
    const int64_t up = 4 * ((threadIdx.x & 63) >> 5);
    lo = clamp_rel(key - p0 - up);
    int64_t end = nq - i0;
    if (a.window > 0 && key >= a.sinks && key + a.window - p0 < end) end = key + a.window - p0;
    hi = in ? clamp_rel(end - up) : -(1 << 20);
  }
  __device__ __forceinline__ bool operator()(int j) const { return (j >= lo) & (j < hi); }
};

// True where a value is NaN or infinite.
__device__ __forceinline__ bool not_finite(float x) { return !(fabsf(x) < INFINITY); }

template <typename T, int DP, int NW>
__global__ __launch_bounds__(64 * NW, sizeof(T) == 2 ? 2 : 1) void attn_fwd_kernel(AttnView a, int64_t n_slots, int* err) {
  using TL = Tile<T, DP>;
  constexpr int kKeys = sizeof(T) == 2 ? 64 : 32;      // keys per tile
  constexpr int kTile = kKeys * TL::kRow;
  extern __shared__ __align__(1024) char smem[];
  lds_char* const lds = (lds_char*)smem;               // [2][K, V]
  check_offsets(a, err);
  const Work wk = work_of(n_slots, a.n_heads);
  const TileOf tile = tile_of_slot(a.cu_q, a.n_seqs, 32 * NW, wk.slot);
  if (tile.seq < 0) return;
  int64_t q0, q1, k0, k1;
  seq_rows(a.cu_q, tile.seq, a.total_q, &q0, &q1, err);
  seq_rows(a.cu_k, tile.seq, a.total_k, &k0, &k1, err);
  const int64_t nq = q1 - q0, nk = k1 - k0, past = nk - nq;
  if (tile.first >= nq) return;
  const int lane = threadIdx.x & 63, half = lane >> 5;
  const int head = wk.head, hk = head / a.group;

  // this wave's queries, one a column
  const int64_t wq = tile.first + 32 * (threadIdx.x >> 6);
  const int64_t row = wq + (lane & 31);
  const bool in = row < nq;
  const int64_t p = past + row;
  const int64_t p_min = past + wq, p_max = past + (wq + 31 < nq ? wq + 31 : nq - 1);
  const bool wave_in = wq < nq && p_max >= 0;
  u32x4_t qf[TL::kSteps];
#pragma unroll
  for (int s = 0; s < TL::kSteps; ++s) {
    qf[s] = load_frag<T>(a.q, q0 + row, head, a.head_dim, s, in);
    if (a.scale < 0.0f) qf[s] = flip_sign<T>(qf[s]);
  }
  const float c = fabsf(a.scale) * 1.44269504088896340736f;   // scores in powers of two

  const KeyTiles keys(a, past + tile.first, past + (tile.first + 32 * NW < nq ? tile.first + 32 * NW : nq) - 1, kKeys);
  TileLoader<T, DP, kKeys, NW> kl, vl;
  kl.init(a.k, k0, hk, a.head_dim);
  vl.init(a.v, k0, hk, a.head_dim);
  f32x16_t o[TL::kDT] = {};
  float top = -INFINITY, sum = 0.0f;   // of the lane's column; sum: this half-wave's keys
  if (keys.n > 0) {
    kl.load(keys.first(0), nk, lds);
    vl.load(keys.first(0), nk, lds + kTile);
  }
  for (int64_t it = 0; it < keys.n; ++it) {
    wait_vmcnt<0>();
    lds_barrier();
    const lds_char* kt = lds + (it & 1) * 2 * kTile;
    const lds_char* vt = kt + kTile;
    if (it + 1 < keys.n) {
      lds_char* next = lds + ((it + 1) & 1) * 2 * kTile;
      kl.load(keys.first(it + 1), nk, next);
      vl.load(keys.first(it + 1), nk, next + kTile);
    }
    const int64_t key = keys.first(it);
    if (!wave_in || none_visible(a, p_min, p_max, key, kKeys)) continue;
    const bool all = wq + 31 < nq && all_visible(a, p_min, p_max, key, kKeys);
    f32x16_t s[kKeys / 32];
#pragma unroll
    for (int n = 0; n < kKeys / 32; ++n) {
      s[n] = f32x16_t{};
#pragma unroll
      for (int st = 0; st < TL::kSteps; ++st) s[n] = mma16(TL::row_frag(kt, 32 * n, st), qf[st], s[n], T{});
    }
    // scaled scores, -inf where hidden
#pragma unroll
    for (int n = 0; n < kKeys / 32; ++n) s[n] *= c;
    if (!all) {
      const SeenKeys seen(a, p, in, key);
#pragma unroll
      for (int n = 0; n < kKeys / 32; ++n)
#pragma unroll
        for (int r = 0; r < 16; ++r) s[n][r] = seen(32 * n + 8 * (r >> 2) + (r & 3)) ? s[n][r] : -INFINITY;
    }
    float m = s[0][0];
#pragma unroll
    for (int n = 0; n < kKeys / 32; ++n)
#pragma unroll
      for (int r = 0; r < 16; ++r) m = fmaxf(m, s[n][r]);
    m = fmaxf(m, other_half(m));
    // the sums stay relative to an earlier maximum until one grows past it by
    // a factor of 2^8: the exponentials stay below 2^8, far from fp32's range
    if (__any(m > top + 8.0f || (top == -INFINITY && m > top))) {
      const float t = fmaxf(top, m);
      const float keep = top == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(top - t);
      top = t;
      sum *= keep;
#pragma unroll
      for (int d = 0; d < TL::kDT; ++d) o[d] *= keep;
    }
    const float base = top == -INFINITY ? 0.0f : top;
    Column<T> pc[kKeys / 32];
#pragma unroll
    for (int n = 0; n < kKeys / 32; ++n) {
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        s[n][r] = __builtin_amdgcn_exp2f(s[n][r] - base);
        sum += s[n][r];
      }
      pc[n].set(s[n]);
    }
#pragma unroll
    for (int n = 0; n < kKeys / 32; ++n)
#pragma unroll
      for (int d = 0; d < TL::kDT; ++d) o[d] = mma_transposed<DP>(vt, 32 * n, d, pc[n], o[d]);
  }
  sum += other_half(sum);
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
  bool bad = false;
#pragma unroll
  for (int d = 0; d < TL::kDT; ++d) {
#pragma unroll
    for (int r = 0; r < 16; ++r) bad |= not_finite(o[d][r]);
    store_column<T>(a.o, q0 + row, head, a.head_dim, d, o[d], inv, in);
  }
  if (in && half == 0)
    a.lse[(q0 + row) * a.n_heads + head] = (top + __builtin_amdgcn_logf(sum)) * 0.69314718055994530942f;
  // A NaN or an infinity may have come from a value row that the query does
  // not see (its zero weight times it): such rows are done again one by one.
  uint64_t again = __ballot(bad && in);
  again = (again | (again >> 32)) & 0xffffffffull;
  while (again) {
    const int i = __builtin_ctzll(again);
    again &= again - 1;
    attn_fwd_row<T>(a, q0 + wq + i, head, past + wq + i, k0);
  }
}

template <typename T, int DP>
static hipError_t fwd_launch(const AttnView& a, hipStream_t s, int* err) {
  constexpr int kNW = 4;
  constexpr int kKeys = sizeof(T) == 2 ? 64 : 32;
  constexpr size_t kLds = size_t(4) * kKeys * Tile<T, DP>::kRow;
  const int64_t n = slots(a.total_q, a.n_seqs, 32 * kNW);
  attn_fwd_kernel<T, DP, kNW><<<static_cast<unsigned>(n * a.n_heads), 64 * kNW, kLds, s>>>(a, n, err);
  return hipGetLastError();
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

// The queries [begin, end) of a sequence that see key j.
__device__ __forceinline__ void seeing_queries(const AttnView& a, int64_t j, int64_t past, int64_t nq, int64_t* begin,
                                               int64_t* end) {
  *begin = j > past ? j - past : 0;
  *end = nq;
  if (a.window > 0 && j >= a.sinks && j + a.window - past < nq) *end = j + a.window - past;
}

// One key's rows of dk and dv, by a whole wave.
template <typename T>
__device__ __forceinline__ void attn_dkv_row(const AttnView& a, const float* delta, int64_t j, int64_t hk, int64_t q0,
                                             int64_t nq, int64_t k0, int64_t nk) {
  const Row2 k = load_row<T>(a.k, k0 + j, hk, a.head_dim), v = load_row<T>(a.v, k0 + j, hk, a.head_dim);
  Row2 dk{{0.0f, 0.0f}}, dv{{0.0f, 0.0f}};
  int64_t i0, i1;
  seeing_queries(a, j, nk - nq, nq, &i0, &i1);
  for (int64_t g = 0; g < a.group; ++g) {
    const int64_t h = hk * a.group + g;
    for (int64_t i = i0; i < i1; ++i) {
      const Row2 q = load_row<T>(a.q, q0 + i, h, a.head_dim);
      const Row2 d_o = load_row<T>(a.d_o, q0 + i, h, a.head_dim);
      const float pr = __expf(dot(q, k) * a.scale - a.lse[(q0 + i) * a.n_heads + h]);
      const float ds = pr * (dot(d_o, v) - delta[h * a.total_q + q0 + i]);
      dk.x[0] += ds * q.x[0];
      dk.x[1] += ds * q.x[1];
      dv.x[0] += pr * d_o.x[0];
      dv.x[1] += pr * d_o.x[1];
    }
  }
  dk.x[0] *= a.scale;
  dk.x[1] *= a.scale;
  store_row<T>(a.dk, k0 + j, hk, a.head_dim, dk);
  store_row<T>(a.dv, k0 + j, hk, a.head_dim, dv);
}

// dq, and for the other kernel lse2 = lse in powers of two (0 where no key is
// seen) and delta, both [n_heads][total_q].
template <typename T, int DP, int NW>
__global__ __launch_bounds__(64 * NW, sizeof(T) == 2 ? 2 : 1) void attn_dq_kernel(AttnView a, int64_t n_slots, float* lse2_out,
                                                                                  float* delta_out, int* err) {
  using TL = Tile<T, DP>;
  constexpr int kKeys = sizeof(T) == 2 ? 64 : 32;
  constexpr int kTile = kKeys * TL::kRow;
  extern __shared__ __align__(1024) char smem[];
  lds_char* const lds = (lds_char*)smem;
  check_offsets(a, err);
  const Work wk = work_of(n_slots, a.n_heads);
  const TileOf tile = tile_of_slot(a.cu_q, a.n_seqs, 32 * NW, wk.slot);
  if (tile.seq < 0) return;
  int64_t q0, q1, k0, k1;
  seq_rows(a.cu_q, tile.seq, a.total_q, &q0, &q1, err);
  seq_rows(a.cu_k, tile.seq, a.total_k, &k0, &k1, err);
  const int64_t nq = q1 - q0, nk = k1 - k0, past = nk - nq;
  if (tile.first >= nq) return;
  const int lane = threadIdx.x & 63, half = lane >> 5;
  const int head = wk.head, hk = head / a.group;
  const int64_t wq = tile.first + 32 * (threadIdx.x >> 6);
  const int64_t row = wq + (lane & 31);
  const bool in = row < nq;
  const int64_t p = past + row;
  const int64_t p_min = past + wq, p_max = past + (wq + 31 < nq ? wq + 31 : nq - 1);
  const bool wave_in = wq < nq && p_max >= 0;
  const KeyTiles keys(a, past + tile.first, past + (tile.first + 32 * NW < nq ? tile.first + 32 * NW : nq) - 1, kKeys);
  TileLoader<T, DP, kKeys, NW> kl, vl;
  kl.init(a.k, k0, hk, a.head_dim);
  vl.init(a.v, k0, hk, a.head_dim);
  if (keys.n > 0) {
    kl.load(keys.first(0), nk, lds);
    vl.load(keys.first(0), nk, lds + kTile);
  }
  u32x4_t qf[TL::kSteps], dof[TL::kSteps];
  float delta = 0.0f;
#pragma unroll
  for (int s = 0; s < TL::kSteps; ++s) {
    qf[s] = load_frag<T>(a.q, q0 + row, head, a.head_dim, s, in);
    dof[s] = load_frag<T>(a.d_o, q0 + row, head, a.head_dim, s, in);
    delta += dot_frag(dof[s], load_frag<T>(a.o, q0 + row, head, a.head_dim, s, in), T{});
  }
  delta += other_half(delta);
  const float lse = in ? a.lse[(q0 + row) * a.n_heads + head] : 0.0f;
  const float lse2 = lse == -INFINITY ? 0.0f : lse * 1.44269504088896340736f;
  if (in && half == 0) {
    lse2_out[head * a.total_q + q0 + row] = lse2;
    delta_out[head * a.total_q + q0 + row] = delta;
  }
  const float c = a.scale * 1.44269504088896340736f;
  f32x16_t dq[TL::kDT] = {};
  for (int64_t it = 0; it < keys.n; ++it) {
    wait_vmcnt<0>();
    lds_barrier();
    const lds_char* kt = lds + (it & 1) * 2 * kTile;
    const lds_char* vt = kt + kTile;
    if (it + 1 < keys.n) {
      lds_char* next = lds + ((it + 1) & 1) * 2 * kTile;
      kl.load(keys.first(it + 1), nk, next);
      vl.load(keys.first(it + 1), nk, next + kTile);
    }
    const int64_t key = keys.first(it);
    if (!wave_in || none_visible(a, p_min, p_max, key, kKeys)) continue;
    const bool all = wq + 31 < nq && all_visible(a, p_min, p_max, key, kKeys);
#pragma unroll
    for (int n = 0; n < kKeys / 32; ++n) {
      f32x16_t s = {}, dp = {};
#pragma unroll
      for (int st = 0; st < TL::kSteps; ++st) {
        s = mma16(TL::row_frag(kt, 32 * n, st), qf[st], s, T{});
        dp = mma16(TL::row_frag(vt, 32 * n, st), dof[st], dp, T{});
      }
#pragma unroll
      for (int r = 0; r < 16; ++r) s[r] = __builtin_amdgcn_exp2f(fmaf(s[r], c, -lse2)) * (dp[r] - delta);
      if (!all) {
        const SeenKeys seen(a, p, in, key);
#pragma unroll
        for (int r = 0; r < 16; ++r) s[r] = seen(32 * n + 8 * (r >> 2) + (r & 3)) ? s[r] : 0.0f;
      }
      Column<T> ds;
      ds.set(s);
#pragma unroll
      for (int d = 0; d < TL::kDT; ++d) dq[d] = mma_transposed<DP>(kt, 32 * n, d, ds, dq[d]);
    }
  }
  bool bad = false;
#pragma unroll
  for (int d = 0; d < TL::kDT; ++d) {
#pragma unroll
    for (int r = 0; r < 16; ++r) bad |= not_finite(dq[d][r]);
    store_column<T>(a.dq, q0 + row, head, a.head_dim, d, dq[d], a.scale, in);
  }
  // a hidden key's rows may have brought it (zero times them): see the forward
  uint64_t again = __ballot(bad && in);
  again = (again | (again >> 32)) & 0xffffffffull;
  while (again) {
    const int i = __builtin_ctzll(again);
    again &= again - 1;
    attn_dq_row<T>(a, q0 + wq + i, head, past + wq + i, k0);
  }
}

// dk and dv: one key a column, 32 a wave; the queries that see them (of every
// head of the group) go through LDS.
template <typename T, int DP, int NW>
__global__ __launch_bounds__(64 * NW, 1) void attn_dkv_kernel(AttnView a, int64_t n_slots, const float* lse2_in,
                                                              const float* delta_in, int* err) {
  using TL = Tile<T, DP>;
  constexpr int kRows = sizeof(T) == 2 ? 64 : 32;      // queries per tile
  constexpr int kTile = kRows * TL::kRow;
  constexpr int kStage = 2 * kTile + 512;              // Q, dO, lse2 [64], delta [64]
  extern __shared__ __align__(1024) char smem[];
  lds_char* const lds = (lds_char*)smem;
  const Work wk = work_of(n_slots, a.n_kv_heads);
  const TileOf tile = tile_of_slot(a.cu_k, a.n_seqs, 32 * NW, n_slots - 1 - wk.slot);
  if (tile.seq < 0) return;
  int64_t q0, q1, k0, k1;
  seq_rows(a.cu_q, tile.seq, a.total_q, &q0, &q1, err);
  seq_rows(a.cu_k, tile.seq, a.total_k, &k0, &k1, err);
  const int64_t nq = q1 - q0, nk = k1 - k0, past = nk - nq;
  if (tile.first >= nk) return;
  const int lane = threadIdx.x & 63;
  const int hk = wk.head;
  const int64_t wkey = tile.first + 32 * (threadIdx.x >> 6);   // the wave's first key
  const int64_t key = wkey + (lane & 31);
  const bool in = key < nk;
  u32x4_t kf[TL::kSteps], vf[TL::kSteps];
#pragma unroll
  for (int s = 0; s < TL::kSteps; ++s) {
    kf[s] = load_frag<T>(a.k, k0 + key, hk, a.head_dim, s, in);
    vf[s] = load_frag<T>(a.v, k0 + key, hk, a.head_dim, s, in);
  }
  const float c = a.scale * 1.44269504088896340736f;

  // query tiles that see some key of the workgroup
  const int64_t last_key = (tile.first + 32 * NW < nk ? tile.first + 32 * NW : nk) - 1;
  const int64_t i_lo = tile.first > past ? tile.first - past : 0;
  int64_t i_hi = nq;
  if (a.window > 0 && tile.first >= a.sinks && last_key + a.window - past < nq) i_hi = last_key + a.window - past;
  const int64_t t_lo = i_lo / kRows, per_head = i_hi > i_lo ? (i_hi + kRows - 1) / kRows - t_lo : 0;
  const int64_t n_it = per_head * a.group;

  TileLoader<T, DP, kRows, NW> ql, dl;
  auto load = [&](int64_t it, lds_char* to) {
    const int64_t h = static_cast<int64_t>(hk) * a.group + it / per_head, first = (t_lo + it % per_head) * kRows;
    ql.init(a.q, q0, h, a.head_dim);
    dl.init(a.d_o, q0, h, a.head_dim);
    ql.load(first, nq, to);
    dl.load(first, nq, to + kTile);
    const int w = threadIdx.x >> 6;
    if (w < 2) {
      const int64_t i = first + lane < nq ? first + lane : nq - 1;
      dma4((w ? delta_in : lse2_in) + h * a.total_q + q0 + i, static_cast<lds_void*>(to + 2 * kTile + 256 * w));
    }
  };
  f32x16_t dk[TL::kDT] = {}, dv[TL::kDT] = {};
  if (n_it > 0) load(0, lds);
  for (int64_t it = 0; it < n_it; ++it) {
    wait_vmcnt<0>();
    lds_barrier();
    const lds_char* qt = lds + (it & 1) * kStage;
    const lds_char* dot = qt + kTile;
    if (it + 1 < n_it) load(it + 1, lds + ((it + 1) & 1) * kStage);
    const int64_t first = (t_lo + it % per_head) * kRows;
#pragma unroll
    for (int n = 0; n < kRows / 32; ++n) {
      const int64_t i0 = first + 32 * n;                       // queries i0 .. i0 + 31, at these positions
      const int64_t p_min = past + i0, p_max = past + (i0 + 31 < nq ? i0 + 31 : nq - 1);
      if (wkey >= nk || i0 >= nq || none_visible(a, p_min, p_max, wkey, 32)) continue;
      const bool all = i0 + 31 < nq && wkey + 31 < nk && all_visible(a, p_min, p_max, wkey, 32);
      f32x16_t s = {}, dp = {};
#pragma unroll
      for (int st = 0; st < TL::kSteps; ++st) {
        s = mma16(TL::row_frag(qt, 32 * n, st), kf[st], s, T{});
        dp = mma16(TL::row_frag(dot, 32 * n, st), vf[st], dp, T{});
      }
      const lds_char* stat = qt + 2 * kTile + (32 * n + 4 * (lane >> 5)) * 4;
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const f32x4_t l4 = *reinterpret_cast<const lds_f32x4*>(stat + 32 * g);
        const f32x4_t d4 = *reinterpret_cast<const lds_f32x4*>(stat + 256 + 32 * g);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int r = 4 * g + e;
          s[r] = __builtin_amdgcn_exp2f(fmaf(s[r], c, -l4[e]));
          dp[r] = s[r] * (dp[r] - d4[e]);
        }
      }
      if (!all) {
        const SeenBy seen(a, key, in, past + i0, i0, nq);
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const bool yes = seen(8 * (r >> 2) + (r & 3));
          s[r] = yes ? s[r] : 0.0f;
          dp[r] = yes ? dp[r] : 0.0f;
        }
      }
      Column<T> pc, ds;
      pc.set(s);
      ds.set(dp);
#pragma unroll
      for (int d = 0; d < TL::kDT; ++d) {
        dv[d] = mma_transposed<DP>(dot, 32 * n, d, pc, dv[d]);
        dk[d] = mma_transposed<DP>(qt, 32 * n, d, ds, dk[d]);
      }
    }
  }
  bool bad = false;
#pragma unroll
  for (int d = 0; d < TL::kDT; ++d) {
#pragma unroll
    for (int r = 0; r < 16; ++r) bad |= not_finite(dk[d][r]) || not_finite(dv[d][r]);
    store_column<T>(a.dk, k0 + key, hk, a.head_dim, d, dk[d], a.scale, in);
    store_column<T>(a.dv, k0 + key, hk, a.head_dim, d, dv[d], 1.0f, in);
  }
  // a query that does not see the key may have brought it: see the forward
  uint64_t again = __ballot(bad && in);
  again = (again | (again >> 32)) & 0xffffffffull;
  while (again) {
    const int i = __builtin_ctzll(again);
    again &= again - 1;
    attn_dkv_row<T>(a, delta_in, wkey + i, hk, q0, nq, k0, nk);
  }
}

hipError_t launch_attn_fwd(const AttnView& a, int dtype, hipStream_t s, int* err) {
  if (dtype == STAPLE_BF16)
    return a.head_dim <= 64 ? fwd_launch<bf16_t, 64>(a, s, err) : fwd_launch<bf16_t, 128>(a, s, err);
  return a.head_dim <= 64 ? fwd_launch<float, 64>(a, s, err) : fwd_launch<float, 128>(a, s, err);
}

size_t attn_bwd_workspace_bytes(const AttnView& a, int) {
  return 2 * align_up(static_cast<size_t>(a.total_q) * a.n_heads * sizeof(float), 256);
}

template <typename T, int DP>
static hipError_t bwd_launch(const AttnView& a, void* ws, hipStream_t s, int* err) {
  constexpr int kNW = 4;
  constexpr int kRows = sizeof(T) == 2 ? 64 : 32;
  constexpr size_t kLds = size_t(4) * kRows * Tile<T, DP>::kRow;
  Workspace w(ws, attn_bwd_workspace_bytes(a, 0));
  const size_t bytes = static_cast<size_t>(a.total_q) * a.n_heads * sizeof(float);
  float* lse2 = w.take<float>(bytes);
  float* delta = w.take<float>(bytes);
  const int64_t nq = slots(a.total_q, a.n_seqs, 32 * kNW), nk = slots(a.total_k, a.n_seqs, 32 * kNW);
  attn_dq_kernel<T, DP, kNW><<<static_cast<unsigned>(nq * a.n_heads), 64 * kNW, kLds, s>>>(a, nq, lse2, delta, err);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  // more than the 64 KB of LDS that a launch gets unasked
  const auto dkv = attn_dkv_kernel<T, DP, kNW>;
  static const hipError_t attr = hipFuncSetAttribute(reinterpret_cast<const void*>(dkv),
                                                     hipFuncAttributeMaxDynamicSharedMemorySize, kLds + 1024);
  if (attr != hipSuccess) return attr;
  dkv<<<static_cast<unsigned>(nk * a.n_kv_heads), 64 * kNW, kLds + 1024, s>>>(a, nk, lse2, delta, err);
  return hipGetLastError();
}

hipError_t launch_attn_bwd(const AttnView& a, int dtype, void* ws, hipStream_t s, int* err) {
  if (dtype == STAPLE_BF16)
    return a.head_dim <= 64 ? bwd_launch<bf16_t, 64>(a, ws, s, err) : bwd_launch<bf16_t, 128>(a, ws, s, err);
  return a.head_dim <= 64 ? bwd_launch<float, 64>(a, ws, s, err) : bwd_launch<float, 128>(a, ws, s, err);
}

}  // namespace staple
