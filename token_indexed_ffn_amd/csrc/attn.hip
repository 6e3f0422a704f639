// Attention over packed sequences with a causal mask, a sliding window and
// sinks: forward and backward.
#include "attn_row.h"
#include "attn_tile.h"

namespace staple {

constexpr int kRowWaves = 4;

// The sequence that packed row t belongs to, or -1.
__device__ __forceinline__ int64_t seq_of_row(const int32_t* cu, int64_t n_seqs, int64_t t) {
  int64_t lo = 0, hi = n_seqs;   // cu[lo] <= t < cu[hi], where such entries exist
  while (hi - lo > 1) {
    const int64_t mid = (lo + hi) >> 1;
    if (cu[mid] <= t) lo = mid;
    else hi = mid;
  }
  return cu[lo] <= t && t < cu[lo + 1] ? lo : -1;
}

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

  // key tiles that some query of the workgroup sees: those of the sinks, then
  // the window's
  const int64_t g_max = past + (tile.first + 32 * NW < nq ? tile.first + 32 * NW : nq) - 1;
  const int64_t g_lo = a.window > 0 && past + tile.first >= a.window ? past + tile.first - a.window + 1 : 0;
  const int64_t t_lo = g_lo / kKeys, t_end = g_max < 0 ? t_lo : g_max / kKeys + 1;
  const int64_t sink_keys = a.sinks < t_lo * kKeys ? a.sinks : t_lo * kKeys;
  const int64_t n_sink = g_max < 0 ? 0 : (sink_keys + kKeys - 1) / kKeys;
  const int64_t n_it = n_sink + (t_end - t_lo);

  TileLoader<T, DP, kKeys, NW> kl, vl;
  kl.init(a.k, k0, hk, a.head_dim);
  vl.init(a.v, k0, hk, a.head_dim);
  f32x16_t o[TL::kDT] = {};
  float top = -INFINITY, sum = 0.0f;   // of the lane's column; sum: this half-wave's keys
  auto key_of = [&](int64_t it) { return (it < n_sink ? it : t_lo + it - n_sink) * kKeys; };
  if (n_it > 0) {
    kl.load(key_of(0), nk, lds);
    vl.load(key_of(0), nk, lds + kTile);
  }
  for (int64_t it = 0; it < n_it; ++it) {
    wait_vmcnt<0>();
    lds_barrier();
    const lds_char* kt = lds + (it & 1) * 2 * kTile;
    const lds_char* vt = kt + kTile;
    if (it + 1 < n_it) {
      lds_char* next = lds + ((it + 1) & 1) * 2 * kTile;
      kl.load(key_of(it + 1), nk, next);
      vl.load(key_of(it + 1), nk, next + kTile);
    }
    const int64_t key = key_of(it);
    const int64_t last = key + kKeys - 1;
    if (!wave_in || key > p_max || (a.window > 0 && last <= p_min - a.window && key >= a.sinks)) continue;
    const bool all = last <= p_min && wq + 31 < nq && (a.window == 0 || key > p_max - a.window || last < a.sinks);
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
      const int hi = in ? clamp_rel(p - key - 4 * half) : -(1 << 20);
      const int lo = a.window > 0 ? clamp_rel(p - a.window + 1 - key - 4 * half) : -(1 << 20);
      const int sk = clamp_rel(a.sinks - key - 4 * half);
#pragma unroll
      for (int n = 0; n < kKeys / 32; ++n)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const int j = 32 * n + 8 * (r >> 2) + (r & 3);
          if (!(j <= hi && (j >= lo || j < sk))) s[n][r] = -INFINITY;
        }
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

template <typename T>
__global__ __launch_bounds__(64 * kRowWaves) void attn_dq_row_kernel(AttnView a, float* delta, int* err) {
  check_offsets(a, err);
  const int64_t w = static_cast<int64_t>(blockIdx.x) * kRowWaves + (threadIdx.x >> 6);
  if (w >= a.total_q * a.n_heads) return;
  const int64_t t = w / a.n_heads, h = w % a.n_heads, hk = h / a.group;
  const int64_t b = seq_of_row(a.cu_q, a.n_seqs, t);
  if (b < 0) return;
  int64_t q0, q1, k0, k1;
  seq_rows(a.cu_q, b, a.total_q, &q0, &q1, err);
  seq_rows(a.cu_k, b, a.total_k, &k0, &k1, err);
  const int64_t p = (t - q0) + (k1 - k0) - (q1 - q0);
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
  if ((threadIdx.x & 63) == 0) delta[t * a.n_heads + h] = dl;
}

template <typename T>
__global__ __launch_bounds__(64 * kRowWaves) void attn_dkv_row_kernel(AttnView a, const float* delta, int* err) {
  const int64_t w = static_cast<int64_t>(blockIdx.x) * kRowWaves + (threadIdx.x >> 6);
  if (w >= a.total_k * a.n_kv_heads) return;
  const int64_t t = w / a.n_kv_heads, hk = w % a.n_kv_heads;
  const int64_t b = seq_of_row(a.cu_k, a.n_seqs, t);
  if (b < 0) return;
  int64_t q0, q1, k0, k1;
  seq_rows(a.cu_q, b, a.total_q, &q0, &q1, err);
  seq_rows(a.cu_k, b, a.total_k, &k0, &k1, err);
  const int64_t past = (k1 - k0) - (q1 - q0), j = t - k0;
  const Row2 k = load_row<T>(a.k, t, hk, a.head_dim), v = load_row<T>(a.v, t, hk, a.head_dim);
  Row2 dk{{0.0f, 0.0f}}, dv{{0.0f, 0.0f}};
  const int64_t i0 = j > past ? j - past : 0;
  int64_t i1 = q1 - q0;
  if (a.window > 0 && j >= a.sinks && j + a.window - past < i1) i1 = j + a.window - past;
  for (int64_t g = 0; g < a.group; ++g) {
    const int64_t h = hk * a.group + g;
    for (int64_t i = i0; i < i1; ++i) {
      const Row2 q = load_row<T>(a.q, q0 + i, h, a.head_dim);
      const Row2 d_o = load_row<T>(a.d_o, q0 + i, h, a.head_dim);
      const int64_t at = (q0 + i) * a.n_heads + h;
      const float pr = __expf(dot(q, k) * a.scale - a.lse[at]);
      const float ds = pr * (dot(d_o, v) - delta[at]);
      dk.x[0] += ds * q.x[0];
      dk.x[1] += ds * q.x[1];
      dv.x[0] += pr * d_o.x[0];
      dv.x[1] += pr * d_o.x[1];
    }
  }
  dk.x[0] *= a.scale;
  dk.x[1] *= a.scale;
  store_row<T>(a.dk, t, hk, a.head_dim, dk);
  store_row<T>(a.dv, t, hk, a.head_dim, dv);
}

static unsigned row_wgs(int64_t rows) { return static_cast<unsigned>((rows + kRowWaves - 1) / kRowWaves); }

hipError_t launch_attn_fwd(const AttnView& a, int dtype, hipStream_t s, int* err) {
  if (dtype == STAPLE_BF16)
    return a.head_dim <= 64 ? fwd_launch<bf16_t, 64>(a, s, err) : fwd_launch<bf16_t, 128>(a, s, err);
  return a.head_dim <= 64 ? fwd_launch<float, 64>(a, s, err) : fwd_launch<float, 128>(a, s, err);
}

size_t attn_bwd_workspace_bytes(const AttnView& a, int dtype) {
  return align_up(static_cast<size_t>(a.total_q) * a.n_heads * sizeof(float), 256);
}

hipError_t launch_attn_bwd(const AttnView& a, int dtype, void* ws, hipStream_t s, int* err) {
  float* delta = static_cast<float*>(ws);
  const unsigned wq = row_wgs(a.total_q * a.n_heads), wk = row_wgs(a.total_k * a.n_kv_heads);
  if (wq) {
    if (dtype == STAPLE_BF16) attn_dq_row_kernel<bf16_t><<<wq, 64 * kRowWaves, 0, s>>>(a, delta, err);
    else attn_dq_row_kernel<float><<<wq, 64 * kRowWaves, 0, s>>>(a, delta, err);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (wk) {
    if (dtype == STAPLE_BF16) attn_dkv_row_kernel<bf16_t><<<wk, 64 * kRowWaves, 0, s>>>(a, delta, err);
    else attn_dkv_row_kernel<float><<<wk, 64 * kRowWaves, 0, s>>>(a, delta, err);
  }
  return hipGetLastError();
}

}  // namespace staple
