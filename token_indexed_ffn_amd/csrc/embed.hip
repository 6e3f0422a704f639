// Embedding lookup with scaling, and its gradient by sorted tokens.
//
//   y_i = scale E[t_i],    dE_t = scale sum over the positions i with t_i = t of dy_i.
//
// Both are bound by bytes: the rows of distinct tokens and the output, the gradients and a row in fp32 for each
// distinct token.  32768 positions, 7700 distinct, of 2048 in bf16: 41 us (4.0 TB/s) and, with the join of
// cut tokens, 49 (4.1 TB/s), from rows in fp32 75 (4.4 TB/s).
#include "model_ops.h"
#include "row_io.h"

namespace staple {

constexpr int kEmbedCols = 512;     // 64 lanes x 8 columns
constexpr int kEmbedAhead = 8;      // rows in flight a lane

// One wave writes U blocks of 512 columns of one token's row: four where that leaves waves enough to fill the
// GPU, whose loads are then in flight together (32768 x 2048: 41 us, one block a wave 46), otherwise one (64 x
// 2048: 2.9 us, four 3.3 to 5.4).
template <typename E, typename O, Layout LAYOUT, int U>
__global__ __launch_bounds__(256) void embed_fwd_kernel(const E* __restrict__ table, int64_t vocab, int d,
                                                        const int32_t* __restrict__ ids, int64_t n,
                                                        float scale, O* __restrict__ y, int64_t y_stride,
                                                        int blocks, int* err) {
  using R = RowGroup<64, LAYOUT>;
  const int lane = threadIdx.x & 63;
  const int64_t items = n * blocks;
  for (int64_t w = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6); w < items;
       w += static_cast<int64_t>(gridDim.x) * 4) {
    const int64_t i = w / blocks;
    const int g0 = static_cast<int>(w - i * blocks) * U;
    const int32_t t = ids[i];
    const bool fine = t >= 0 && t < vocab;
    if (!fine && lane == 0 && g0 == 0) flag_index_error(err);
    float v[U][8];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (fine) {
        R::load(table + static_cast<int64_t>(t) * d, g0 + u, lane, d, v[u]);
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) v[u][k] = 0.0f;
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int k = 0; k < 8; ++k) v[u][k] *= scale;
      R::store(y + i * y_stride, g0 + u, lane, d, v[u]);
    }
  }
}

static bool vec_rows(const void* p, int64_t stride, int bytes) {
  return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && stride * bytes % 16 == 0;
}

template <typename E, typename O>
static void embed_fwd(const void* table, int64_t vocab, int d, const int32_t* ids, int64_t n, float scale,
                      RowsView y, hipStream_t s, int* err) {
  const bool aligned = d % 8 == 0 && vec_rows(table, d, sizeof(E)) && vec_rows(y.data, y.stride, sizeof(O));
  const int groups = (d + kEmbedCols - 1) / kEmbedCols;
  const E* tab = static_cast<const E*>(table);
  O* out = reinterpret_cast<O*>(y.data);
  const bool wide = groups >= 4 && n * groups > 16384;
  const int blocks = wide ? (groups + 3) / 4 : groups;
  const int64_t wgs = (n * blocks + 3) / 4;
  const dim3 grid(static_cast<unsigned>(wgs < (1 << 20) ? wgs : (1 << 20)));
#define GO(V, U) embed_fwd_kernel<E, O, V, U><<<grid, dim3(256), 0, s>>>(tab, vocab, d, ids, n, scale, out, y.stride, blocks, err)
  if (aligned) {
    if (wide) GO(kAligned, 4); else GO(kAligned, 1);
  } else if (d >= 8) {
    if (wide) GO(kLoose, 4); else GO(kLoose, 1);
  } else {
    GO(kSingle, 1);
  }
#undef GO
}

hipError_t launch_embed_fwd(const void* table, int64_t vocab, int64_t d, int32_t dtype, const int32_t* ids,
                            int64_t n, float scale, RowsView y, int32_t out_dtype, hipStream_t s, int* err) {
  const int dim = static_cast<int>(d);
  if (dtype == STAPLE_BF16) {
    if (out_dtype == STAPLE_BF16) embed_fwd<bf16_t, bf16_t>(table, vocab, dim, ids, n, scale, y, s, err);
    else embed_fwd<bf16_t, float>(table, vocab, dim, ids, n, scale, y, s, err);
  } else {
    if (out_dtype == STAPLE_BF16) embed_fwd<float, bf16_t>(table, vocab, dim, ids, n, scale, y, s, err);
    else embed_fwd<float, float>(table, vocab, dim, ids, n, scale, y, s, err);
  }
  return hipGetLastError();
}

// ------------------------------------------------------------------------------- gradient
// One token can hold half of a batch, so the sorted positions, not the tokens, are dealt out: a wave sums
// the runs of equal tokens within a chunk of kChunk positions, for 512 columns.  A run that is a whole
// token's goes to its row.  The parts of one that a chunk's border cuts meet in LDS, and where the run is
// cut by the border of the workgroup's kSpan positions too, in first[span] (begun in an earlier span) or
// last[span] (goes on in the next): the second kernel adds last[s0], first[s0 + 1], ..., first[s1], where
// they are many eight waves an eighth of them each and the eighths in turn.  The order is fixed, and the
// result does not change from run to run.
// Without LDS, chunks of 32 took 49 and the join 10 us for 32768 x 2048, of 8 42 and 19; 30000 x 300, of which
// 60% are one token, took 39 and 60 us, where it now takes 19.
constexpr int kChunk = 8;                    // as many rows as a lane has in flight: sixteen spill
constexpr int kChunks = 8;                   // of a workgroup: one a wave
constexpr int kSpan = kChunk * kChunks;
constexpr int kJoinWaves = 8;

// Eight elements of a row; columns past d repeat the last ones: no branch around any load (the sums of such
// columns are stored nowhere).
template <Layout LAYOUT, bool ONCE, typename E>
__device__ __forceinline__ void load_row(const E* row, int g, int lane, int d, float (&v)[8]) {
  using R = RowGroup<64, LAYOUT>;
  if (LAYOUT == kSingle) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = load1(row + min(R::column(g, lane, i), d - 1));
    return;
  }
  const E* p = row + min(R::column(g, lane, 0), d - 8);
  Raw<E> raw;
  if (LAYOUT == kAligned) {
    if (ONCE) raw.load_once(p);
    else raw.load(p);
  } else {
    if (ONCE) raw.load_loose_once(p);
    else raw.load_loose(p);
  }
  raw.get(v);
}

// Unique index of sorted position p, -1 where the maps are out of range.
__device__ __forceinline__ int32_t unique_of(int64_t p, int64_t n, int64_t nu, const int32_t* sorted_pos,
                                             const int32_t* inv, int32_t& row) {
  row = sorted_pos[p];
  if (row < 0 || row >= n) return row = -1;
  const int32_t u = inv[row];
  return u >= 0 && u < nu ? u : -1;
}

// Row of grad of unique token u, NULL (and the error word) where it is out of range.
__device__ __forceinline__ float* grad_row(const EmbedGrad& a, int32_t u, int lane, int* err) {
  int64_t r = -1;
  if (u >= 0) r = a.uniq ? a.uniq[u] : u;
  if (r < 0 || r >= a.grad_rows) {
    if (lane == 0) flag_index_error(err);
    return nullptr;
  }
  return a.grad + r * a.d;
}

template <Layout LAYOUT>
__device__ __forceinline__ void finish(const EmbedGrad& a, float* row, int g, int lane, float (&acc)[8]) {
  using R = RowGroup<64, LAYOUT>;
  const int d = static_cast<int>(a.d);
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[i] *= a.scale;
  if (a.accumulate) {
    float old[8];
    R::load(row, g, lane, d, old);
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] += old[i];
  }
  R::store(row, g, lane, d, acc);
}

template <typename E, Layout LAYOUT>
__global__ __launch_bounds__(64 * kChunks) void embed_bwd_kernel(EmbedGrad a, int groups, float* __restrict__ first,
                                                                 float* __restrict__ last, int64_t ld, int* err) {
  using R = RowGroup<64, LAYOUT>;
  // the sums of a chunk's run that began before it, and of the one that goes on after it
  __shared__ float begun_sum[kChunks][kEmbedCols], open_sum[kChunks][kEmbedCols];
  __shared__ bool ended[kChunks];              // whether the former ends in the chunk
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t n = a.n_tokens;
  int64_t nu = *a.n_unique;
  if (nu < 0 || nu > a.max_unique) {
    if (lane == 0) flag_index_error(err);
    return;
  }
  nu = nu < n ? nu : n;
  const int64_t span = blockIdx.x / groups;
  const int g = static_cast<int>(blockIdx.x - span * groups);
  const int d = static_cast<int>(a.d);
  const int64_t p0 = span * kSpan + wave * kChunk;
  const int len = static_cast<int>(max(int64_t(0), min(n - p0, int64_t(kChunk))));
  // lane i: position p0 + i; the lane after the last one and lane 63: the neighbours outside
  int32_t row = -1, u = -2;
  const int64_t p = lane == 63 ? p0 - 1 : p0 + lane;
  if (len > 0 && (lane <= len || lane == 63) && p >= 0 && p < n) {
    u = unique_of(p, n, nu, a.sorted_pos, a.inv, row);
    if (u < 0 && lane < len) flag_index_error(err);
  }
  const int32_t next = __shfl(u, lane < 62 ? lane + 1 : 62, 64);
  const uint64_t ends = __ballot(lane < len && u != next);   // a run's last position
  const bool begun = len > 0 && __shfl(u, 63, 64) == __shfl(u, 0, 64);
  const bool open = len > 0 && !(ends >> (len - 1) & 1) && !(begun && ends == 0);
  float acc[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
  if (len > 0) {
    float v[kChunk][8];
#pragma unroll
    for (int j = 0; j < kChunk; ++j) {
      const int32_t r = __builtin_amdgcn_readlane(row, min(j, len - 1));
      // a position out of range: row 0, in a run whose sum is stored nowhere
      // (read past the caches: 32768 rows of 2048 that are not in them take 41 us, through them 54; ones that
      // were just written take 41 and 31)
      load_row<LAYOUT, true>(reinterpret_cast<const E*>(a.dy.data) + (r >= 0 ? r : 0) * a.dy.stride, g, lane, d, v[j]);
    }
    bool first_run = begun;
#pragma unroll
    for (int k = 0; k < kChunk; ++k) {
      if (k >= len) break;
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] += v[k][i];
      const bool end = (ends >> k) & 1;
      if (!end && k + 1 < len) continue;
      if (first_run || !end) {
        float* to = first_run ? begun_sum[wave] : open_sum[wave];
#pragma unroll
        for (int i = 0; i < 8; ++i) to[i * 64 + lane] = acc[i];
      } else {
        float* to = grad_row(a, __builtin_amdgcn_readlane(u, k), lane, err);
        if (to) finish<LAYOUT>(a, to, g, lane, acc);
      }
      first_run = false;
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] = 0.0f;
    }
  }
  if (lane == 0) ended[wave] = ends != 0;
  // the maps agree, also where no border asks for a token's first and last position
  if (g == 0 && lane < len && u >= 0) {
    const int64_t begin = a.seg_start[u], end = a.seg_start[u + 1];
    if (begin < 0 || begin > p || end <= p || end > n) flag_index_error(err);
  }
  __syncthreads();
  // a cut run's parts, from that of the chunk in which it begins, or of the span's first chunk
#pragma unroll 1
  for (int from_before = 0; from_before < 2; ++from_before) {
    if (from_before ? !(wave == 0 && begun) : !open) continue;
    const float(*parts)[kEmbedCols] = from_before ? begun_sum : open_sum;
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = parts[wave][i * 64 + lane];
    bool over = from_before && ended[0];
#pragma unroll 1
    for (int k = wave + 1; k < kChunks && !over; ++k) {
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] += begun_sum[k][i * 64 + lane];
      over = ended[k];
    }
    if (from_before) {
      R::store(first + span * ld, g, lane, d, acc);
    } else if (!over) {
      R::store(last + span * ld, g, lane, d, acc);
    } else {
      float* to = grad_row(a, __builtin_amdgcn_readlane(u, len - 1), lane, err);
      if (to) finish<LAYOUT>(a, to, g, lane, acc);
    }
  }
}

// The span in which a cut run begins adds its parts: part 0 is last[c], part k first[c + k].
template <Layout LAYOUT>
__device__ __forceinline__ void add_parts(const float* first, const float* last, int64_t ld, int64_t c, int64_t k0,
                                          int64_t k1, int g, int lane, int d, float (&acc)[8]) {
  for (int64_t b = k0; b < k1; b += kEmbedAhead) {
    float v[kEmbedAhead][8];
#pragma unroll
    for (int j = 0; j < kEmbedAhead; ++j) {
      const int64_t k = b + j < k1 ? b + j : k1 - 1;
      load_row<LAYOUT, false>(k == 0 ? last + c * ld : first + (c + k) * ld, g, lane, d, v[j]);
    }
#pragma unroll
    for (int j = 0; j < kEmbedAhead; ++j)
      if (b + j < k1) {
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] += v[j][i];
      }
  }
}

// A wave looks at one span (for 512 columns) and adds up to kEmbedAhead parts itself; runs of more are
// added by the whole workgroup.
template <Layout LAYOUT>
__global__ __launch_bounds__(64 * kJoinWaves) void embed_bwd_join_kernel(EmbedGrad a, int groups,
                                                                         const float* __restrict__ first,
                                                                         const float* __restrict__ last, int64_t ld,
                                                                         int* err) {
  __shared__ float part[kJoinWaves][512];
  __shared__ int64_t long_parts[kJoinWaves];
  __shared__ int32_t long_token[kJoinWaves];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t n = a.n_tokens;
  int64_t nu = *a.n_unique;
  if (nu < 0 || nu > a.max_unique) return;   // flagged by the first kernel
  nu = nu < n ? nu : n;
  const int64_t c0 = blockIdx.x / groups * kJoinWaves, c = c0 + wave;
  const int g = static_cast<int>(blockIdx.x % groups);
  const int d = static_cast<int>(a.d);
  const int64_t p0 = c * kSpan, p1 = p0 + kSpan;
  int64_t parts = 0;
  int32_t u = -1;
  if (p1 < n) {
    int32_t row;
    u = unique_of(p1 - 1, n, nu, a.sorted_pos, a.inv, row);
    const int32_t after = unique_of(p1, n, nu, a.sorted_pos, a.inv, row);
    if (u >= 0 && after == u) {
      const int64_t begin = a.seg_start[u], end = a.seg_start[u + 1];
      if (begin >= p1 || end <= p1 || end > n) {
        if (lane == 0) flag_index_error(err);
      } else if (begin >= p0) {
        parts = (end - 1) / kSpan - c + 1;
      }
    }
  }
  if (lane == 0) {
    long_parts[wave] = parts > kEmbedAhead ? parts : 0;
    long_token[wave] = u;
  }
  if (parts > 0 && parts <= kEmbedAhead) {
    float acc[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
    add_parts<LAYOUT>(first, last, ld, c, 0, parts, g, lane, d, acc);
    float* to = grad_row(a, u, lane, err);
    if (to) finish<LAYOUT>(a, to, g, lane, acc);
  }
  __syncthreads();
  for (int w = 0; w < kJoinWaves; ++w) {
    const int64_t all = long_parts[w];
    if (all == 0) continue;
    const int64_t each = (all + kJoinWaves - 1) / kJoinWaves;
    const int64_t k0 = wave * each, k1 = k0 + each < all ? k0 + each : all;
    float acc[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
    add_parts<LAYOUT>(first, last, ld, c0 + w, k0, k1, g, lane, d, acc);
#pragma unroll
    for (int i = 0; i < 8; ++i) part[wave][i * 64 + lane] = acc[i];
    __syncthreads();
    if (wave == 0) {
#pragma unroll
      for (int k = 1; k < kJoinWaves; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] += part[k][i * 64 + lane];
      float* to = grad_row(a, long_token[w], lane, err);
      if (to) finish<LAYOUT>(a, to, g, lane, acc);
    }
    __syncthreads();
  }
}

static int64_t part_stride(int64_t d) { return (d + 7) / 8 * 8; }

size_t embed_bwd_workspace_bytes(int64_t n, int64_t d) {
  const int64_t spans = (n + kSpan - 1) / kSpan;
  return spans > 1 ? static_cast<size_t>(2 * spans * part_stride(d)) * sizeof(float) : 0;
}

template <typename E, Layout LAYOUT>
static void embed_bwd(const EmbedGrad& a, void* ws, hipStream_t s, int* err) {
  const int64_t spans = (a.n_tokens + kSpan - 1) / kSpan, ld = part_stride(a.d);
  float* first = static_cast<float*>(ws);
  float* last = first + spans * ld;
  const int groups = static_cast<int>((a.d + kEmbedCols - 1) / kEmbedCols);
  embed_bwd_kernel<E, LAYOUT><<<dim3(static_cast<unsigned>(spans * groups)), dim3(64 * kChunks), 0, s>>>(
      a, groups, first, last, ld, err);
  if (spans > 1)
    embed_bwd_join_kernel<LAYOUT><<<dim3(static_cast<unsigned>((spans + kJoinWaves - 1) / kJoinWaves * groups)),
                                 dim3(64 * kJoinWaves), 0, s>>>(a, groups, first, last, ld, err);
}

template <typename E>
static void embed_bwd(const EmbedGrad& a, void* ws, hipStream_t s, int* err) {
  const bool aligned = a.d % 8 == 0 && vec_rows(a.dy.data, a.dy.stride, sizeof(E)) && vec_rows(a.grad, a.d, 4);
  if (aligned) embed_bwd<E, kAligned>(a, ws, s, err);
  else if (a.d >= 8) embed_bwd<E, kLoose>(a, ws, s, err);
  else embed_bwd<E, kSingle>(a, ws, s, err);
}

hipError_t launch_embed_bwd(const EmbedGrad& a, int32_t dtype, void* ws, hipStream_t s, int* err) {
  if (dtype == STAPLE_BF16) embed_bwd<bf16_t>(a, ws, s, err);
  else embed_bwd<float>(a, ws, s, err);
  return hipGetLastError();
}

}  // namespace staple
