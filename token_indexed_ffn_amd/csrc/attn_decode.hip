// Attention of one new token per sequence over a paged key-value cache.
//
// One wave takes up to 16 query heads that share a key-value head, and a block
// of keys at a time (32 in bf16, 16 in fp32), straight from memory into
// registers; nothing but the final join of a workgroup's waves goes through
// LDS:
//   scores  S^T = K Q^T by v_mfma_f32_16x16x32_bf16 (fp32: 16x16x4): a key a
//           row (lane % 16), so that a K row's 16-byte pieces are the A
//           operand as they are loaded.  Lane q + 16 g then holds the scores of
//           head q and keys 4 g .. 4 g + 3 of each 16.
//   values  O^T = V^T P^T: the lane's own scores are the B operand when its
//           slot of the contraction stands for those same keys, so a lane loads
//           V rows 4 g .. 4 g + 3 of each 16 keys, elements E c .. E c + E - 1
//           (c = lane % 16, E = head_dim / 16); one byte permute a dword gathers
//           the 8 keys of one element: the A operand, rows in the order E c + t.
// The 16 columns are mostly idle for a small group, but the matrix cores are
// far from busy: a block is 16 KB of cache and 24 MFMAs.  Bound by HBM: the
// cache is read once, and the waves of a CU keep over 100 KB in flight.
//
// A key that is not seen (past the length, outside the window and the sinks)
// is never loaded and counts as zeros with weight zero.
//
// The cache is split along its length over workgroups where the (sequence,
// head) pairs alone are too few; the splits' partial results are joined by a
// second kernel in split order.
//
// Measured: two sequences of 100001 to 131071 keys, 32 heads on 8, 168 us (5.5
// TB/s) and 6 in the join; 64 sequences around 256 keys, 16 heads, 32 us (4.2
// TB/s, no join); one of 37 keys 8 us, its chain of loads: length, page, rows.
#include "attn.h"

namespace staple {

constexpr int kDecWaves = 4;

template <typename T, int DP>
struct DecBlock {
  static constexpr int kKeys = 64 / static_cast<int>(sizeof(T));          // 32 (bf16) or 16 keys
  static constexpr int kRB = kKeys / 16;                                  // 16-key row blocks
  static constexpr int kSteps = DP * static_cast<int>(sizeof(T)) / 64;    // 16-byte K pieces per lane and row block
  static constexpr int kE = DP / 16;                                      // head elements per lane of V
  static constexpr int kVB = kE * static_cast<int>(sizeof(T));            // bytes of V per lane and key: 8, 16 or 32
  static constexpr int kVK = 4 * kRB;                                     // V keys per lane
};

// kVB bytes of V.
template <int N> struct __align__(N < 16 ? N : 16) VPiece { uint32_t w[N / 4]; };

template <typename T, int DP>
struct DecKV {
  using B = DecBlock<T, DP>;
  u32x4_t k[B::kRB][B::kSteps];
  VPiece<B::kVB> v[B::kVK];
};

// Where a wave's keys come from.
struct DecSource {
  const char* kp;            // this kv head's slots of page 0
  const char* vp;
  const char* k_new;         // the new token's rows, or null
  const char* v_new;
  int64_t page_bytes;        // from one page to the next
  int row_bytes, page_log2, page_mask;
  int64_t n_pages;
  const int32_t* pages;      // the sequence's row of the table
  int64_t last, lo, sink;    // the query's position; keys [0, sink) and [lo, last] are seen
  bool write_new;            // this wave also writes k_new, v_new to the cache
};

__device__ __forceinline__ int64_t page_of(const DecSource& s, int64_t key, int* err) {
  const int p = s.pages[key >> s.page_log2];
  if (p < 0 || p >= s.n_pages) {
    flag_index_error(err);
    return -1;
  }
  return p;
}
__device__ __forceinline__ bool seen(const DecSource& s, int64_t key) {
  return (key <= s.last) & ((key >= s.lo) | (key < s.sink));
}

// Byte offset of a key's row within the pool's kv head, -1 where it may not be read.
__device__ __forceinline__ int64_t row_offset(const DecSource& s, int64_t key, int64_t page) {
  return page < 0 ? -1 : page * s.page_bytes + static_cast<int64_t>(key & s.page_mask) * s.row_bytes;
}

template <typename T, int DP>
__device__ __forceinline__ void load_k(const DecSource& s, int64_t key0, const int64_t* page, bool whole,
                                       DecKV<T, DP>& b) {
  using B = DecBlock<T, DP>;
  const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
#pragma unroll
  for (int rb = 0; rb < B::kRB; ++rb) {
    const int64_t key = key0 + 16 * rb + r;
    const int64_t at = row_offset(s, key, page[rb]);
    const char* row = s.kp + at;
    bool in = at >= 0;
    if (!whole) {
      in = in && seen(s, key);
      if (s.k_new && key == s.last) row = s.k_new;
    }
#pragma unroll
    for (int st = 0; st < B::kSteps; ++st) {
      const int off = 16 * (4 * st + g);
      b.k[rb][st] = in && off < s.row_bytes ? *reinterpret_cast<const u32x4_t*>(row + off) : u32x4_t{0, 0, 0, 0};
      if (!whole && s.write_new && in && key == s.last && off < s.row_bytes)
        *reinterpret_cast<u32x4_t*>(const_cast<char*>(s.kp) + at + off) = b.k[rb][st];
    }
  }
}

template <typename T, int DP>
__device__ __forceinline__ void load_v(const DecSource& s, int64_t key0, const int64_t* page, bool whole,
                                       DecKV<T, DP>& b) {
  using B = DecBlock<T, DP>;
  using P = VPiece<B::kVB>;
  const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
#pragma unroll
  for (int j = 0; j < B::kVK; ++j) {
    const int64_t key = key0 + 16 * (j >> 2) + 4 * g + (j & 3);
    const int64_t at = row_offset(s, key, page[j >> 2]);
    const char* row = s.vp + at;
    const int off = c * B::kVB;
    bool in = at >= 0 && off < s.row_bytes;
    if (!whole) {
      in = in && seen(s, key);
      if (s.v_new && key == s.last) row = s.v_new;
    }
    b.v[j] = P{};
    if (in) b.v[j] = *reinterpret_cast<const P*>(row + off);
    if (!whole && s.write_new && in && key == s.last)
      *reinterpret_cast<P*>(const_cast<char*>(s.vp) + at + off) = b.v[j];
  }
}

// Scores of the block: s[rb][r] is key 16 rb + 4 g + r of column lane % 16.
template <int DP>
__device__ __forceinline__ void dec_scores(const DecKV<bf16_t, DP>& b, const u32x4_t* q, f32x4_t* s) {
  using B = DecBlock<bf16_t, DP>;
#pragma unroll
  for (int rb = 0; rb < B::kRB; ++rb) {
    s[rb] = f32x4_t{0, 0, 0, 0};
#pragma unroll
    for (int st = 0; st < B::kSteps; ++st)
      s[rb] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, b.k[rb][st]),
                                                      __builtin_bit_cast(bf16x8_t, q[st]), s[rb], 0, 0, 0);
  }
}
template <int DP>
__device__ __forceinline__ void dec_scores(const DecKV<float, DP>& b, const u32x4_t* q, f32x4_t* s) {
  using B = DecBlock<float, DP>;
#pragma unroll
  for (int rb = 0; rb < B::kRB; ++rb) {
    s[rb] = f32x4_t{0, 0, 0, 0};
#pragma unroll
    for (int st = 0; st < B::kSteps; ++st)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        s[rb] = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(b.k[rb][st][i]), __uint_as_float(q[st][i]),
                                                     s[rb], 0, 0, 0);
  }
}

// o[t] += the block's weighted values (weights p), element E (4 g + r) + t in register r.
// bf16: a weight is the sum of two bf16 numbers, itself rounded and what that
// leaves, off by 2^-17 of it at most: o is then as close as its own rounding.
// The matrix cores have the time: two sequences of 100001 to 131071 keys take 169
// us, and 167 with weights of one bf16 number.
template <int DP>
__device__ __forceinline__ void dec_values(const DecKV<bf16_t, DP>& b, const f32x4_t* p, f32x4_t* o) {
  using B = DecBlock<bf16_t, DP>;
  u32x4_t high, low;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float x = p[i >> 1][2 * (i & 1)], y = p[i >> 1][2 * (i & 1) + 1];
    high[i] = pack_bf16x2(x, y);
    low[i] = pack_bf16x2(x - __uint_as_float(high[i] << 16), y - __uint_as_float(high[i] & 0xffff0000u));
  }
#pragma unroll
  for (int t = 0; t < B::kE; ++t) {
    u32x4_t a;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      a[i] = __builtin_amdgcn_perm(b.v[2 * i + 1].w[t >> 1], b.v[2 * i].w[t >> 1], (t & 1) ? 0x07060302u : 0x05040100u);
    o[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, high),
                                                   o[t], 0, 0, 0);
    o[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, low),
                                                   o[t], 0, 0, 0);
  }
}
template <int DP>
__device__ __forceinline__ void dec_values(const DecKV<float, DP>& b, const f32x4_t* p, f32x4_t* o) {
  using B = DecBlock<float, DP>;
#pragma unroll
  for (int t = 0; t < B::kE; ++t)
#pragma unroll
    for (int j = 0; j < B::kVK; ++j)
      o[t] = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(b.v[j].w[t]), p[0][j], o[t], 0, 0, 0);
}

// The blocks of `keys` keys that hold a seen key: the sinks', then the window's.
struct DecBlocks {
  int64_t n_sink, lo, n;
  __device__ __forceinline__ DecBlocks(const DecSource& s, int keys) {
    lo = s.lo / keys;
    const int64_t sink = s.sink < lo * keys ? s.sink : lo * keys;
    n_sink = s.last < 0 ? 0 : (sink + keys - 1) / keys;
    n = s.last < 0 ? 0 : n_sink + s.last / keys + 1 - lo;
  }
  __device__ __forceinline__ int64_t at(int64_t i) const { return i < n_sink ? i : lo + i - n_sink; }
};

// Partial results of one (sequence, head, split): DP sums of weighted values,
// then the reference score and the sum of the weights.
struct DecPartials {
  float* o;      // [n_seqs][n_heads][splits][DP]
  float* stat;   // [n_seqs][n_heads][splits][2]
};

template <typename T, int DP>
__global__ __launch_bounds__(64 * kDecWaves) void attn_decode_kernel(KvView kv, DecodeView a, int chunk, int splits,
                                                                     int head_tiles, DecPartials part, int* err) {
  using B = DecBlock<T, DP>;
  constexpr int kLd = DP + 4;   // LDS row of a head's sums: 16 rows spread over the banks
  __shared__ __align__(16) float joined[kDecWaves][16][kLd];
  __shared__ float stats[kDecWaves][16][2];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int per_seq = kv.kv_heads * head_tiles;
  const int64_t id = blockIdx.x;
  const int hk = static_cast<int>(id % per_seq) / head_tiles, ht = static_cast<int>(id % per_seq) % head_tiles;
  const int64_t i = id / per_seq % a.n_seqs;
  const int split = static_cast<int>(id / per_seq / a.n_seqs);
  const int h0 = hk * a.group + 16 * ht;                             // first query head
  const int heads = a.group - 16 * ht < 16 ? a.group - 16 * ht : 16;

  const int64_t row = a.seqs ? a.seqs[i] : i;
  const bool row_in = row >= 0 && row < kv.n_rows;
  int64_t len = row_in ? kv.lens[row] : 0;
  const bool fits = row_in && len >= 0 && len <= a.max_len;
  if (!fits) {
    flag_index_error(err);
    len = len < 0 ? 0 : len > a.max_len ? a.max_len : len;
  }
  const int64_t es = sizeof(T);
  DecSource src;
  src.row_bytes = kv.row_bytes;
  src.page_log2 = kv.page_log2;
  src.page_mask = kv.page - 1;
  const int64_t head_bytes = static_cast<int64_t>(kv.page) * kv.row_bytes;
  src.page_bytes = kv.kv_heads * head_bytes;
  src.kp = kv.k_pages + hk * head_bytes;
  src.vp = kv.v_pages + hk * head_bytes;
  src.n_pages = kv.n_pages;
  src.pages = kv.table + (row_in ? row : 0) * kv.max_pages;
  src.last = len - 1;
  visible_keys(src.last, a.window, a.sinks, &src.sink, &src.lo);
  // a sequence that is cut, or was not grown, ends in an older token, which
  // keeps its rows
  const bool has_new = a.k_new.data && fits && !was_refused(kv, row);
  src.k_new = has_new ? a.k_new.data + (i * a.k_new.row_stride + hk * a.k_new.head_stride) * es : nullptr;
  src.v_new = has_new ? a.v_new.data + (i * a.v_new.row_stride + hk * a.v_new.head_stride) * es : nullptr;
  src.write_new = src.k_new != nullptr && ht == 0;
  const DecBlocks blocks(src, B::kKeys);

  // the query heads, one a column
  u32x4_t q[B::kSteps];
  {
    const int h = lane & 15, g = lane >> 4;
    const char* p = a.q.data + (i * a.q.row_stride + (h0 + h) * a.q.head_stride) * es;
#pragma unroll
    for (int st = 0; st < B::kSteps; ++st) {
      const int off = 16 * (4 * st + g);
      q[st] = h < heads && off < kv.row_bytes ? *reinterpret_cast<const u32x4_t*>(p + off) : u32x4_t{0, 0, 0, 0};
      if (a.scale < 0.0f) q[st] ^= sizeof(T) == 2 ? u32x4_t{0x80008000u, 0x80008000u, 0x80008000u, 0x80008000u}
                                                  : u32x4_t{0x80000000u, 0x80000000u, 0x80000000u, 0x80000000u};
    }
  }
  const float c = fabsf(a.scale) * kLog2e;

  f32x4_t o[B::kE] = {};
  float top = -INFINITY, sum = 0.0f;   // sum: this lane's keys
  const int64_t end = (split + 1) * static_cast<int64_t>(chunk) < blocks.n ? (split + 1) * static_cast<int64_t>(chunk) : blocks.n;
  int64_t b = split * static_cast<int64_t>(chunk) + w;
  DecKV<T, DP> kvb;
  int64_t page[2] = {-1, -1};
  // the pages of block `n`: a block's 16-key halves lie in one page each
  auto find = [&](int64_t n) {
    const int64_t key = blocks.at(n) * B::kKeys;
#pragma unroll
    for (int rb = 0; rb < B::kRB; ++rb) {
      const int64_t k = key + 16 * rb;
      const bool any = k <= src.last && (k + 15 >= src.lo || k < src.sink);
      page[rb] = any ? page_of(src, k, err) : -1;
    }
  };
  auto whole_of = [&](int64_t n) {
    const int64_t key = blocks.at(n) * B::kKeys;
    return key + B::kKeys - 1 + (src.k_new ? 1 : 0) <= src.last && (key >= src.lo || key + B::kKeys <= src.sink);
  };
  if (b < end) {
    find(b);
    load_k<T, DP>(src, blocks.at(b) * B::kKeys, page, whole_of(b), kvb);
  }
  for (; b < end; b += kDecWaves) {
    const int64_t key0 = blocks.at(b) * B::kKeys;
    const bool whole = whole_of(b);
    load_v<T, DP>(src, key0, page, whole, kvb);
    f32x4_t s[B::kRB];
    dec_scores<DP>(kvb, q, s);
    bool there[B::kRB];
#pragma unroll
    for (int rb = 0; rb < B::kRB; ++rb) there[rb] = page[rb] >= 0;
    if (b + kDecWaves < end) {   // the next block's keys come while this one's values are weighted
      find(b + kDecWaves);
      load_k<T, DP>(src, blocks.at(b + kDecWaves) * B::kKeys, page, whole_of(b + kDecWaves), kvb);
    }
    float m = -INFINITY;
#pragma unroll
    for (int rb = 0; rb < B::kRB; ++rb)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int64_t key = key0 + 16 * rb + 4 * (lane >> 4) + r;
        s[rb][r] = there[rb] & (whole | seen(src, key)) ? s[rb][r] * c : -INFINITY;
        m = fmaxf(m, s[rb][r]);
      }
    // the sums stay relative to an earlier maximum until a score passes it by
    // 2^8: no exchange between lanes before that
    if (__any((m > top + 8.0f) | ((top == -INFINITY) & (m > top)))) {
      m = fmaxf(m, __shfl_xor(m, 16));
      m = fmaxf(m, __shfl_xor(m, 32));
      const float t = fmaxf(top, m);
      const float keep = top == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(top - t);
      top = t;
      sum *= keep;
#pragma unroll
      for (int e = 0; e < B::kE; ++e) o[e] *= keep;
    }
    const float base = top == -INFINITY ? 0.0f : top;
#pragma unroll
    for (int rb = 0; rb < B::kRB; ++rb)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        s[rb][r] = __builtin_amdgcn_exp2f(s[rb][r] - base);
        sum += s[rb][r];
      }
    dec_values<DP>(kvb, s, o);
  }
  sum += __shfl_xor(sum, 16);
  sum += __shfl_xor(sum, 32);

  // the waves' sums to LDS, then joined
#pragma unroll
  for (int r = 0; r < 4; ++r)
#pragma unroll
    for (int e = 0; e < B::kE; e += 4)
      *reinterpret_cast<f32x4_t*>(&joined[w][lane & 15][(4 * (lane >> 4) + r) * B::kE + e]) =
          f32x4_t{o[e][r], o[e + 1][r], o[e + 2][r], o[e + 3][r]};
  if (lane < 16) {
    stats[w][lane][0] = top;
    stats[w][lane][1] = sum;
  }
  __syncthreads();
  constexpr int kPieces = DP / 4;
  for (int x = threadIdx.x; x < heads * kPieces; x += 64 * kDecWaves) {
    const int h = x / kPieces, e = x % kPieces * 4;
    float t = -INFINITY;
#pragma unroll
    for (int u = 0; u < kDecWaves; ++u) t = fmaxf(t, stats[u][h][0]);
    f32x4_t v = {0, 0, 0, 0};
    float total = 0.0f;
#pragma unroll
    for (int u = 0; u < kDecWaves; ++u) {
      const float keep = stats[u][h][0] == -INFINITY && stats[u][h][1] == 0.0f ? 0.0f : __builtin_amdgcn_exp2f(stats[u][h][0] - t);
      total += stats[u][h][1] * keep;
      v += *reinterpret_cast<const f32x4_t*>(&joined[u][h][e]) * keep;
    }
    const int64_t at = i * a.n_heads + h0 + h;
    if (splits > 1) {
      *reinterpret_cast<f32x4_t*>(part.o + (at * splits + split) * DP + e) = v;
      if (e == 0) {
        part.stat[(at * splits + split) * 2] = t;
        part.stat[(at * splits + split) * 2 + 1] = total;
      }
      continue;
    }
    const float inv = total == 0.0f ? 0.0f : 1.0f / total;
    if (e < a.head_dim) {
      char* p = a.o.data + (i * a.o.row_stride + (h0 + h) * a.o.head_stride + e) * es;
      if constexpr (sizeof(T) == 2)
        *reinterpret_cast<u32x2_t*>(p) = u32x2_t{pack_bf16x2(v[0] * inv, v[1] * inv), pack_bf16x2(v[2] * inv, v[3] * inv)};
      else
        *reinterpret_cast<f32x4_t*>(p) = v * inv;
    }
    if (a.lse && e == 0) a.lse[at] = (t + __builtin_amdgcn_logf(total)) * kLn2;
  }
}

// One workgroup a (sequence, head): every wave joins the splits w, w + 4, ...
// in that order, and then the waves' sums are added in wave order.
template <typename T, int DP>
__global__ __launch_bounds__(64 * kDecWaves) void attn_decode_join_kernel(DecodeView a, int splits, DecPartials part) {
  constexpr int kPer = DP / 64;
  __shared__ float joined[kDecWaves][DP], totals[kDecWaves];
  const int64_t at = blockIdx.x;
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const float* stat = part.stat + at * splits * 2;
  // at most 128 splits: two a lane
  float t = fmaxf(lane < splits ? stat[2 * lane] : -INFINITY, lane + 64 < splits ? stat[2 * (lane + 64)] : -INFINITY);
#pragma unroll
  for (int d = 32; d > 0; d /= 2) t = fmaxf(t, __shfl_xor(t, d));
  float v[kPer] = {}, total = 0.0f;
#pragma unroll 4
  for (int s = w; s < splits; s += kDecWaves) {
    const float top = stat[2 * s], sum = stat[2 * s + 1];
    const float keep = top == -INFINITY && sum == 0.0f ? 0.0f : __builtin_amdgcn_exp2f(top - t);
    total += sum * keep;
#pragma unroll
    for (int e = 0; e < kPer; ++e) v[e] += part.o[(at * splits + s) * DP + kPer * lane + e] * keep;
  }
#pragma unroll
  for (int e = 0; e < kPer; ++e) joined[w][kPer * lane + e] = v[e];
  if (lane == 0) totals[w] = total;
  __syncthreads();
  if (w != 0) return;
#pragma unroll
  for (int u = 1; u < kDecWaves; ++u) {
    total += totals[u];
#pragma unroll
    for (int e = 0; e < kPer; ++e) v[e] += joined[u][kPer * lane + e];
  }
  const float inv = total == 0.0f ? 0.0f : 1.0f / total;
  const int64_t i = at / a.n_heads, h = at % a.n_heads;
  T* p = reinterpret_cast<T*>(a.o.data) + i * a.o.row_stride + h * a.o.head_stride;
#pragma unroll
  for (int e = 0; e < kPer; ++e)
    if (kPer * lane + e < a.head_dim) Elem<T>::store(p, kPer * lane + e, v[e] * inv);
  if (a.lse && lane == 0) a.lse[at] = (t + __builtin_amdgcn_logf(total)) * kLn2;
}

constexpr int kDecMaxSplits = 128;   // what a wave's lanes hold two each of

// How the cache is split: `chunk` blocks a workgroup, `splits` of them at most.
struct DecPlan {
  int chunk, splits, head_tiles;
};
static DecPlan plan(const KvView& kv, const DecodeView& a, int dtype) {
  const int keys = dtype == STAPLE_BF16 ? 32 : 16;
  int64_t seen = a.max_len;
  // a window and the sinks touch at most two blocks more than they fill
  if (a.window > 0 && a.sinks < a.max_len && a.window + a.sinks < a.max_len) seen = a.window + a.sinks;
  const int64_t blocks = (seen + keys - 1) / keys + 2;
  DecPlan p;
  p.head_tiles = (a.group + 15) / 16;
  const int64_t pairs = a.n_seqs * kv.kv_heads * p.head_tiles;
  const int64_t want = (int64_t(4) * device_cus() + pairs - 1) / pairs;   // four workgroups a CU
  // at least two blocks a wave in a split
  int64_t splits = blocks / (2 * kDecWaves);
  if (splits > want) splits = want;
  if (splits > kDecMaxSplits) splits = kDecMaxSplits;
  if (splits < 1) splits = 1;
  const int64_t chunk = (blocks + splits - 1) / splits;
  p.chunk = static_cast<int>((chunk + kDecWaves - 1) / kDecWaves * kDecWaves);
  p.splits = static_cast<int>((blocks + p.chunk - 1) / p.chunk);
  return p;
}
static int padded(int head_dim) { return head_dim <= 64 ? 64 : 128; }

size_t attn_decode_workspace_bytes(const KvView& kv, const DecodeView& a, int dtype) {
  if (a.n_seqs == 0) return 0;
  const DecPlan p = plan(kv, a, dtype);
  if (p.splits <= 1) return 0;
  const size_t rows = static_cast<size_t>(a.n_seqs) * a.n_heads * p.splits;
  return align_up(rows * padded(a.head_dim) * sizeof(float), 256) + align_up(rows * 2 * sizeof(float), 256);
}

template <typename T, int DP>
static hipError_t decode_launch(const KvView& kv, const DecodeView& a, int dtype, void* ws, hipStream_t s, int* err) {
  const DecPlan p = plan(kv, a, dtype);
  DecPartials part{};
  if (p.splits > 1) {
    const size_t rows = static_cast<size_t>(a.n_seqs) * a.n_heads * p.splits;
    Workspace w(ws, attn_decode_workspace_bytes(kv, a, dtype));
    part.o = w.take<float>(rows * DP * sizeof(float));
    part.stat = w.take<float>(rows * 2 * sizeof(float));
  }
  const int64_t wgs = a.n_seqs * kv.kv_heads * p.head_tiles * p.splits;
  attn_decode_kernel<T, DP><<<static_cast<unsigned>(wgs), 64 * kDecWaves, 0, s>>>(kv, a, p.chunk, p.splits, p.head_tiles, part, err);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.splits <= 1) return e;
  attn_decode_join_kernel<T, DP><<<static_cast<unsigned>(a.n_seqs * a.n_heads), 64 * kDecWaves, 0, s>>>(a, p.splits, part);
  return hipGetLastError();
}

hipError_t launch_attn_decode(const KvView& kv, const DecodeView& a, int dtype, void* ws, hipStream_t s, int* err) {
  if (dtype == STAPLE_BF16)
    return a.head_dim <= 64 ? decode_launch<bf16_t, 64>(kv, a, dtype, ws, s, err)
                            : decode_launch<bf16_t, 128>(kv, a, dtype, ws, s, err);
  return a.head_dim <= 64 ? decode_launch<float, 64>(kv, a, dtype, ws, s, err)
                          : decode_launch<float, 128>(kv, a, dtype, ws, s, err);
}

}  // namespace staple
