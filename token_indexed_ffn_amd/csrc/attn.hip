// Attention over packed sequences with a causal mask, a sliding window and
// sinks: forward and backward.
//
// bf16 (fp32: attn_f32.hip).  A workgroup has 128 queries (or, for dk and dv,
// keys), 32 a wave, one a column of the products of attn_tile.h; the rows they
// meet come through LDS, 32 at a time, in rings of slots filled a few blocks
// ahead.  All three kernels are bound by what a wave can issue: matrix
// products, exponentials and LDS reads together.  So they spread one block's
// vector work between the products of other blocks, and keep their loop free of
// address and mask work: positions are 32-bit, a head's rows are one buffer,
// and only blocks at the edge of what is seen apply a mask.
//
// Measured on 6 causal sequences of 700 to 4096 tokens, 32 heads on 8 of 128:
// forward 487 us (820 TFLOP/s), dq 684 us (876, its three products), dk and dv
// 943 us (847, their four).  A large matrix product reaches 1234 with a larger
// share of busy cycles at a lower clock: the product of the two is 0.84 to 0.92
// GHz here and 1.05 there.
#include <type_traits>

#include "attn_seq.h"

namespace staple {

// ------------------------------------------------------------------- forward
// o / sum and lse of the wave's columns.
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
  bad = bad && w.in && !is_nan(sum);   // a NaN among the weights makes the row NaN
  if (bad && w.p >= 0) {
    bad = false;
#pragma unroll
    for (int d = 0; d < Tile<T, DP>::kDT; ++d) bad |= !own_value_explains<T>(a, w, d, o[d]);
  }
  redo(columns(bad), 0, 1, [&](int i) { attn_fwd_row<T>(a, w.q0 + w.wq + i, w.head, w.past + w.wq + i, w.k0); });
}

// bf16.  A block (32 keys x 32 queries at DP 128) is 16 MFMAs, 512 cycles, and
// 16 exponentials a lane, nearly as many cycles of vector work.  So the wave
// runs three blocks at a time: between the exponentials of block b stand the
// score products of block b + 1 and the value products of block b - 1.  The
// workgroup meets every second block: a stage loads two blocks of K and of V
// while the two before are worked on.  64 sequences of 256 tokens, 16 heads: 73
// us, 3.7 TB/s of q, k, v and o, bound by them.
//
// P is rounded to bf16 for its product, by 2^-8 of a weight at most, which the
// sum averages; the sum of the weights is of the unrounded ones.  o is then off
// by 2.0e-3 to 2.4e-3 of its norm, of which its own rounding is 1.6e-3.  A weight
// of two bf16 numbers leaves that alone, but has eight products more a block: the
// calls of 8 x 4096 tokens, 16 heads, window 1024, take 450 us so and 368 as it
// is, those of the ragged batch above 645 and 501.
template <int DP>
struct FwdShape {
  static constexpr int kBlock = 32 * Tile<bf16_t, DP>::kRow;
  static constexpr int kLds = 8 * kBlock;   // rings of four K blocks and four V blocks
};
template <int DP, bool kWide>
__global__ __launch_bounds__(64 * kWaves, 2) void attn_fwd_bf16_kernel(AttnView a, int64_t n_slots, KeyParts parts, int* err) {
  using T = bf16_t;
  using TL = Tile<T, DP>;
  constexpr int kBlock = FwdShape<DP>::kBlock;
  extern __shared__ __align__(1024) char smem[];
  lds_char* const kring = (lds_char*)smem;
  lds_char* const vring = kring + 4 * kBlock;
  check_offsets(a, err);
  QueryCols w;
  const int tile = static_cast<int>(blockIdx.x) / parts.n, part = static_cast<int>(blockIdx.x) - tile * parts.n;
  if (!w.find(a, kBf16RowsLog2, n_slots, tile, wave_id(), err)) return;
  KeyBlocks keys = w.blocks(a);
  int shares = 1;
  if (parts.n > 1) {
    shares = keys.share(parts.n, part);
    if (part >= shares) return;
  }
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
  if (shares == 1) return finish_fwd<T, DP>(a, w, sm, o);
  if (w.wq >= w.nq) return;
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * kWaves + wave_id();
  parts.put_rows(unit, sm.top, sm.sum + other_half(sm.sum));
#pragma unroll
  for (int d = 0; d < TL::kDT; ++d) parts.put<TL::kDT>(unit, d, o[d]);
}

// ------------------------------------------------------------------ backward
// dq, and the row statistics for the other kernel.  A block is 16 MFMAs for the
// scores and their gradients, then 16 elements of vector work with the 8 MFMAs
// of the block before in between.  8 sequences of 4096 tokens, window 1024, 16
// heads: 510 us.  dS is rounded to bf16 for its product, as P is in the forward:
// dq is off by 2.4e-3 of its norm, of which its own rounding is 1.7e-3.  Of two
// bf16 numbers, the calls of the whole backward take 1320 us in place of 1233.
template <int DP>
struct DqShape {
  static constexpr int kAhead = 2;
  static constexpr int kKSlots = kAhead + 2, kVSlots = kAhead + 1;
  static constexpr int kBlock = 32 * Tile<bf16_t, DP>::kRow;
  static constexpr int kLds = (kKSlots + kVSlots) * kBlock;
};
template <int DP, bool kWide>
__global__ __launch_bounds__(64 * kWaves, 2) void attn_dq_bf16_kernel(AttnView a, int64_t n_slots, KeyParts parts, RowStats stats,
                                                                      DkvPlan plan, int* err) {
  using T = bf16_t;
  using TL = Tile<T, DP>;
  using Shape = DqShape<DP>;
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
  const int id = static_cast<int>(blockIdx.x) - 1, tile = id / parts.n, part = id - tile * parts.n;
  if (!w.find(a, kBf16RowsLog2, n_slots, tile, wave_id(), err)) return;
  KeyBlocks keys = w.blocks(a);
  const bool few = keys.n <= kFew;
  int shares = 1;
  if (parts.n > 1) {
    shares = keys.share(parts.n, part);
    if (part >= shares) return;
  }
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
  // delta from the rounded o is off by sum d_o (o's rounding), which counts
  // where o is large: where few keys share a query's weight.  A workgroup of
  // few blocks therefore meets them once before, for delta + sum P (dP -
  // delta), exact as sum P = 1.
  static_assert(kFew <= kMinShare, "all of the tile's blocks are here");
  if (few) {
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
  if (part == 0 && w.in && half == 0) {
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
  };
  if (keys.n > 0) {
    step(std::true_type{}, 0);
    for (int b = 1; b < keys.n; ++b) step(std::false_type{}, b);
#pragma unroll
    for (int d = 0; d < TL::kDT; ++d) dq[d] = mma_transposed<DP>(kprev, 0, d, prev, dq[d]);
  }
  wait_vmcnt<0>();   // no load into LDS outlives the workgroup
  if (shares > 1) {
    if (w.wq >= w.nq) return;
#pragma unroll
    for (int d = 0; d < TL::kDT; ++d) parts.put<TL::kDT>(static_cast<int64_t>(id) * kWaves + wave_id(), d, dq[d]);
    return;
  }
  bool bad = false;
#pragma unroll
  for (int d = 0; d < TL::kDT; ++d) {
#pragma unroll
    for (int r = 0; r < 16; ++r) bad |= not_finite(dq[d][r]);
    store_column<T>(a.dq, w.q0 + w.row, w.head, a.head_dim, d, dq[d], a.scale, w.in);
  }
  // a NaN in the query's statistics makes the row NaN
  bad = bad && w.in && !(w.p >= 0 && (is_nan(delta) || is_nan(lse2)));
  redo(columns(bad), 0, 1, [&](int i) { attn_dq_row<T>(a, w.q0 + w.wq + i, w.head, w.past + w.wq + i, w.k0); });
}

// dk and dv of 32 keys take 2 DP registers a lane, too many beside the
// operands for two waves a SIMD.  So two waves share 32 keys: of a stage of
// two query blocks each forms the probabilities and score gradients of one,
// they trade them through LDS, and each adds both to its half of head_dim.
// Between the elements of a stage stand the gradient products of the stage
// before.  P and dS are rounded to bf16 (dk and dv are off by 2.3e-3 of their
// norms, of which their own rounding is 1.7e-3): of two numbers each, the trade
// would not fit beside the ring.  8 sequences of 4096 tokens, window 1024, 16
// heads: 807 us, a workgroup's 37 blocks at a time; one workgroup a CU, so that
// its first loads and its last stores overlap nothing.
constexpr int kDkvWaves = 8;
template <int DP>
struct DkvPair {
  // a ring slot: a query block's Q and dO, then lse2 and delta (256 bytes each,
  // half of it used)
  static constexpr int kBlock = 32 * Tile<bf16_t, DP>::kRow;
  static constexpr int kStage = 2 * kBlock + 512;
  static constexpr int kTrade = 4 * 2 * 4 * 1024;              // [keys / 32][block][P, P, dS, dS][lane]
  static constexpr int kLds = 6 * kStage + kTrade;             // three pairs of slots: before, at hand, loading
};
template <int DP, bool kWide>
__global__ __launch_bounds__(64 * kDkvWaves, 2) void attn_dkv_bf16_kernel(AttnView a, RowStats stats, DkvPlan plan) {
  using T = bf16_t;
  using TL = Tile<T, DP>;
  using Shape = DkvPair<DP>;
  constexpr int kBlock = Shape::kBlock, kStage = Shape::kStage, kPair = 2 * kStage;
  constexpr int kHalf = TL::kDT / 2;   // 32-element blocks of head_dim a wave
  extern __shared__ __align__(1024) char smem[];
  lds_char* const ring = (lds_char*)smem;
  const int keys_of = wave_id() & 3, side = wave_id() >> 2;
  DkvItem w;
  if (!w.find(a, plan, keys_of)) return;
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
  if (w.parts > 1) {
    if (w.wkey >= w.nk) return;
    f32x4_t* to = part_sums<2 * TL::kDT>(plan, w.sums + w.part, w.hk, a.n_kv_heads, keys_of);
#pragma unroll
    for (int d = 0; d < kHalf; ++d) {
      put_sums(to, side * kHalf + d, x[d]);
      put_sums(to, TL::kDT + side * kHalf + d, x[kHalf + d]);
    }
    return;
  }
  bool bad = false;
#pragma unroll
  for (int d = 0; d < kHalf; ++d) {
    bad |= has_unexplained<T>(a, stats, w, false, side * kHalf + d, x[d]);
    bad |= has_unexplained<T>(a, stats, w, true, side * kHalf + d, x[kHalf + d]);
    store_column<T>(a.dk, w.k0 + w.key, w.hk, a.head_dim, side * kHalf + d, x[d], a.scale, w.in);
    store_column<T>(a.dv, w.k0 + w.key, w.hk, a.head_dim, side * kHalf + d, x[kHalf + d], 1.0f, w.in);
  }
  redo_keys<T>(a, stats, w, bad, keys_of, 4, 2, side);
}

// ------------------------------------------------------------------- launches
size_t attn_fwd_workspace_bytes(const AttnView& a, int dtype) {
  Workspace w(nullptr, ~size_t(0));
  take_parts(a, dtype == STAPLE_F32 ? kF32RowsLog2 : kBf16RowsLog2, w);
  return w.used;
}

template <int DP, bool kWide>
static hipError_t fwd_launch(const AttnView& a, const KeyParts& parts, hipStream_t s, int* err) {
  const int64_t n = tile_slots(a.total_q, a.n_seqs, kBf16RowsLog2);
  const hipError_t e =
      launch_lds<attn_fwd_bf16_kernel<DP, kWide>, FwdShape<DP>::kLds>(n * a.n_heads * parts.n, s, a, n, parts, err);
  return e != hipSuccess ? e : launch_join<bf16_t, DP, false>(a, kBf16RowsLog2, n, parts, s, err);
}

hipError_t launch_attn_fwd(const AttnView& a, int dtype, void* ws, hipStream_t s, int* err) {
  if (dtype == STAPLE_F32) return launch_attn_fwd_f32(a, ws, s, err);
  Workspace w(ws, ~size_t(0));
  const KeyParts parts = take_parts(a, kBf16RowsLog2, w);
  const bool far = spans_buffer(a.k, a.total_k, 2) || spans_buffer(a.v, a.total_k, 2);
  if (a.head_dim <= 64) return far ? fwd_launch<64, true>(a, parts, s, err) : fwd_launch<64, false>(a, parts, s, err);
  return far ? fwd_launch<128, true>(a, parts, s, err) : fwd_launch<128, false>(a, parts, s, err);
}

// A split tile has more than `chunk` blocks, so that all of them together have
// at most 2 total / chunk <= 2 target parts, and no more than two for every
// kMinChunk blocks.
static BwdSpace bwd_space(const AttnView& a, int dtype, void* ws) {
  BwdSpace b{};
  const int dp = a.head_dim <= 64 ? 64 : 128;
  b.plan.rows_log2 = dtype == STAPLE_F32 ? kF32RowsLog2 : kBf16RowsLog2;
  const int64_t n = tile_slots(a.total_k, a.n_seqs, b.plan.rows_log2);
  b.plan.n_slots = n;
  b.plan.target = (2 * device_cus() + a.n_kv_heads - 1) / a.n_kv_heads;   // two parts a CU
  const int64_t blocks = (a.total_q / 32 + a.n_seqs) * a.group * n;       // more than there are
  const int64_t most = 2 * (blocks / kMinChunk) + 2;
  b.plan.max_parts = static_cast<int>(most < 2 * b.plan.target ? most : 2 * b.plan.target);
  // a tile of kMinChunk blocks or less is never split
  int64_t per_head = (a.total_q + 31) / 32;
  const int64_t window = (a.window + (int64_t(1) << b.plan.rows_log2) + 31) / 32 + 1;
  if (a.window > 0 && a.sinks == 0 && window < per_head) per_head = window;
  if (per_head * a.group <= kMinChunk) b.plan.max_parts = 0;
  Workspace w(ws, ~size_t(0));
  const size_t rows = static_cast<size_t>(a.total_q) * a.n_heads * sizeof(float);
  const size_t ints = static_cast<size_t>(n) * sizeof(int32_t);
  b.stats.lse2 = w.take<float>(rows);
  b.stats.delta = w.take<float>(rows);
  b.plan.head = w.take<int32_t>(2 * sizeof(int32_t));
  b.plan.blocks = w.take<int32_t>(ints);
  b.plan.tiles = w.take<DkvRecord>(static_cast<size_t>(n) * sizeof(DkvRecord));
  b.plan.split = w.take<int32_t>(b.plan.max_parts * sizeof(int32_t));
  b.plan.items = w.take<DkvRecord>((static_cast<size_t>(n) + b.plan.max_parts) * sizeof(DkvRecord));
  const size_t sums = (size_t(2) << b.plan.rows_log2) * dp * sizeof(float);   // dk and dv of a tile
  b.plan.sums = w.take<f32x4_t>(static_cast<size_t>(b.plan.max_parts) * a.n_kv_heads * sums);
  b.parts = take_parts(a, b.plan.rows_log2, w);
  b.bytes = w.used;
  return b;
}
size_t attn_bwd_workspace_bytes(const AttnView& a, int dtype) { return bwd_space(a, dtype, nullptr).bytes; }

template <int DP, bool kWide>
static hipError_t bwd_launch(const AttnView& a, const BwdSpace& b, hipStream_t s, int* err) {
  const int64_t nq = tile_slots(a.total_q, a.n_seqs, kBf16RowsLog2);
  // one workgroup more than there are query tiles: it makes the plan
  hipError_t e = launch_lds<attn_dq_bf16_kernel<DP, kWide>, DqShape<DP>::kLds>(nq * a.n_heads * b.parts.n + 1, s, a, nq, b.parts,
                                                                                 b.stats, b.plan, err);
  if (e != hipSuccess) return e;
  e = launch_join<bf16_t, DP, true>(a, kBf16RowsLog2, nq, b.parts, s, err);
  if (e != hipSuccess) return e;
  const int64_t items = (b.plan.n_slots + b.plan.max_parts) * a.n_kv_heads;   // at most
  e = launch_lds<attn_dkv_bf16_kernel<DP, kWide>, DkvPair<DP>::kLds, 64 * kDkvWaves>(items, s, a, b.stats, b.plan);
  return e != hipSuccess ? e : launch_dkv_join<bf16_t, DP>(a, b, s);
}

hipError_t launch_attn_bwd(const AttnView& a, int dtype, void* ws, hipStream_t s, int* err) {
  const BwdSpace b = bwd_space(a, dtype, ws);
  if (dtype == STAPLE_F32) return launch_attn_bwd_f32(a, b, s, err);
  const bool far = spans_buffer(a.q, a.total_q, 2) || spans_buffer(a.d_o, a.total_q, 2) || spans_buffer(a.k, a.total_k, 2) ||
                   spans_buffer(a.v, a.total_k, 2);
  if (a.head_dim <= 64) return far ? bwd_launch<64, true>(a, b, s, err) : bwd_launch<64, false>(a, b, s, err);
  return far ? bwd_launch<128, true>(a, b, s, err) : bwd_launch<128, false>(a, b, s, err);
}

}  // namespace staple
