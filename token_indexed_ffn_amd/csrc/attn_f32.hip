// Attention in fp32: forward and backward (see attn.hip for the operator).
//
// fp32 products run at a sixteenth of the bf16 rate, so one block of 32 x 32
// pairs keeps a wave's matrix core busy for thousands of cycles and everything
// else is small beside it: what matters is that all matrix cores have work.  A
// workgroup has only 32 queries (or keys), and its four waves share the blocks
// that these meet: each takes every fourth one, loads it into LDS of its own
// (no wave waits for another) and sums its part; the parts are joined in LDS in
// wave order.
//
// Measured (MI355X; fp32 products reach 154 TFLOP/s in a large matrix
// product), forward and backward, beside tiles of 128 queries whose waves share
// the blocks that a workgroup loads:
//   512 tokens, 4 heads of 64:         12 + 33 us;     28 + 79
//   8 x 1024 tokens, 8 heads of 64:    122 + 411 us;   141 + 492
//   4 x 2048 tokens, 16 heads of 128:  748 + 2421 us (92, 99 TFLOP/s);
//                                      749 + 2613
#include "attn_seq.h"

namespace staple {

using F32 = float;

// The wave's reads of its LDS have completed: what follows may overwrite it.
__device__ __forceinline__ void lds_reads_done() {
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
  __builtin_amdgcn_s_waitcnt(0xF | (3 << 14) | (7 << 4));   // lgkmcnt(0) only
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
}
// The wave's loads into LDS but the last N instructions have arrived.
template <int N>
__device__ __forceinline__ void loads_done() {
  wait_vmcnt<N>();
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
}

template <int DP>
struct F32Shape {
  static constexpr int kBlock = 32 * Tile<F32, DP>::kRow;
  static constexpr int kPerWave = 2 * kBlock + 512;   // two blocks, two rows of statistics
  static constexpr int kLds = kWaves * kPerWave;
  // The forward of wide heads holds one block a wave, keys and values in turn:
  // what a wave then waits for its loads the second workgroup of the CU uses.  2
  // x 4096 tokens, 16 heads of 128, window 1024: 592 us; 777 with two blocks a
  // wave and one workgroup.
  static constexpr bool kTurns = DP > 64;
  // With 64-bit addresses (kWide) two would spill 39 registers a lane: 512 tokens
  // of the same heads on 4 take 45 us with one workgroup and 54 with two, 2 x
  // 4096 with the window 891 and 914, 4 x 2048 without 977 and 963.
  static constexpr int fwd_workgroups(bool wide) { return wide && kTurns ? 1 : 2; }
  static constexpr int kFwdPerWave = kTurns ? kBlock : kPerWave, kFwdLds = kWaves * kFwdPerWave;
};

// Adds the waves' parts x[0 .. N) (each times the wave's own factor `mine`): a
// wave gets results wave_id(), wave_id() + 4, ... in out[].
template <int DP, int kPerWave, int N>
__device__ __forceinline__ void join_waves(char* smem, const f32x16_t (&x)[N], float mine, f32x16_t (&out)[(N + kWaves - 1) / kWaves]) {
  static_assert(N * 64 * 64 <= kPerWave, "the parts lie where the blocks were");
  const int lane = threadIdx.x & 63, w = wave_id();
  __syncthreads();
  f32x4_t* own = reinterpret_cast<f32x4_t*>(smem + w * kPerWave) + lane;
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int g = 0; g < 4; ++g)
      own[(i * 4 + g) * 64] = f32x4_t{x[i][4 * g] * mine, x[i][4 * g + 1] * mine, x[i][4 * g + 2] * mine, x[i][4 * g + 3] * mine};
  __syncthreads();
#pragma unroll
  for (int o = 0; o < (N + kWaves - 1) / kWaves; ++o) {
    const int i = o * kWaves + w;
    out[o] = f32x16_t{};
    if (i >= N) continue;
    for (int u = 0; u < kWaves; ++u)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const f32x4_t v = reinterpret_cast<const f32x4_t*>(smem + u * kPerWave)[(i * 4 + g) * 64 + lane];
#pragma unroll
        for (int e = 0; e < 4; ++e) out[o][4 * g + e] += v[e];
      }
  }
}

// ------------------------------------------------------------------- forward
template <int DP, bool kWide>
__global__ __launch_bounds__(64 * kWaves, F32Shape<DP>::fwd_workgroups(kWide)) void attn_fwd_f32_kernel(AttnView a, int64_t n_slots, KeyParts parts, int* err) {
  using TL = Tile<F32, DP>;
  using Loader = TileLoader<F32, DP, 32, 1, kWide>;
  using Shape = F32Shape<DP>;
  constexpr bool kTurns = Shape::kTurns;
  constexpr int kUnder = kTurns ? 0 : Loader::kPer;   // loads that may be under way when a block is read
  extern __shared__ __align__(1024) char smem[];
  __shared__ float tops[kWaves][32], sums[kWaves][32];
  check_offsets(a, err);
  QueryCols w;
  const int tile = static_cast<int>(blockIdx.x) / parts.n, part = static_cast<int>(blockIdx.x) - tile * parts.n;
  if (!w.find(a, kF32RowsLog2, n_slots, tile, 0, err)) return;
  KeyBlocks keys = w.blocks(a);
  int shares = 1;
  if (parts.n > 1) {
    shares = keys.share(parts.n, part);
    if (part >= shares) return;
  }
  const int lane = threadIdx.x & 63, wave = wave_id();
  lds_char* const kt = (lds_char*)smem + wave * Shape::kFwdPerWave;
  lds_char* const vt = kTurns ? kt : kt + Shape::kBlock;
  Loader kl, vl;
  kl.init(a.k, w.k0, w.nk, w.hk, a.head_dim, 0);
  vl.init(a.v, w.k0, w.nk, w.hk, a.head_dim, 0);
  kl.load(keys.first(wave), kt);
  u32x4_t qf[TL::kSteps];
  const float c = load_queries<F32, DP>(a, w, qf);
  f32x16_t o[TL::kDT] = {};
  ColumnSoftmax sm;
  if constexpr (!kTurns) vl.load(keys.first(wave), vt);
  for (int b = wave; b < keys.n; b += kWaves) {
    loads_done<kUnder>();   // K
    f32x16_t s = {};
#pragma unroll
    for (int st = 0; st < TL::kSteps; ++st) s = mma16(TL::row_frag(kt, 0, st), qf[st], s, F32{});
    lds_reads_done();
    if constexpr (kTurns) vl.load(keys.first(b), vt);
    else kl.load(keys.first(b + kWaves), kt);
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
    Column<F32> p;
    p.set(s);
    loads_done<kUnder>();   // V
#pragma unroll
    for (int d = 0; d < TL::kDT; ++d) o[d] = mma_transposed<DP>(vt, 0, d, p, o[d]);
    lds_reads_done();
    if constexpr (kTurns) kl.load(keys.first(b + kWaves), kt);
    else vl.load(keys.first(b + kWaves), vt);
  }
  loads_done<0>();   // none outlives the workgroup
  // the waves' references and sums, then their values relative to the largest
  const float sum = sm.sum + other_half(sm.sum);
  if (lane < 32) {
    tops[wave][lane] = sm.top;
    sums[wave][lane] = sum;
  }
  __syncthreads();
  float top = -INFINITY, total = 0.0f;
#pragma unroll
  for (int u = 0; u < kWaves; ++u) top = fmaxf(top, tops[u][lane & 31]);
#pragma unroll
  for (int u = 0; u < kWaves; ++u) total += sums[u][lane & 31] * rebase(tops[u][lane & 31], sums[u][lane & 31], top);
  constexpr int kOut = (TL::kDT + kWaves - 1) / kWaves;
  f32x16_t out[kOut];
  join_waves<DP, Shape::kFwdPerWave>(smem, o, rebase(sm.top, sum, top), out);
  if (shares == 1) return finish_dims<F32, DP>(a, w, kWaves, top, total, out);
  if (wave == 0) parts.put_rows(blockIdx.x, top, total);
#pragma unroll
  for (int i = 0; i < kOut; ++i)
    if (i * kWaves + wave < TL::kDT) parts.put<TL::kDT>(blockIdx.x, i * kWaves + wave, out[i]);
}

// ------------------------------------------------------------------ backward
template <int DP, bool kWide>
__global__ __launch_bounds__(64 * kWaves, 1) void attn_dq_f32_kernel(AttnView a, int64_t n_slots, KeyParts parts, RowStats stats,
                                                                     DkvPlan plan, int* err) {
  using TL = Tile<F32, DP>;
  using Loader = TileLoader<F32, DP, 32, 1, kWide>;
  constexpr int kBlock = F32Shape<DP>::kBlock;
  extern __shared__ __align__(1024) char smem[];
  check_offsets(a, err);
  if (blockIdx.x == 0) {
    plan_dkv(a, plan, err);
    return;
  }
  QueryCols w;
  const int id = static_cast<int>(blockIdx.x) - 1, tile = id / parts.n, part = id - tile * parts.n;
  if (!w.find(a, kF32RowsLog2, n_slots, tile, 0, err)) return;
  KeyBlocks keys = w.blocks(a);
  int shares = 1;
  if (parts.n > 1) {
    shares = keys.share(parts.n, part);
    if (part >= shares) return;
  }
  const int lane = threadIdx.x & 63, wave = wave_id();
  lds_char* const kt = (lds_char*)smem + wave * F32Shape<DP>::kPerWave;
  lds_char* const vt = kt + kBlock;
  Loader kl, vl;
  kl.init(a.k, w.k0, w.nk, w.hk, a.head_dim, 0);
  vl.init(a.v, w.k0, w.nk, w.hk, a.head_dim, 0);
  kl.load(keys.first(wave), kt);
  vl.load(keys.first(wave), vt);
  u32x4_t qf[TL::kSteps], dof[TL::kSteps];
  float delta = 0.0f;
#pragma unroll
  for (int s = 0; s < TL::kSteps; ++s) {
    dof[s] = load_frag<F32>(a.d_o, w.q0 + w.row, w.head, a.head_dim, s, w.in);
    delta += dot_frag(dof[s], load_frag<F32>(a.o, w.q0 + w.row, w.head, a.head_dim, s, w.in), F32{});
  }
  delta += other_half(delta);
  const float lse = w.in ? a.lse[(w.q0 + w.row) * a.n_heads + w.head] : 0.0f;
  const float lse2 = lse == -INFINITY ? 0.0f : lse * kLog2e;
  if (wave == 0 && part == 0 && w.in && lane < 32) {
    stats.lse2[w.head * a.total_q + w.q0 + w.row] = lse2;
    stats.delta[w.head * a.total_q + w.q0 + w.row] = delta;
  }
  const float c = load_queries<F32, DP>(a, w, qf);
  f32x16_t dq[TL::kDT] = {};
  for (int b = wave; b < keys.n; b += kWaves) {
    loads_done<0>();
    f32x16_t s = {}, dp = {};
#pragma unroll
    for (int st = 0; st < TL::kSteps; ++st) dp = mma16(TL::row_frag(vt, 0, st), dof[st], dp, F32{});
    lds_reads_done();
    vl.load(keys.first(b + kWaves), vt);
#pragma unroll
    for (int st = 0; st < TL::kSteps; ++st) s = mma16(TL::row_frag(kt, 0, st), qf[st], s, F32{});
    const bool whole = keys.whole(b);
    const SeenKeys seen(a, w.p, w.in, keys.first(b));
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      const float g = __builtin_amdgcn_exp2f(fmaf(s[r], c, -lse2)) * (dp[r] - delta);
      s[r] = (whole | seen(r)) ? g : 0.0f;
    }
    Column<F32> ds;
    ds.set(s);
#pragma unroll
    for (int d = 0; d < TL::kDT; ++d) dq[d] = mma_transposed<DP>(kt, 0, d, ds, dq[d]);
    lds_reads_done();
    kl.load(keys.first(b + kWaves), kt);
  }
  loads_done<0>();
  constexpr int kOut = (TL::kDT + kWaves - 1) / kWaves;
  f32x16_t out[kOut];
  join_waves<DP, F32Shape<DP>::kPerWave>(smem, dq, 1.0f, out);
  if (shares == 1) return finish_dq_dims<F32, DP>(a, w, kWaves, out);
#pragma unroll
  for (int i = 0; i < kOut; ++i)
    if (i * kWaves + wave < TL::kDT) parts.put<TL::kDT>(id, i * kWaves + wave, out[i]);
}

template <int DP, bool kWide>
__global__ __launch_bounds__(64 * kWaves, 1) void attn_dkv_f32_kernel(AttnView a, RowStats stats, DkvPlan plan) {
  using TL = Tile<F32, DP>;
  using Loader = TileLoader<F32, DP, 32, 1, kWide>;
  constexpr int kBlock = F32Shape<DP>::kBlock;
  extern __shared__ __align__(1024) char smem[];
  DkvItem w;
  if (!w.find(a, plan, 0)) return;
  const int lane = threadIdx.x & 63, wave = wave_id();
  lds_char* const qt = (lds_char*)smem + wave * F32Shape<DP>::kPerWave;
  lds_char* const dt = qt + kBlock;
  lds_char* const st = dt + kBlock;
  // the wave's blocks: number `at`, at + 4, ... of the item's, block bn of head h0 + g
  int at = wave, g = 0, bn = w.ln + wave;
  auto settle = [&]() {
    while (bn >= w.per_head) {
      bn -= w.per_head;
      ++g;
    }
  };
  Loader ql, dl;
  ql.init(a.q, w.q0, w.nq, w.h0, a.head_dim, 0);
  dl.init(a.d_o, w.q0, w.nq, w.h0, a.head_dim, 0);
  const char* const q_base = ql.base;
  const char* const d_base = dl.base;
  auto load = [&]() {
    if (at >= w.n) return;
    const int64_t head = g * static_cast<int64_t>(sizeof(F32));
    ql.set_base(q_base + head * a.q.head_stride);
    dl.set_base(d_base + head * a.d_o.head_stride);
    const int i0 = (w.b_lo + bn) * 32;
    ql.load(i0, qt);
    dl.load(i0, dt);
    const int64_t row = (w.h0 + g) * a.total_q + w.q0 + min(i0 + lane, w.nq - 1);
    dma4(stats.lse2 + row, static_cast<lds_void*>(st));
    dma4(stats.delta + row, static_cast<lds_void*>(st + 256));
  };
  f32x16_t x[2 * TL::kDT] = {};   // dk, then dv
  const float c = score_factor(a);
  if (w.n > 0) {
    settle();
    load();
    u32x4_t kf[TL::kSteps], vf[TL::kSteps];
#pragma unroll
    for (int s = 0; s < TL::kSteps; ++s) {
      kf[s] = signed_frag<F32>(a, load_frag<F32>(a.k, w.k0 + w.key, w.hk, a.head_dim, s, w.in));
      vf[s] = load_frag<F32>(a.v, w.k0 + w.key, w.hk, a.head_dim, s, w.in);
    }
    for (; at < w.n;) {
      loads_done<0>();
      f32x16_t s = {}, ds = {};
#pragma unroll
      for (int i = 0; i < TL::kSteps; ++i) {
        s = mma16(TL::row_frag(qt, 0, i), kf[i], s, F32{});
        ds = mma16(TL::row_frag(dt, 0, i), vf[i], ds, F32{});
      }
      const bool every = w.whole(bn);
      const SeenBy seen(a, w, w.key, w.in, (w.b_lo + bn) * 32);
      const lds_char* const rows = st + 16 * (lane >> 5);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const f32x4_t l4 = *reinterpret_cast<const lds_f32x4*>(rows + 32 * q);
        const f32x4_t d4 = *reinterpret_cast<const lds_f32x4*>(rows + 256 + 32 * q);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int r = 4 * q + e;
          const bool yes = every | seen(r);
          const float pr = __builtin_amdgcn_exp2f(fmaf(s[r], c, -l4[e]));
          ds[r] = yes ? pr * (ds[r] - d4[e]) : 0.0f;
          s[r] = yes ? pr : 0.0f;
        }
      }
      Column<F32> pc, dc;
      pc.set(s);
      dc.set(ds);
#pragma unroll
      for (int d = 0; d < TL::kDT; ++d) {
        x[d] = mma_transposed<DP>(qt, 0, d, dc, x[d]);
        x[TL::kDT + d] = mma_transposed<DP>(dt, 0, d, pc, x[TL::kDT + d]);
      }
      lds_reads_done();
      at += kWaves;
      bn += kWaves;
      settle();
      load();
    }
  }
  constexpr int kOut = 2 * TL::kDT / kWaves;
  f32x16_t out[kOut];
  join_waves<DP, F32Shape<DP>::kPerWave>(smem, x, 1.0f, out);
  if (w.parts > 1) {
    f32x4_t* to = part_sums<2 * TL::kDT>(plan, w.sums + w.part, w.hk, a.n_kv_heads, 0);
#pragma unroll
    for (int i = 0; i < kOut; ++i) put_sums(to, i * kWaves + wave, out[i]);
    return;
  }
  bool bad = false;
#pragma unroll
  for (int i = 0; i < kOut; ++i) {
    const int d = i * kWaves + wave;
    const bool value = d >= TL::kDT;
    bad |= has_unexplained<F32>(a, stats, w, value, value ? d - TL::kDT : d, out[i]);
    store_column<F32>(value ? a.dv : a.dk, w.k0 + w.key, w.hk, a.head_dim, value ? d - TL::kDT : d, out[i], value ? 1.0f : a.scale,
                      w.in);
  }
  redo_keys<F32>(a, stats, w, bad, 0, 1, kWaves, wave);
}

// ------------------------------------------------------------------- launches
template <int DP, bool kWide>
static hipError_t fwd_launch(const AttnView& a, const KeyParts& parts, hipStream_t s, int* err) {
  const int64_t n = tile_slots(a.total_q, a.n_seqs, kF32RowsLog2);
  const hipError_t e =
      launch_lds<attn_fwd_f32_kernel<DP, kWide>, F32Shape<DP>::kFwdLds>(n * a.n_heads * parts.n, s, a, n, parts, err);
  return e != hipSuccess ? e : launch_join<F32, DP, false>(a, kF32RowsLog2, n, parts, s, err);
}

hipError_t launch_attn_fwd_f32(const AttnView& a, void* ws, hipStream_t s, int* err) {
  Workspace w(ws, ~size_t(0));
  const KeyParts parts = take_parts(a, kF32RowsLog2, w);
  const bool far = spans_buffer(a.k, a.total_k, 4) || spans_buffer(a.v, a.total_k, 4);
  if (a.head_dim <= 64) return far ? fwd_launch<64, true>(a, parts, s, err) : fwd_launch<64, false>(a, parts, s, err);
  return far ? fwd_launch<128, true>(a, parts, s, err) : fwd_launch<128, false>(a, parts, s, err);
}

template <int DP, bool kWide>
static hipError_t bwd_launch(const AttnView& a, const BwdSpace& b, hipStream_t s, int* err) {
  const int64_t n = tile_slots(a.total_q, a.n_seqs, kF32RowsLog2);
  // one workgroup more than there are query tiles: it makes the plan
  hipError_t e = launch_lds<attn_dq_f32_kernel<DP, kWide>, F32Shape<DP>::kLds>(n * a.n_heads * b.parts.n + 1, s, a, n, b.parts,
                                                                               b.stats, b.plan, err);
  if (e != hipSuccess) return e;
  e = launch_join<F32, DP, true>(a, kF32RowsLog2, n, b.parts, s, err);
  if (e != hipSuccess) return e;
  const int64_t items = (b.plan.n_slots + b.plan.max_parts) * a.n_kv_heads;   // at most
  e = launch_lds<attn_dkv_f32_kernel<DP, kWide>, F32Shape<DP>::kLds>(items, s, a, b.stats, b.plan);
  return e != hipSuccess ? e : launch_dkv_join<F32, DP>(a, b, s);
}

hipError_t launch_attn_bwd_f32(const AttnView& a, const BwdSpace& b, hipStream_t s, int* err) {
  const bool far = spans_buffer(a.q, a.total_q, 4) || spans_buffer(a.d_o, a.total_q, 4) || spans_buffer(a.k, a.total_k, 4) ||
                   spans_buffer(a.v, a.total_k, 4);
  if (a.head_dim <= 64) return far ? bwd_launch<64, true>(a, b, s, err) : bwd_launch<64, false>(a, b, s, err);
  return far ? bwd_launch<128, true>(a, b, s, err) : bwd_launch<128, false>(a, b, s, err);
}

}  // namespace staple
