// Norms before and after a block, with the block's gate and residual sum.
//
//   b = z / rms(z) w_post  (or z),   r = x + s gate b,   h = r / rms(r) w_pre,
//   rms(v) = sqrt(mean(v^2) + eps)
//
// backward, with t = dh w_pre and hat(v) = v / rms(v):
//   dx = g = dr + (t - hat(r) mean(t hat(r))) / rms(r),       dw_pre = sum over rows of dh hat(r)
//   dgate = s g b,   q = s gate g,
//   dz = q, or (q w_post - hat(z) mean(q w_post hat(z))) / rms(z),   dw_post = sum of q hat(z)
//
// Bound by bytes: a row stays in registers between its sums and its outputs, so that each operand is read
// once.  32768 x 2048 in bf16, both norms and a gate shared by the rows: forward 112 us (4.8 TB/s), backward,
// which reads x and z again, 146 (5.5 TB/s), and 6 for the sums over the rows.  16384 x 4096 with x and r in
// fp32: 145 to 169 (4.8 to 5.5 TB/s) and 169 (6.4).
#include "model_ops.h"
#include "row_io.h"

namespace staple {

// Eight elements of a vector shared by the rows (ones when NULL).
template <int T, Layout LAYOUT>
__device__ __forceinline__ void load_shared(const void* p, bool bf16, int g, int t, int d, float (&v)[8]) {
  using R = RowGroup<T, LAYOUT>;
  if (p == nullptr) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 1.0f;
  } else if (bf16) {
    R::load(static_cast<const bf16_t*>(p), g, t, d, v);
  } else {
    R::load(static_cast<const float*>(p), g, t, d, v);
  }
}

template <typename E>
__device__ __forceinline__ E* row_of(const RowsView& v, int64_t i) {
  return reinterpret_cast<E*>(v.data) + i * v.stride;
}

// T lanes a row, G groups of eight elements a lane; rows of one wave share a workgroup.
template <typename X, typename Z, int T, int G, Layout LAYOUT>
__global__ __launch_bounds__(T < 256 ? 256 : T) void norm_fwd_kernel(NormView a) {
  using R = RowGroup<T, LAYOUT>;
  constexpr int kRows = T < 256 ? 256 / T : 1;
  __shared__ float tmp[2][kRows][T < 64 ? 1 : T / 64];
  const int t = threadIdx.x % T, slot = threadIdx.x / T, d = a.d;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kRows + slot;
  if (i >= a.n_rows) return;   // T >= 256: the whole workgroup; otherwise lanes that meet no barrier
  const float inv_d = 1.0f / static_cast<float>(d);
  float r[G][8], b[G][8];
#pragma unroll
  for (int g = 0; g < G; ++g) {
    if (a.x.data) R::load(row_of<const X>(a.x, i), g, t, d, r[g]);
    if (a.z.data) R::load(row_of<const Z>(a.z, i), g, t, d, b[g]);
  }
  if (a.z.data) {
    float rstd = a.scale;
    if (a.post) {
      float ss = 0.0f;
#pragma unroll
      for (int g = 0; g < G; ++g)
#pragma unroll
        for (int k = 0; k < 8; ++k) ss += b[g][k] * b[g][k];
      const float inv = rsqrtf(row_sum<T>(ss, tmp[0][slot], t) * inv_d + a.eps);
      if (a.rstd_z && t == 0) a.rstd_z[i] = inv;
      rstd *= inv;
    }
#pragma unroll
    for (int g = 0; g < G; ++g) {
      float w[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) b[g][k] *= rstd;
      if (a.post && a.w_post) {
        load_shared<T, LAYOUT>(a.w_post, a.w_bf16, g, t, d, w);
#pragma unroll
        for (int k = 0; k < 8; ++k) b[g][k] *= w[k];
      }
      if (a.gate_kind != Gate::kNone) {
        if (a.gate_kind == Gate::kVector) load_shared<T, LAYOUT>(a.gate.data, a.w_bf16, g, t, d, w);
        else R::load(row_of<const Z>(a.gate, i), g, t, d, w);
#pragma unroll
        for (int k = 0; k < 8; ++k) b[g][k] *= w[k];
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) r[g][k] = a.x.data ? r[g][k] + b[g][k] : b[g][k];
      R::store(row_of<X>(a.r, i), g, t, d, r[g]);
    }
  }
  if (!a.pre) return;
  float ss = 0.0f;
#pragma unroll
  for (int g = 0; g < G; ++g)
#pragma unroll
    for (int k = 0; k < 8; ++k) ss += r[g][k] * r[g][k];
  const float inv = rsqrtf(row_sum<T>(ss, tmp[1][slot], t) * inv_d + a.eps);
  if (a.rstd_r && t == 0) a.rstd_r[i] = inv;
#pragma unroll
  for (int g = 0; g < G; ++g) {
    float w[8];
    load_shared<T, LAYOUT>(a.w_pre, a.w_bf16, g, t, d, w);
#pragma unroll
    for (int k = 0; k < 8; ++k) r[g][k] *= inv * w[k];
    R::store(row_of<Z>(a.h, i), g, t, d, r[g]);
  }
}

// V (4 or 8) elements of a row that a lane of the backward holds of group g, as they lie in memory: as in a
// RowGroup, with V for eight.
template <typename E, int T, Layout LAYOUT, int V>
struct Part {
  static constexpr int kWords = LAYOUT == kSingle ? V : V * static_cast<int>(sizeof(E)) / 4;
  typedef __attribute__((ext_vector_type(kWords))) uint32_t words_t;
  typedef typename LooseWords<E, kWords>::type loose_t;
  words_t w;
  __device__ __forceinline__ static int column(int g, int t, int i) {
    return LAYOUT == kSingle ? (g * V + i) * T + t : (g * T + t) * V + i;
  }
  __device__ __forceinline__ static int skip(int g, int t, int d) { return max(column(g, t, 0) - (d - V), 0); }
  // ONCE: rows, which nothing reads again soon, past the caches
  template <bool ONCE>
  __device__ __forceinline__ void load(const E* row, int g, int t, int d) {
    if (LAYOUT == kAligned) {   // lanes past the end: the last elements again
      const words_t* p = reinterpret_cast<const words_t*>(row + min(column(g, t, 0), d - V));
      w = ONCE ? __builtin_nontemporal_load(p) : *p;
    } else if (LAYOUT == kLoose) {
      const loose_t* p = reinterpret_cast<const loose_t*>(row + min(column(g, t, 0), d - V));
      w = ONCE ? __builtin_nontemporal_load(p) : *p;
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) w[i] = __float_as_uint(load1(row + min(column(g, t, i), d - 1)));
    }
  }
  // 0 past the row's end.
  __device__ __forceinline__ void get(float (&v)[V], int g, int t, int d) const {
    const int none = skip(g, t, d);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if (LAYOUT != kSingle && sizeof(E) == 2) v[i] = __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
      else v[i] = __uint_as_float(w[i]);
      if (LAYOUT == kLoose ? i < none : column(g, t, i) >= d) v[i] = 0.0f;
    }
  }
  __device__ __forceinline__ static void store(E* row, int g, int t, int d, const float (&v)[V]) {
    if (LAYOUT == kSingle) {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (column(g, t, i) < d) store1(row + column(g, t, i), v[i]);
      return;
    }
    const int none = skip(g, t, d);
    if (none == 0) {
      words_t x;
#pragma unroll
      for (int i = 0; i < kWords; ++i) {
        if (sizeof(E) == 2) x[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
        else x[i] = __float_as_uint(v[i]);
      }
      E* p = row + column(g, t, 0);
      if (LAYOUT == kAligned) *reinterpret_cast<words_t*>(p) = x;
      else *reinterpret_cast<loose_t*>(p) = x;
    } else if (LAYOUT == kLoose && none < V) {
#pragma unroll
      for (int i = 1; i < V; ++i)
        if (i >= none) store1(row + d - V + i, v[i]);
    }
  }
};

// A vector shared by the rows: ones when NULL.
template <int T, Layout LAYOUT, int V>
__device__ __forceinline__ void load_vector(const void* p, bool bf16, int g, int t, int d, float (&v)[V]) {
  if (p == nullptr) {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = 1.0f;
  } else if (bf16) {
    Part<bf16_t, T, LAYOUT, V> x;
    x.template load<false>(static_cast<const bf16_t*>(p), g, t, d);
    x.get(v, g, t, d);
  } else {
    Part<float, T, LAYOUT, V> x;
    x.template load<false>(static_cast<const float*>(p), g, t, d);
    x.get(v, g, t, d);
  }
}

// What the backward reads of group g of a row.
template <typename X, typename Z, int T, Layout LAYOUT, int V>
struct NormRow {
  Part<X, T, LAYOUT, V> dr, r;   // r: the stored sum, or x
  Part<Z, T, LAYOUT, V> dh, z, gate;
  float rstd_r, rstd_z;
  template <bool ONCE>
  __device__ __forceinline__ void load(const NormView& a, int64_t i, int g, int t, bool need_z) {
    const RowsView& sum = a.r.data ? a.r : a.x;
    if (a.dr.data) dr.template load<ONCE>(row_of<const X>(a.dr, i), g, t, a.d);
    if (a.pre) {
      if (sum.data) r.template load<ONCE>(row_of<const X>(sum, i), g, t, a.d);
      dh.template load<ONCE>(row_of<const Z>(a.dh, i), g, t, a.d);
    }
    if (need_z) z.template load<ONCE>(row_of<const Z>(a.z, i), g, t, a.d);
    if (a.gate_kind == Gate::kRows) gate.template load<ONCE>(row_of<const Z>(a.gate, i), g, t, a.d);
    rstd_r = a.pre ? a.rstd_r[i] : 0.0f;
    rstd_z = a.post && need_z ? a.rstd_z[i] : 1.0f;   // given only where z is read
  }
};

// Waves a SIMD that the backward is held to the registers of; its grid fills the GPU with them once.
constexpr int norm_bwd_waves(int lanes, int v) { return lanes >= 512 || v == 4 ? 4 : 3; }

// Workgroups work off rows in turn, the next row's loads in flight, and keep the sums over their rows, and
// the weights, in registers; parts: [vectors][workgroups][d], added up by norm_columns_kernel in their
// order.  SLABS: a workgroup takes group blockIdx.y of its rows, T V columns, and norm_means_kernel's means,
// two a row, from the last row on, of which the caches still have most; otherwise whole rows, whose means it
// forms itself.
template <typename X, typename Z, int T, Layout LAYOUT, int V, bool SLABS>
__global__ __launch_bounds__(T < 256 ? 256 : T, norm_bwd_waves(T, V)) void norm_bwd_kernel(NormView a, const float* means,
                                                                                         float* parts) {
  constexpr int kRows = T < 256 ? 256 / T : 1;
  // two sums a row, in buffers of their own for rows in turn: between a sum's reads and the
  // next writes to its buffer stands the barrier of the row between
  __shared__ float tmp[2][2][kRows][T < 64 ? 1 : T / 64];
  const int t = threadIdx.x % T, slot = threadIdx.x / T, d = a.d, g = SLABS ? blockIdx.y : 0;
  const float inv_d = 1.0f / static_cast<float>(d);
  const int64_t slots = static_cast<int64_t>(gridDim.x) * kRows;
  const int64_t me = static_cast<int64_t>(blockIdx.x) * kRows + slot;
  const auto row_at = [&](int64_t i) { return SLABS ? a.n_rows - 1 - i : i; };
  const bool branch = norm_bwd_branch(a), need_z = norm_bwd_reads_z(a);
  const bool rows_gate = a.gate_kind == Gate::kRows;
  float sum_pre[V], sum_post[V], sum_gate[V], w_pre[V], w_post[V], gate[V];
#pragma unroll
  for (int k = 0; k < V; ++k) sum_pre[k] = sum_post[k] = sum_gate[k] = 0.0f;
  load_vector<T, LAYOUT, V>(a.w_pre, a.w_bf16, g, t, d, w_pre);
  load_vector<T, LAYOUT, V>(a.post ? a.w_post : nullptr, a.w_bf16, g, t, d, w_post);
  load_vector<T, LAYOUT, V>(rows_gate ? nullptr : a.gate.data, a.w_bf16, g, t, d, gate);
  NormRow<X, Z, T, LAYOUT, V> next;
  float next_mean = 0.0f, next_mean_z = 0.0f;
  const auto read_means = [&](int64_t i) {
    if (!SLABS) return;
    next_mean = means[2 * i];
    next_mean_z = means[2 * i + 1];
  };
  if (me < a.n_rows) read_means(row_at(me));
  if (me < a.n_rows) next.template load<!SLABS>(a, row_at(me), g, t, need_z);
  int odd = 0;
  for (int64_t i = me; i < a.n_rows; i += slots, odd ^= 1) {
    const int64_t at = row_at(i);
    const NormRow<X, Z, T, LAYOUT, V> row = next;
    const float given_mean = next_mean, given_mean_z = next_mean_z;
    if (i + slots < a.n_rows) read_means(row_at(i + slots));
    if (i + slots < a.n_rows) next.template load<!SLABS>(a, row_at(i + slots), g, t, need_z);
    float q[V], hat_z[V];
    const float inv_z = row.rstd_z;
    if (need_z) {
      row.z.get(hat_z, g, t, d);
#pragma unroll
      for (int k = 0; k < V; ++k) hat_z[k] *= inv_z;
    }
    if (rows_gate) row.gate.get(gate, g, t, d);
    if (a.pre) {
      const float inv = row.rstd_r;
      float hat[V], dt[V], dot = 0.0f;
      if (a.r.data) {
        row.r.get(hat, g, t, d);
      } else {   // as the forward had it before r was rounded
        float x[V];
#pragma unroll
        for (int k = 0; k < V; ++k) x[k] = 0.0f;
        if (a.x.data) row.r.get(x, g, t, d);
#pragma unroll
        for (int k = 0; k < V; ++k) hat[k] = x[k] + a.scale * gate[k] * w_post[k] * hat_z[k];
      }
      row.dh.get(dt, g, t, d);
#pragma unroll
      for (int k = 0; k < V; ++k) {
        hat[k] *= inv;
        sum_pre[k] += dt[k] * hat[k];
        dt[k] *= w_pre[k];
        dot += dt[k] * hat[k];
      }
      const float mean = SLABS ? given_mean : row_sum<T>(dot, tmp[odd][0][slot], t) * inv_d;
#pragma unroll
      for (int k = 0; k < V; ++k) q[k] = inv * (dt[k] - hat[k] * mean);
    } else {
#pragma unroll
      for (int k = 0; k < V; ++k) q[k] = 0.0f;
    }
    if (a.dr.data) {
      float v[V];
      row.dr.get(v, g, t, d);
#pragma unroll
      for (int k = 0; k < V; ++k) q[k] += v[k];
    }
    if (a.dx.data) Part<X, T, LAYOUT, V>::store(row_of<X>(a.dx, at), g, t, d, q);
    if (!branch) continue;
    float dot = 0.0f;
#pragma unroll
    for (int k = 0; k < V; ++k) q[k] *= a.scale;
    if (a.gate_kind != Gate::kNone) {
      if (a.dgate.data || a.dgate_sum) {
        float dg[V];
#pragma unroll
        for (int k = 0; k < V; ++k) {
          dg[k] = q[k] * hat_z[k] * w_post[k];
          sum_gate[k] += dg[k];
        }
        if (a.dgate.data) Part<Z, T, LAYOUT, V>::store(row_of<Z>(a.dgate, at), g, t, d, dg);
      }
#pragma unroll
      for (int k = 0; k < V; ++k) q[k] *= gate[k];
    }
    if (a.post) {
#pragma unroll
      for (int k = 0; k < V; ++k) {
        sum_post[k] += q[k] * hat_z[k];
        q[k] *= w_post[k];
        dot += q[k] * hat_z[k];
      }
      const float mean = SLABS ? given_mean_z : row_sum<T>(dot, tmp[odd][1][slot], t) * inv_d;
#pragma unroll
      for (int k = 0; k < V; ++k) q[k] = inv_z * (q[k] - hat_z[k] * mean);
    }
    if (a.dz.data) Part<Z, T, LAYOUT, V>::store(row_of<Z>(a.dz, at), g, t, d, q);
  }
  // the workgroup's rows in turn, then its part
  float* part = parts + static_cast<int64_t>(blockIdx.x) * d;
  const int64_t one = static_cast<int64_t>(gridDim.x) * d;
  const auto put = [&](float (&v)[V]) {
    if (kRows > 1) {
      __shared__ float all[kRows][V][T];
      __syncthreads();
#pragma unroll
      for (int k = 0; k < V; ++k) all[slot][k][t] = v[k];
      __syncthreads();
      for (int j = 1; j < kRows; ++j)
#pragma unroll
        for (int k = 0; k < V; ++k) v[k] = j == 1 ? all[0][k][t] + all[1][k][t] : v[k] + all[j][k][t];
    }
    if (slot == 0) Part<float, T, LAYOUT, V>::store(part, g, t, d, v);
    part += one;
  };
  if (a.dw_pre) put(sum_pre);
  if (a.dw_post) put(sum_post);
  if (a.dgate_sum) put(sum_gate);
}

// The means of wide rows, for norm_bwd_kernel's slabs, both from sums of one pass: with c = s gate w_post hat(z),
// a = dr + t / rms(r) and m = mean(t hat(r)),
//   g = a - hat(r) m / rms(r),    mean(q w_post hat(z)) = mean(c g) = mean(c a) - m mean(c hat(r) / rms(r)).
template <typename X, typename Z, Layout LAYOUT>
__global__ __launch_bounds__(512) void norm_means_kernel(NormView a, float* means) {
  constexpr int T = 512, V = 8;
  __shared__ float tmp[3][T / 64];
  const int t = threadIdx.x, d = a.d;
  const int64_t i = blockIdx.x;
  const bool need_z = norm_bwd_reads_z(a), rows_gate = a.gate_kind == Gate::kRows;
  float s[3] = {0.0f, 0.0f, 0.0f};
  for (int g = 0; g * T * V < d; ++g) {
    NormRow<X, Z, T, LAYOUT, V> row;
    row.template load<false>(a, i, g, t, need_z);
    float sums[V], hat[V], dh[V], hat_z[V], w_pre[V], w_post[V], gate[V];
    load_vector<T, LAYOUT, V>(a.pre ? a.w_pre : nullptr, a.w_bf16, g, t, d, w_pre);
    load_vector<T, LAYOUT, V>(a.post ? a.w_post : nullptr, a.w_bf16, g, t, d, w_post);
    if (rows_gate) row.gate.get(gate, g, t, d);
    else load_vector<T, LAYOUT, V>(a.gate.data, a.w_bf16, g, t, d, gate);
#pragma unroll
    for (int k = 0; k < V; ++k) sums[k] = hat[k] = dh[k] = hat_z[k] = 0.0f;
    if (need_z) row.z.get(hat_z, g, t, d);
    if (a.dr.data) row.dr.get(sums, g, t, d);
    if (a.pre) {
      row.dh.get(dh, g, t, d);
      if (a.r.data || a.x.data) row.r.get(hat, g, t, d);
    }
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const float c = a.scale * gate[k] * w_post[k] * (hat_z[k] * row.rstd_z), tk = dh[k] * w_pre[k];
      if (!a.r.data) hat[k] += c;   // as the forward had it
      hat[k] *= row.rstd_r;
      s[0] += tk * hat[k];
      s[1] += c * (sums[k] + row.rstd_r * tk);
      s[2] += c * (hat[k] * row.rstd_r);
    }
  }
#pragma unroll
  for (int j = 0; j < 3; ++j) {
    s[j] = wave_sum(s[j]);
    if ((t & 63) == 0) tmp[j][t >> 6] = s[j];
  }
  __syncthreads();
  if (t > 0) return;
  const float inv_d = 1.0f / static_cast<float>(d);
#pragma unroll
  for (int j = 0; j < 3; ++j) {
    s[j] = tmp[j][0];
#pragma unroll
    for (int k = 1; k < T / 64; ++k) s[j] += tmp[j][k];
    s[j] *= inv_d;
  }
  means[2 * i] = s[0];
  means[2 * i + 1] = s[1] - s[0] * s[2];
}

// Sums of the parts (slots), 16 columns a workgroup: 64 of its lanes a column, which add slots k, k + 64, ... and
// are then added up in turn.
__global__ __launch_bounds__(1024) void norm_columns_kernel(const float* __restrict__ parts, int slots, int d,
                                                            float* o0, float* o1, float* o2) {
  constexpr int kAhead = 8;
  __shared__ float tmp[64][16];
  const int c = threadIdx.x & 15, k0 = threadIdx.x >> 4;
  const int col = min(static_cast<int>(blockIdx.x) * 16 + c, d - 1);
  const float* p = parts + static_cast<int64_t>(blockIdx.y) * slots * d + col;
  float* out = blockIdx.y == 0 ? o0 : blockIdx.y == 1 ? o1 : o2;
  float s = 0.0f;
  for (int i = k0; i < slots; i += 64 * kAhead) {
    float v[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) v[u] = i + 64 * u < slots ? p[static_cast<int64_t>(i + 64 * u) * d] : 0.0f;
#pragma unroll
    for (int u = 0; u < kAhead; ++u) s += v[u];
  }
  tmp[k0][c] = s;
  __syncthreads();
  if (threadIdx.x >= 16 || static_cast<int>(blockIdx.x) * 16 + c >= d) return;
  s = 0.0f;
#pragma unroll 8
  for (int k = 0; k < 64; ++k) s += tmp[k][c];
  out[col] = s;
}

static bool vec_view(const RowsView& v, int bytes) {
  return v.data == nullptr || ((reinterpret_cast<uintptr_t>(v.data) & 15) == 0 && v.stride * bytes % 16 == 0);
}
static bool vec_ptr(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

static Layout norm_layout(const NormView& v, int32_t r_dtype, int32_t dtype) {
  const int xb = r_dtype == STAPLE_BF16 ? 2 : 4, zb = dtype == STAPLE_BF16 ? 2 : 4;
  const bool gate = v.gate_kind == Gate::kRows ? vec_view(v.gate, zb) : vec_ptr(v.gate.data);
  if (v.d < 8) return kSingle;
  const bool aligned =
      v.d % 8 == 0 && vec_view(v.x, xb) && vec_view(v.r, xb) && vec_view(v.dr, xb) && vec_view(v.dx, xb) &&
         vec_view(v.z, zb) && vec_view(v.h, zb) && vec_view(v.dh, zb) && vec_view(v.dz, zb) &&
         vec_view(v.dgate, zb) && gate && vec_ptr(v.w_pre) && vec_ptr(v.w_post);
  return aligned ? kAligned : kLoose;
}

// Lanes a row and groups of eight elements a lane: rows of up to 1024 in a wave or less, whose sums need no LDS,
// wider ones in four waves and more.  2048 in 64 x 4: 122 us, in 256 x 1 112 (32768 rows of bf16); 524288 rows of 64 in
// 8 lanes: 49 us, in 64 215.
#define NORM_SHAPES(GO)                          \
  do {                                           \
    if (v.d <= 64) GO(8, 1);                     \
    else if (v.d <= 128) GO(16, 1);              \
    else if (v.d <= 256) GO(32, 1);              \
    else if (v.d <= 512) GO(64, 1);              \
    else if (v.d <= 1024) GO(64, 2);             \
    else if (v.d <= 2048) GO(256, 1);            \
    else if (v.d <= 4096) GO(256, 2);            \
    else if (v.d <= 8192) GO(512, 2);            \
    else GO(1024, 2);                            \
  } while (0)

// The backward's, with elements a group: its sums, weights and loads in flight are some 20 registers an
// element, so that four elements a lane in more lanes leave more waves a SIMD: 2048 in 512 x 4 takes 153 us, in
// 256 x 8 233; 4096 in 1024 x 4 198, in 512 x 8 230 (both before rows were read past the caches); 64 in
// 16 lanes 76, in 64 176.
// Wider rows spill there (8192 with r in fp32: 252 to 350 us for 4096 rows; bf16, 16384: 493 for 2048) and are
// read twice, means first, then slabs of 1024 columns: 202 to 324, 149.  bf16 of 8192 in 1024 x 8: 92, in slabs 166.
// Of the shapes that are taken 1024 x 8 in bf16 spills 25 registers (rows at any element: 3), and 64 x 8 in fp32, for
// widths of 257 to 512, 5 (15): 32768 rows of 512 take 86 us, of 511 98, 60000 of 300 109, and in 256 x 4, which spills
// none, 87, 98 and 108.
#define NORM_BWD_SHAPES(GO, SLABS)                    \
  do {                                                \
    if (v.d <= 64) GO(16, 4);                         \
    else if (v.d <= 128) GO(32, 4);                   \
    else if (v.d <= 256) GO(64, 4);                   \
    else if (v.d <= 512) GO(64, 8);                   \
    else if (v.d <= 1024) GO(256, 4);                 \
    else if (v.d <= 2048) GO(512, 4);                 \
    else if (v.d <= 4096) GO(1024, 4);                \
    else if (v.d <= 8192 && v.r_bf16) GO(1024, 8);    \
    else SLABS(256, 4);                               \
  } while (0)
struct NormBwdShape {
  int lanes, elements, slabs;
  int rows() const { return lanes < 256 ? 256 / lanes : 1; }                 // of a workgroup
  int64_t workgroups() const {                                               // that fill the GPU
    const int waves = (lanes < 256 ? 256 : lanes) / 64;
    const int a_cu = norm_bwd_waves(lanes, elements) * 4 / waves;
    return (static_cast<int64_t>(device_cus()) * (a_cu > 0 ? a_cu : 1) + slabs - 1) / slabs;
  }
};
static NormBwdShape norm_bwd_shape(const NormView& v) {
#define GO(T, V) return NormBwdShape{T, V, 1}
#define SLABS(T, V) return NormBwdShape{T, V, (v.d + T * V - 1) / (T * V)}
  NORM_BWD_SHAPES(GO, SLABS);
#undef SLABS
#undef GO
}

template <typename X, typename Z, Layout LAYOUT>
static void norm_fwd(const NormView& v, hipStream_t s) {
#define GO(T, G)                                                                                    \
  do {                                                                                              \
    constexpr int kRows = T < 256 ? 256 / T : 1;                                                    \
    norm_fwd_kernel<X, Z, T, G, LAYOUT>                                                             \
        <<<dim3(static_cast<unsigned>((v.n_rows + kRows - 1) / kRows)), dim3(T * kRows), 0, s>>>(v); \
  } while (0)
  if constexpr (LAYOUT == kSingle) GO(8, 1);
  else NORM_SHAPES(GO);
#undef GO
}

static int norm_vectors(const NormView& v) {
  return (v.dw_pre != nullptr) + (v.dw_post != nullptr) + (v.dgate_sum != nullptr);
}

static int64_t norm_bwd_grid(const NormView& v) {
  const NormBwdShape shape = norm_bwd_shape(v);
  const int64_t all = (v.n_rows + shape.rows() - 1) / shape.rows(), most = shape.workgroups();
  return all < most ? all : most;
}

// Floats of the workspace before the parts: two means a row where there are slabs, in 16 bytes.
static size_t norm_means(const NormView& v) {
  return norm_bwd_shape(v).slabs > 1 ? (2 * static_cast<size_t>(v.n_rows) + 3) / 4 * 4 : 0;
}

size_t norm_bwd_workspace_bytes(const NormView& v) {
  return (norm_means(v) + static_cast<size_t>(norm_vectors(v)) * norm_bwd_grid(v) * v.d) * sizeof(float);
}

template <typename X, typename Z, Layout LAYOUT>
static void norm_bwd(const NormView& v, float* ws, hipStream_t s) {
  const NormBwdShape shape = norm_bwd_shape(v);
  const dim3 grid(static_cast<unsigned>(norm_bwd_grid(v)));
  float *means = ws, *parts = ws + norm_means(v);
  if (v.n_rows > 0) {
#define GO(T, V)                                                                                             \
  do {                                                                                                       \
    if constexpr (T * V <= 4096 || sizeof(X) == 2)                                                           \
      norm_bwd_kernel<X, Z, T, LAYOUT, V, false><<<grid, dim3(T < 256 ? 256 : T), 0, s>>>(v, nullptr, parts); \
  } while (0)
#define SLABS(T, V)                                                                                          \
  do {                                                                                                       \
    norm_means_kernel<X, Z, LAYOUT><<<dim3(static_cast<unsigned>(v.n_rows)), dim3(512), 0, s>>>(v, means);   \
    norm_bwd_kernel<X, Z, T, LAYOUT, V, true><<<dim3(grid.x, shape.slabs), dim3(T), 0, s>>>(v, means, parts); \
  } while (0)
    if constexpr (LAYOUT == kSingle) GO(16, 4);
    else NORM_BWD_SHAPES(GO, SLABS);
#undef SLABS
#undef GO
  }
  const int n = norm_vectors(v);
  if (n == 0) return;
  float* out[3] = {};
  int k = 0;
  for (float* p : {v.dw_pre, v.dw_post, v.dgate_sum})
    if (p) out[k++] = p;
  norm_columns_kernel<<<dim3((v.d + 15) / 16, n), dim3(1024), 0, s>>>(
      parts, static_cast<int>(grid.x), v.d, out[0], out[1], out[2]);
}

#define NORM_LAYOUTS(CALL, X, Z)                  \
  do {                                            \
    if (layout == kAligned) CALL(X, Z, kAligned); \
    else if (layout == kLoose) CALL(X, Z, kLoose); \
    else CALL(X, Z, kSingle);                     \
  } while (0)
#define NORM_TYPES(CALL)                                                         \
  const Layout layout = norm_layout(v, r_dtype, dtype);                          \
  if (r_dtype == STAPLE_BF16) NORM_LAYOUTS(CALL, bf16_t, bf16_t);                \
  else if (dtype == STAPLE_BF16) NORM_LAYOUTS(CALL, float, bf16_t);              \
  else NORM_LAYOUTS(CALL, float, float);

hipError_t launch_norm_fwd(const NormView& v, int32_t r_dtype, int32_t dtype, hipStream_t s) {
#define CALL(X, Z, V) norm_fwd<X, Z, V>(v, s)
  NORM_TYPES(CALL)
#undef CALL
  return hipGetLastError();
}

hipError_t launch_norm_bwd(const NormView& v, int32_t r_dtype, int32_t dtype, void* ws, hipStream_t s) {
#define CALL(X, Z, V) norm_bwd<X, Z, V>(v, static_cast<float*>(ws), s)
  NORM_TYPES(CALL)
#undef CALL
  return hipGetLastError();
}

}  // namespace staple
