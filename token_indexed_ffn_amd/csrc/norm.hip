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
template <int T, bool VEC>
__device__ __forceinline__ void load_shared(const void* p, bool bf16, int g, int t, int d, float (&v)[8]) {
  using R = RowGroup<T, VEC>;
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
template <typename X, typename Z, int T, int G, bool VEC>
__global__ __launch_bounds__(T < 256 ? 256 : T) void norm_fwd_kernel(NormView a) {
  using R = RowGroup<T, VEC>;
  constexpr int kRows = T < 256 ? 256 / T : 1;
  __shared__ float tmp[2][kRows][T / 64];
  const int t = threadIdx.x % T, slot = threadIdx.x / T, d = a.d;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kRows + slot;
  if (i >= a.n_rows) return;   // T >= 256: the whole workgroup; T = 64: a wave, which meets no barrier
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
        load_shared<T, VEC>(a.w_post, a.w_bf16, g, t, d, w);
#pragma unroll
        for (int k = 0; k < 8; ++k) b[g][k] *= w[k];
      }
      if (a.gate_kind != Gate::kNone) {
        if (a.gate_kind == Gate::kVector) load_shared<T, VEC>(a.gate.data, a.w_bf16, g, t, d, w);
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
    load_shared<T, VEC>(a.w_pre, a.w_bf16, g, t, d, w);
#pragma unroll
    for (int k = 0; k < 8; ++k) r[g][k] *= inv * w[k];
    R::store(row_of<Z>(a.h, i), g, t, d, r[g]);
  }
}

// V (4 or 8) elements of a row that a lane of the backward holds of group g, as they lie in memory where
// they are aligned (VEC): elements (g T + t) V on, otherwise (g V + i) T + t.
template <typename E, int T, bool VEC, int V>
struct Part {
  static constexpr int kWords = VEC ? V * static_cast<int>(sizeof(E)) / 4 : V;
  typedef __attribute__((ext_vector_type(kWords))) uint32_t words_t;
  words_t w;
  __device__ __forceinline__ static int column(int g, int t, int i) { return VEC ? (g * T + t) * V + i : (g * V + i) * T + t; }
  // ONCE: rows, which nothing reads again soon, past the caches
  template <bool ONCE>
  __device__ __forceinline__ void load(const E* row, int g, int t, int d) {
    if (VEC) {   // lanes past the end: the last elements again
      const words_t* p = reinterpret_cast<const words_t*>(row + min(column(g, t, 0), d - V));
      w = ONCE ? __builtin_nontemporal_load(p) : *p;
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) w[i] = __float_as_uint(load1(row + min(column(g, t, i), d - 1)));
    }
  }
  // 0 past the row's end.
  __device__ __forceinline__ void get(float (&v)[V], int g, int t, int d) const {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if (VEC && sizeof(E) == 2) v[i] = __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
      else v[i] = __uint_as_float(w[i]);
      if (column(g, t, i) >= d) v[i] = 0.0f;
    }
  }
  __device__ __forceinline__ static void store(E* row, int g, int t, int d, const float (&v)[V]) {
    if (VEC) {
      if (column(g, t, 0) >= d) return;
      words_t x;
#pragma unroll
      for (int i = 0; i < kWords; ++i) {
        if (sizeof(E) == 2) x[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
        else x[i] = __float_as_uint(v[i]);
      }
      *reinterpret_cast<words_t*>(row + column(g, t, 0)) = x;
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (column(g, t, i) < d) store1(row + column(g, t, i), v[i]);
    }
  }
};

// A vector shared by the rows: ones when NULL.
template <int T, bool VEC, int V>
__device__ __forceinline__ void load_vector(const void* p, bool bf16, int g, int t, int d, float (&v)[V]) {
  if (p == nullptr) {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = 1.0f;
  } else if (bf16) {
    Part<bf16_t, T, VEC, V> x;
    x.template load<false>(static_cast<const bf16_t*>(p), g, t, d);
    x.get(v, g, t, d);
  } else {
    Part<float, T, VEC, V> x;
    x.template load<false>(static_cast<const float*>(p), g, t, d);
    x.get(v, g, t, d);
  }
}

// What the backward reads of a row.
template <typename X, typename Z, int T, int G, bool VEC, int V>
struct NormRow {
  Part<X, T, VEC, V> dr[G], r[G];   // r: the stored sum, or x
  Part<Z, T, VEC, V> dh[G], z[G], gate[G];
  float rstd_r, rstd_z;
  __device__ __forceinline__ void load(const NormView& a, int64_t i, int t, bool need_z) {
    const RowsView& sum = a.r.data ? a.r : a.x;
#pragma unroll
    for (int g = 0; g < G; ++g) {
      if (a.dr.data) dr[g].template load<true>(row_of<const X>(a.dr, i), g, t, a.d);
      if (a.pre) {
        if (sum.data) r[g].template load<true>(row_of<const X>(sum, i), g, t, a.d);
        dh[g].template load<true>(row_of<const Z>(a.dh, i), g, t, a.d);
      }
      if (need_z) z[g].template load<true>(row_of<const Z>(a.z, i), g, t, a.d);
      if (a.gate_kind == Gate::kRows) gate[g].template load<true>(row_of<const Z>(a.gate, i), g, t, a.d);
    }
    rstd_r = a.pre ? a.rstd_r[i] : 0.0f;
    rstd_z = a.post ? a.rstd_z[i] : 1.0f;
  }
};

// Waves a SIMD that the backward is held to the registers of; its grid fills the GPU with them once.
constexpr int norm_bwd_waves(int lanes, int v) { return lanes >= 512 ? 4 : v == 4 ? 5 : 3; }

// Workgroups work off rows in turn, the next row's loads in flight, and keep the sums over their rows, and
// the weights, in registers; parts: [vectors][slots of all workgroups][d], added up by norm_columns_kernel in
// slot order.
template <typename X, typename Z, int T, int G, bool VEC, int V>
__global__ __launch_bounds__(T < 256 ? 256 : T, norm_bwd_waves(T, V)) void norm_bwd_kernel(NormView a, float* parts) {
  constexpr int kRows = T < 256 ? 256 / T : 1;
  constexpr bool kKept = G == 1;   // the weights
  // two sums a row, in buffers of their own for rows in turn: between a sum's reads and the
  // next writes to its buffer stands the barrier of the row between
  __shared__ float tmp[2][2][kRows][T / 64];
  const int t = threadIdx.x % T, slot = threadIdx.x / T, d = a.d;
  const float inv_d = 1.0f / static_cast<float>(d);
  const int64_t slots = static_cast<int64_t>(gridDim.x) * kRows;
  const int64_t me = static_cast<int64_t>(blockIdx.x) * kRows + slot;
  const bool branch = norm_bwd_branch(a), need_z = norm_bwd_reads_z(a);
  const bool rows_gate = a.gate_kind == Gate::kRows;
  float sum_pre[G][V], sum_post[G][V], sum_gate[G][V], w_pre[G][V], w_post[G][V], gate[G][V];
#pragma unroll
  for (int g = 0; g < G; ++g) {
#pragma unroll
    for (int k = 0; k < V; ++k) sum_pre[g][k] = sum_post[g][k] = sum_gate[g][k] = 0.0f;
    if (kKept) {
      load_vector<T, VEC, V>(a.w_pre, a.w_bf16, g, t, d, w_pre[g]);
      load_vector<T, VEC, V>(a.post ? a.w_post : nullptr, a.w_bf16, g, t, d, w_post[g]);
      load_vector<T, VEC, V>(rows_gate ? nullptr : a.gate.data, a.w_bf16, g, t, d, gate[g]);
    }
  }
  NormRow<X, Z, T, G, VEC, V> next;
  if (me < a.n_rows) next.load(a, me, t, need_z);
  int odd = 0;
  for (int64_t i = me; i < a.n_rows; i += slots, odd ^= 1) {
    const NormRow<X, Z, T, G, VEC, V> row = next;
    if (i + slots < a.n_rows) next.load(a, i + slots, t, need_z);
    float q[G][V], hat_z[G][V];
    const float inv_z = row.rstd_z;
#pragma unroll
    for (int g = 0; g < G; ++g) {
      if (need_z) {
        row.z[g].get(hat_z[g], g, t, d);
#pragma unroll
        for (int k = 0; k < V; ++k) hat_z[g][k] *= inv_z;
      }
      if (rows_gate) row.gate[g].get(gate[g], g, t, d);
      else if (!kKept) load_vector<T, VEC, V>(a.gate.data, a.w_bf16, g, t, d, gate[g]);
      if (!kKept) load_vector<T, VEC, V>(a.post ? a.w_post : nullptr, a.w_bf16, g, t, d, w_post[g]);
    }
    if (a.pre) {
      const float inv = row.rstd_r;
      float hat[G][V], dt[G][V], dot = 0.0f;
#pragma unroll
      for (int g = 0; g < G; ++g) {
        if (a.r.data) {
          row.r[g].get(hat[g], g, t, d);
        } else {   // as the forward had it before r was rounded
          float x[V];
#pragma unroll
          for (int k = 0; k < V; ++k) x[k] = 0.0f;
          if (a.x.data) row.r[g].get(x, g, t, d);
#pragma unroll
          for (int k = 0; k < V; ++k) hat[g][k] = x[k] + a.scale * gate[g][k] * w_post[g][k] * hat_z[g][k];
        }
        row.dh[g].get(dt[g], g, t, d);
        if (!kKept) load_vector<T, VEC, V>(a.w_pre, a.w_bf16, g, t, d, w_pre[g]);
#pragma unroll
        for (int k = 0; k < V; ++k) {
          hat[g][k] *= inv;
          sum_pre[g][k] += dt[g][k] * hat[g][k];
          dt[g][k] *= w_pre[g][k];
          dot += dt[g][k] * hat[g][k];
        }
      }
      const float mean = row_sum<T>(dot, tmp[odd][0][slot], t) * inv_d;
#pragma unroll
      for (int g = 0; g < G; ++g)
#pragma unroll
        for (int k = 0; k < V; ++k) q[g][k] = inv * (dt[g][k] - hat[g][k] * mean);
    } else {
#pragma unroll
      for (int g = 0; g < G; ++g)
#pragma unroll
        for (int k = 0; k < V; ++k) q[g][k] = 0.0f;
    }
#pragma unroll
    for (int g = 0; g < G; ++g) {
      if (a.dr.data) {
        float v[V];
        row.dr[g].get(v, g, t, d);
#pragma unroll
        for (int k = 0; k < V; ++k) q[g][k] += v[k];
      }
      if (a.dx.data) Part<X, T, VEC, V>::store(row_of<X>(a.dx, i), g, t, d, q[g]);
    }
    if (!branch) continue;
    float dot = 0.0f;
#pragma unroll
    for (int g = 0; g < G; ++g) {
#pragma unroll
      for (int k = 0; k < V; ++k) q[g][k] *= a.scale;
      if (a.gate_kind != Gate::kNone) {
        if (a.dgate.data || a.dgate_sum) {
          float dg[V];
#pragma unroll
          for (int k = 0; k < V; ++k) {
            dg[k] = q[g][k] * hat_z[g][k] * w_post[g][k];
            sum_gate[g][k] += dg[k];
          }
          if (a.dgate.data) Part<Z, T, VEC, V>::store(row_of<Z>(a.dgate, i), g, t, d, dg);
        }
#pragma unroll
        for (int k = 0; k < V; ++k) q[g][k] *= gate[g][k];
      }
      if (a.post) {
#pragma unroll
        for (int k = 0; k < V; ++k) {
          sum_post[g][k] += q[g][k] * hat_z[g][k];
          q[g][k] *= w_post[g][k];
          dot += q[g][k] * hat_z[g][k];
        }
      }
    }
    if (a.post) {
      const float mean = row_sum<T>(dot, tmp[odd][1][slot], t) * inv_d;
#pragma unroll
      for (int g = 0; g < G; ++g)
#pragma unroll
        for (int k = 0; k < V; ++k) q[g][k] = inv_z * (q[g][k] - hat_z[g][k] * mean);
    }
    if (a.dz.data) {
#pragma unroll
      for (int g = 0; g < G; ++g) Part<Z, T, VEC, V>::store(row_of<Z>(a.dz, i), g, t, d, q[g]);
    }
  }
  float* part = parts + me * d;
  const int64_t one = slots * d;
#pragma unroll
  for (int g = 0; g < G; ++g) {
    float* p = part;
    if (a.dw_pre) {
      Part<float, T, VEC, V>::store(p, g, t, d, sum_pre[g]);
      p += one;
    }
    if (a.dw_post) {
      Part<float, T, VEC, V>::store(p, g, t, d, sum_post[g]);
      p += one;
    }
    if (a.dgate_sum) Part<float, T, VEC, V>::store(p, g, t, d, sum_gate[g]);
  }
}

// Sums of the parts, 16 columns a workgroup: 64 of its lanes a column, which add slots k, k + 64, ... and
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

static bool norm_vec(const NormView& v, int32_t r_dtype, int32_t dtype) {
  const int xb = r_dtype == STAPLE_BF16 ? 2 : 4, zb = dtype == STAPLE_BF16 ? 2 : 4;
  const bool gate = v.gate_kind == Gate::kRows ? vec_view(v.gate, zb) : vec_ptr(v.gate.data);
  return v.d % 8 == 0 && vec_view(v.x, xb) && vec_view(v.r, xb) && vec_view(v.dr, xb) && vec_view(v.dx, xb) &&
         vec_view(v.z, zb) && vec_view(v.h, zb) && vec_view(v.dh, zb) && vec_view(v.dz, zb) &&
         vec_view(v.dgate, zb) && gate && vec_ptr(v.w_pre) && vec_ptr(v.w_post);
}

// Lanes a row and groups of eight elements a lane: rows of up to 1024 in a wave, whose sums need no LDS, wider
// ones in four and more.  2048 in 64 x 4: 122 us, in 256 x 1 112 (32768 rows of bf16).
#define NORM_SHAPES(GO)                          \
  do {                                           \
    if (v.d <= 512) GO(64, 1);                   \
    else if (v.d <= 1024) GO(64, 2);             \
    else if (v.d <= 2048) GO(256, 1);            \
    else if (v.d <= 4096) GO(256, 2);            \
    else if (v.d <= 8192) GO(512, 2);            \
    else GO(1024, 2);                            \
  } while (0)

// The backward's, with elements a group: its sums, weights and loads in flight are some 20 registers an
// element, so that four elements a lane in more lanes leave more waves a SIMD: 2048 in 512 x 4 takes 153 us, in
// 256 x 8 233; 4096 in 1024 x 4 198, in 512 x 8 230 (both before rows were read past the caches).
#define NORM_BWD_SHAPES(GO)                      \
  do {                                           \
    if (v.d <= 256) GO(64, 1, 4);                \
    else if (v.d <= 512) GO(64, 1, 8);           \
    else if (v.d <= 1024) GO(256, 1, 4);         \
    else if (v.d <= 2048) GO(512, 1, 4);         \
    else if (v.d <= 4096) GO(1024, 1, 4);        \
    else if (v.d <= 8192) GO(1024, 1, 8);        \
    else GO(1024, 2, 8);                         \
  } while (0)
struct NormBwdShape {
  int lanes, groups, elements;
  int rows() const { return lanes < 256 ? 256 / lanes : 1; }                 // of a workgroup
  int64_t workgroups() const {                                               // that fill the GPU
    const int waves = (lanes < 256 ? 256 : lanes) / 64;
    const int a_cu = norm_bwd_waves(lanes, elements) * 4 / waves;
    return static_cast<int64_t>(device_cus()) * (a_cu > 0 ? a_cu : 1);
  }
};
static NormBwdShape norm_bwd_shape(const NormView& v) {
#define GO(T, G, V) return NormBwdShape{T, G, V}
  NORM_BWD_SHAPES(GO);
#undef GO
}

static int norm_rows_a_workgroup(int d) { return d <= 1024 ? 4 : 1; }

template <typename X, typename Z, bool VEC>
static void norm_fwd(const NormView& v, hipStream_t s) {
  const int rows = norm_rows_a_workgroup(v.d);
  const dim3 grid(static_cast<unsigned>((v.n_rows + rows - 1) / rows));
#define GO(T, G) norm_fwd_kernel<X, Z, T, G, VEC><<<grid, dim3(T < 256 ? 256 : T), 0, s>>>(v)
  NORM_SHAPES(GO);
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

size_t norm_bwd_workspace_bytes(const NormView& v) {
  return static_cast<size_t>(norm_vectors(v)) * norm_bwd_grid(v) * norm_bwd_shape(v).rows() * v.d * sizeof(float);
}

template <typename X, typename Z, bool VEC>
static void norm_bwd(const NormView& v, float* parts, hipStream_t s) {
  const dim3 grid(static_cast<unsigned>(norm_bwd_grid(v)));
  if (v.n_rows > 0) {
#define GO(T, G, V) norm_bwd_kernel<X, Z, T, G, VEC, V><<<grid, dim3(T < 256 ? 256 : T), 0, s>>>(v, parts)
    NORM_BWD_SHAPES(GO);
#undef GO
  }
  const int n = norm_vectors(v);
  if (n == 0) return;
  float* out[3] = {};
  int k = 0;
  for (float* p : {v.dw_pre, v.dw_post, v.dgate_sum})
    if (p) out[k++] = p;
  norm_columns_kernel<<<dim3((v.d + 15) / 16, n), dim3(1024), 0, s>>>(
      parts, static_cast<int>(grid.x) * norm_bwd_shape(v).rows(), v.d, out[0], out[1], out[2]);
}

#define NORM_TYPES(CALL)                                                         \
  const bool vec = norm_vec(v, r_dtype, dtype);                                  \
  if (r_dtype == STAPLE_BF16) {                                                  \
    if (vec) CALL(bf16_t, bf16_t, true); else CALL(bf16_t, bf16_t, false);       \
  } else if (dtype == STAPLE_BF16) {                                             \
    if (vec) CALL(float, bf16_t, true); else CALL(float, bf16_t, false);         \
  } else {                                                                       \
    if (vec) CALL(float, float, true); else CALL(float, float, false);           \
  }

hipError_t launch_norm_fwd(const NormView& v, int32_t r_dtype, int32_t dtype, hipStream_t s) {
#define CALL(X, Z, V) norm_fwd<X, Z, V>(v, s)
  NORM_TYPES(CALL)
#undef CALL
  return hipGetLastError();
}

hipError_t launch_norm_bwd(const NormView& v, int32_t r_dtype, int32_t dtype, void* ws, hipStream_t s) {
  float* parts = static_cast<float*>(ws);
#define CALL(X, Z, V) norm_bwd<X, Z, V>(v, parts, s)
  NORM_TYPES(CALL)
#undef CALL
  return hipGetLastError();
}

}  // namespace staple
