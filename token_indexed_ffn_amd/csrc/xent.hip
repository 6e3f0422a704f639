// Cross entropy of a vocabulary's logits, and its gradient.
//
//   lse = log sum_j exp l_j,   loss = lse - l_t,   dl_j = g (exp(l_j - lse) - [j = t])
//
// A workgroup holds its row in registers, as it lies in memory: one read, the maximum, the sum, and
// with the gradient one write.  What they do not hold of a wide row is read once more for the gradient, its
// sum running with its maximum: (m, s) stands for s exp m, and two such pairs join into one.  Bound by
// bytes: 8192 x 100352 in bf16 with the gradient take 667 us, 4.9 TB/s.
#include "model_ops.h"
#include "row_io.h"

namespace staple {

// What exponents are taken relative to: the maximum, or 0 where it is infinite (a row of
// -inf has the sum 0, one with +inf the sum +inf).
__device__ __forceinline__ float reference(float m) { return __builtin_isinf(m) ? 0.0f : m; }

// Sums and maxima over the T lanes of a row, in a fixed order; every lane gets them.  tmp: T / 64
// floats that no wave still reads.
template <int T>
__device__ __forceinline__ float row_max(float v, float* tmp, int t) {
  v = wave_max(v);
  if (T == 64) return v;
  if ((t & 63) == 0) tmp[t >> 6] = v;
  __syncthreads();
  v = tmp[0];
#pragma unroll
  for (int i = 1; i < T / 64; ++i) v = fmaxf(v, tmp[i]);
  return v;
}

struct MaxSum {
  float m = -__builtin_inff(), s = 0.0f;
  __device__ __forceinline__ void join(float m2, float s2) {
    const float top = fmaxf(m, m2), ref = reference(top);
    const float a = s == 0.0f ? 0.0f : s * __expf(reference(m) - ref);
    const float b = s2 == 0.0f ? 0.0f : s2 * __expf(reference(m2) - ref);
    m = top;
    s = a + b;
  }
  __device__ __forceinline__ void add(const float (&v)[8]) {
    float top = m;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = fmaxf(top, v[i]);
    const float ref = reference(top);
    if (top != m) {
      if (s != 0.0f) s *= __expf(reference(m) - ref);
      m = top;
    }
    float a = 0.0f, b = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      a += __expf(v[i] - ref);
      b += __expf(v[i + 1] - ref);
    }
    s += a + b;
  }
};

// The target of a row: -1 where the row does not count.
__device__ __forceinline__ int target_of(const XentView& a, int64_t i, int t, int* err) {
  const int target = a.targets[i];
  if (target < 0) return -1;
  if (target < a.vocab) return target;
  if (t == 0) flag_index_error(err);
  return -1;
}

__device__ __forceinline__ void store_loss(const XentView& a, int64_t i, int target, float at, float m, float s) {
  const float lse = logf(s) + reference(m);
  a.lse[i] = lse;
  a.loss[i] = target < 0 ? 0.0f : at == -__builtin_inff() && lse == lse ? __builtin_inff() : lse - at;
}

// A row's gradient: p = exp(l - ref) f, without the target's 1.
struct Gradient {
  float ref, f, g;
  int target;   // -1: all zero
  // f: 1 / s, with the reference of the sum; for a sum of +inf p is exp(l - inf)
  __device__ __forceinline__ Gradient(const XentView& a, int64_t i, int t, float m, float s) {
    g = a.g[i];
    const bool top = m == __builtin_inff();
    ref = top ? m : reference(m);
    f = top ? 1.0f : 1.0f / s;
    target = s == 0.0f ? -1 : t;
  }
  __device__ __forceinline__ Gradient(float lse, float gi, int t) : ref(lse), f(1.0f), g(gi) {
    target = lse == -__builtin_inff() ? -1 : t;
  }
  __device__ __forceinline__ float one(float l, int j) const {
    if (target < 0) return 0.0f;
    return g * (__expf(l - ref) * f - (j == target ? 1.0f : 0.0f));
  }
  // Eight from element j on, in place.
  __device__ __forceinline__ void eight(float (&v)[8], int j) const {
    if (target < 0) {
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = 0.0f;
      return;
    }
    const float gf = g * f;
    const unsigned at = static_cast<unsigned>(target - j);
    if (at < 8u) {
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = g * (__expf(v[k] - ref) * f - (k == static_cast<int>(at) ? 1.0f : 0.0f));
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = __expf(v[k] - ref) * gf;
    }
  }
};

// Eight gradients from element j on: at once where the output is aligned as the logits are.
template <typename E>
__device__ __forceinline__ void store_eight(E* out, int j, bool aligned, const float (&v)[8]) {
  if (aligned) {
    store8(out + j, v);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) store1(out + j + k, v[k]);
  }
}

template <typename E, int T, int G>
__global__ __launch_bounds__(T < 256 ? 256 : T) void xent_fwd_kernel(XentView a, int* err) {
  constexpr int kRows = T < 256 ? 256 / T : 1;
  __shared__ float tmp[2][kRows][T / 64];
  const int t = threadIdx.x % T, slot = threadIdx.x / T;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kRows + slot;
  if (i >= a.n_rows) return;   // T >= 256: the whole workgroup; T = 64: a wave, which meets no barrier
  const E* l = reinterpret_cast<const E*>(a.logits) + i * a.stride;
  const RowGroups r(l, a.vocab);
  Raw<E> raw[G];
#pragma unroll
  for (int q = 0; q < G; ++q) {
    const int j = (q * T + t) * 8 - r.shift;
    if (r.full(j)) raw[q].load(l + j);
    else raw[q].clear();
  }
  const int edge = t < 64 ? r.edge(t) : -1;
  const float at_edge = edge >= 0 ? load1(l + edge) : -__builtin_inff();
  const int target = target_of(a, i, t, err);
  const float at = target >= 0 ? load1(l + target) : 0.0f;   // before the gradient, which may be in place
  float m = at_edge;
#pragma unroll
  for (int q = 0; q < G; ++q) {
    float v[8];
    raw[q].get(v);
#pragma unroll
    for (int k = 0; k < 8; ++k) m = fmaxf(m, v[k]);
  }
  m = row_max<T>(m, tmp[0][slot], t);
  const float ref = reference(m);
  float s[4] = {__expf(at_edge - ref), 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int q = 0; q < G; ++q) {
    float v[8];
    raw[q].forget();
    raw[q].get(v);
#pragma unroll
    for (int k = 0; k < 8; ++k) s[k & 3] += __expf(v[k] - ref);
  }
  const float sum = row_sum<T>((s[0] + s[1]) + (s[2] + s[3]), tmp[1][slot], t);
  if (t == 0) store_loss(a, i, target, at, m, sum);
  if (!a.d_logits) return;
  E* out = reinterpret_cast<E*>(a.d_logits) + i * a.d_stride;
  const bool aligned = RowGroups(out, a.vocab).shift == r.shift;
  const Gradient grad(a, i, target, m, sum);
#pragma unroll
  for (int q = 0; q < G; ++q) {
    const int j = (q * T + t) * 8 - r.shift;
    float v[8];
    raw[q].forget();
    raw[q].get(v);
    grad.eight(v, j);
    if (r.full(j)) store_eight(out, j, aligned, v);
  }
  if (edge >= 0) store1(out + edge, grad.one(at_edge, edge));
}

// Rows of any width.  G groups a lane stay in registers for the gradient; the rest of the row is read once more,
// from its end on, where the caches still have it.
template <typename E, int T, int G>
__global__ __launch_bounds__(T) void xent_fwd_long_kernel(XentView a, int* err) {
  __shared__ float2 tmp[T / 64];
  constexpr int kAhead = G > 0 ? 2 : 4;   // with more the kept groups spill
  const int t = threadIdx.x;
  const int64_t i = blockIdx.x;
  const E* l = reinterpret_cast<const E*>(a.logits) + i * a.stride;
  const RowGroups r(l, a.vocab);
  const int steps = (a.vocab + r.shift + T * 8 - 1) / (T * 8);   // a lane's groups
  Raw<E> kept[G > 0 ? G : 1];
#pragma unroll
  for (int q = 0; q < G; ++q) {
    const int j = (q * T + t) * 8 - r.shift;
    if (r.full(j)) kept[q].load(l + j);
    else kept[q].clear();
  }
  const int edge = t < 64 ? r.edge(t) : -1;
  const float at_edge = edge >= 0 ? load1(l + edge) : -__builtin_inff();
  const int target = target_of(a, i, t, err);
  const float at = target >= 0 ? load1(l + target) : 0.0f;
  MaxSum x{at_edge, at_edge == -__builtin_inff() ? 0.0f : __expf(at_edge - reference(at_edge))};
#pragma unroll
  for (int q = 0; q < G; ++q) {
    float v[8];
    kept[q].get(v);
    x.add(v);
  }
  for (int q = G; q < steps; q += kAhead) {
    Raw<E> raw[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int j = ((q + u) * T + t) * 8 - r.shift;
      if (r.full(j)) raw[u].load(l + j);
      else raw[u].clear();
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      float v[8];
      raw[u].get(v);
      x.add(v);
    }
  }
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) x.join(__shfl_xor(x.m, o, 64), __shfl_xor(x.s, o, 64));
  if ((t & 63) == 0) tmp[t >> 6] = make_float2(x.m, x.s);
  __syncthreads();
  x = MaxSum{tmp[0].x, tmp[0].y};
#pragma unroll
  for (int k = 1; k < T / 64; ++k) x.join(tmp[k].x, tmp[k].y);
  if (t == 0) store_loss(a, i, target, at, x.m, x.s);
  if (!a.d_logits) return;
  E* out = reinterpret_cast<E*>(a.d_logits) + i * a.d_stride;
  const bool aligned = RowGroups(out, a.vocab).shift == r.shift;
  const Gradient grad(a, i, target, x.m, x.s);
  for (int q = steps - 1; q >= G; q -= kAhead) {
    Raw<E> raw[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int j = ((q - u) * T + t) * 8 - r.shift;
      if (q - u >= G && r.full(j)) raw[u].load(l + j);
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int j = ((q - u) * T + t) * 8 - r.shift;
      if (q - u < G || !r.full(j)) continue;
      float v[8];
      raw[u].get(v);
      grad.eight(v, j);
      store_eight(out, j, aligned, v);
    }
  }
#pragma unroll
  for (int q = 0; q < G; ++q) {
    const int j = (q * T + t) * 8 - r.shift;
    float v[8];
    kept[q].forget();
    kept[q].get(v);
    grad.eight(v, j);
    if (r.full(j)) store_eight(out, j, aligned, v);
  }
  if (edge >= 0) store1(out + edge, grad.one(at_edge, edge));
}

// The gradient alone: a workgroup takes kBwdGroups times 2048 elements of a row.  4096 rows of 100352: bf16 304 us
// (5.4 TB/s), fp32 589 (5.6); of 100277: 308, 607.
constexpr int kBwdGroups = 4;
template <typename E>
__global__ __launch_bounds__(256) void xent_bwd_kernel(XentView a, int pieces, int* err) {
  const int64_t i = blockIdx.x / pieces;
  const int piece = static_cast<int>(blockIdx.x - i * pieces), t = threadIdx.x;
  const E* l = reinterpret_cast<const E*>(a.logits) + i * a.stride;
  E* out = reinterpret_cast<E*>(a.d_logits) + i * a.d_stride;
  const RowGroups r(l, a.vocab);
  const bool aligned = RowGroups(out, a.vocab).shift == r.shift;
  Raw<E> raw[kBwdGroups];
  const int j0 = (piece * kBwdGroups * 256 + t) * 8 - r.shift;
#pragma unroll
  for (int q = 0; q < kBwdGroups; ++q)
    if (r.full(j0 + q * 2048)) raw[q].load(l + j0 + q * 2048);
  const int edge = piece == 0 && t < 64 ? r.edge(t) : -1;
  const float at_edge = edge >= 0 ? load1(l + edge) : 0.0f;
  const Gradient grad(a.lse[i], a.g[i], target_of(a, i, piece == 0 ? t : 1, err));
#pragma unroll
  for (int q = 0; q < kBwdGroups; ++q) {
    const int j = j0 + q * 2048;
    if (!r.full(j)) continue;
    float v[8];
    raw[q].get(v);
    grad.eight(v, j);
    store_eight(out, j, aligned, v);
  }
  if (edge >= 0) store1(out + edge, grad.one(at_edge, edge));
}

// The narrowest shape that holds a row: lanes and groups of eight a lane (rows that begin between
// 16-byte addresses need up to one group more).  Wider rows in the long kernel, which keeps 32 registers of a bf16 row
// and 64 of a wide one, 64 of an fp32 one: its read of the rest overlaps, where a workgroup with the whole row
// in registers is alone on its CU and first reads, then writes.  us for 4096 bf16 rows with the gradient, nothing
// kept, 32, 64 registers: 70000 classes: -, 286, 326 (all of it in 512 lanes); 100352: 393, 362, 363; 128256: 488, 448, 421;
// 151936: 587, 535, 512; 260001: 1267, -, 950.  fp32, nothing and 64: 100352: 703 (all of it), 662; 128256: 973,
// 838; 256000: 2255, 1916.  The loss alone is only read and keeps nothing: 4096 bf16 rows of 100352 take 178 to 204 us
// (4.0 to 4.6 TB/s), fp32 271 (6.1).
template <typename E>
static void xent_fwd(const XentView& v, hipStream_t s, int* err) {
  const bool aligned = reinterpret_cast<uintptr_t>(v.logits) % 16 == 0 && v.stride * sizeof(E) % 16 == 0;
  const int64_t w = v.vocab + (aligned ? 0 : 7);
#define GO(T, G)                                                                                       \
  if (w <= int64_t(T) * 8 * G) {                                                                       \
    constexpr int kRows = T < 256 ? 256 / T : 1;                                                       \
    xent_fwd_kernel<E, T, G><<<dim3(static_cast<unsigned>((v.n_rows + kRows - 1) / kRows)),            \
                               dim3(T < 256 ? 256 : T), 0, s>>>(v, err);                               \
    return;                                                                                            \
  }
  GO(64, 1)
  GO(64, 2)
  GO(256, 1)
  GO(256, 2)
  GO(256, 4)
  GO(256, 8)
  GO(512, 8)
  GO(512, 16)
#undef GO
  const dim3 grid(static_cast<unsigned>(v.n_rows)), threads(1024);
  if (!v.d_logits) xent_fwd_long_kernel<E, 1024, 0><<<grid, threads, 0, s>>>(v, err);
  else if (sizeof(E) == 4 || w <= 114688) xent_fwd_long_kernel<E, 1024, 8><<<grid, threads, 0, s>>>(v, err);
  else if constexpr (sizeof(E) == 2) xent_fwd_long_kernel<E, 1024, 16><<<grid, threads, 0, s>>>(v, err);
}

hipError_t launch_xent_fwd(const XentView& v, int32_t dtype, hipStream_t s, int* err) {
  if (dtype == STAPLE_BF16) xent_fwd<bf16_t>(v, s, err);
  else xent_fwd<float>(v, s, err);
  return hipGetLastError();
}

hipError_t launch_xent_bwd(const XentView& v, int32_t dtype, hipStream_t s, int* err) {
  const int pieces = (v.vocab + 7 + kBwdGroups * 2048 - 1) / (kBwdGroups * 2048);
  const int64_t at_once = (int64_t(1) << 23) / pieces;   // workgroups of a launch
  for (int64_t i = 0; i < v.n_rows; i += at_once) {
    XentView a = v;
    a.n_rows = v.n_rows - i < at_once ? v.n_rows - i : at_once;
    const int64_t size = dtype == STAPLE_BF16 ? 2 : 4;
    a.logits += i * a.stride * size;
    a.d_logits += i * a.d_stride * size;
    a.targets += i;
    a.lse += i;
    a.g += i;
    const dim3 grid(static_cast<unsigned>(a.n_rows * pieces));
    if (dtype == STAPLE_BF16) xent_bwd_kernel<bf16_t><<<grid, dim3(256), 0, s>>>(a, pieces, err);
    else xent_bwd_kernel<float><<<grid, dim3(256), 0, s>>>(a, pieces, err);
  }
  return hipGetLastError();
}

}  // namespace staple
