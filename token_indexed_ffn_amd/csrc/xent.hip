// Cross entropy of a vocabulary's logits, and its gradient.
//
//   lse = log sum_j exp l_j,   loss = lse - l_t,   dl_j = g (exp(l_j - lse) - [j = t])
//
// A row's sum runs with its maximum: (m, s) stands for s exp m, and two such pairs join into one.
#include "model_ops.h"
#include "row_io.h"

namespace staple {

// What exponents are taken relative to: the maximum, or 0 where it is infinite (a row of
// -inf has the sum 0, one with +inf the sum +inf).
__device__ __forceinline__ float reference(float m) { return __builtin_isinf(m) ? 0.0f : m; }

struct MaxSum {
  float m = -__builtin_inff(), s = 0.0f;
  __device__ __forceinline__ void join(float m2, float s2) {
    const float top = fmaxf(m, m2), ref = reference(top);
    const float a = s == 0.0f ? 0.0f : s * __expf(reference(m) - ref);
    const float b = s2 == 0.0f ? 0.0f : s2 * __expf(reference(m2) - ref);
    m = top;
    s = a + b;
  }
  template <int N>
  __device__ __forceinline__ void add(const float (&v)[N]) {
    float top = m;
#pragma unroll
    for (int i = 0; i < N; ++i) top = fmaxf(top, v[i]);
    const float ref = reference(top);
    if (top != m) {
      if (s != 0.0f) s *= __expf(reference(m) - ref);
      m = top;
    }
#pragma unroll
    for (int i = 0; i < N; ++i) s += __expf(v[i] - ref);
  }
};

// Joined over a workgroup of T lanes, in a fixed order; every lane gets the result.
template <int T>
__device__ __forceinline__ void join_all(MaxSum& x, float2* tmp) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) x.join(__shfl_xor(x.m, o, 64), __shfl_xor(x.s, o, 64));
  if (T == 64) return;
  if ((threadIdx.x & 63) == 0) tmp[threadIdx.x >> 6] = make_float2(x.m, x.s);
  __syncthreads();
  x = MaxSum{tmp[0].x, tmp[0].y};
#pragma unroll
  for (int i = 1; i < T / 64; ++i) x.join(tmp[i].x, tmp[i].y);
}

__device__ __forceinline__ float log_sum(const MaxSum& x) { return logf(x.s) + reference(x.m); }

// The target of a row: -1 where the row does not count.
__device__ __forceinline__ int target_of(const XentView& a, int64_t i, int* err) {
  const int t = a.targets[i];
  if (t < 0) return -1;
  if (t < a.vocab) return t;
  if (threadIdx.x == 0) flag_index_error(err);
  return -1;
}

// g (exp(l - ref) f - [j = t]) for one row; f = 0 where no class is possible.
template <typename E, int T>
__device__ __forceinline__ void gradient_row(const XentView& a, int64_t i, int target, float ref, float f) {
  const E* l = reinterpret_cast<const E*>(a.logits) + i * a.stride;
  E* out = reinterpret_cast<E*>(a.d_logits) + i * a.d_stride;
  const float g = a.g[i];
  if (target < 0 || f == 0.0f) {
    for (int j = threadIdx.x; j < a.vocab; j += T) store1(out + j, 0.0f);
    return;
  }
  for (int j = threadIdx.x; j < a.vocab; j += T)
    store1(out + j, g * (__expf(load1(l + j) - ref) * f - (j == target ? 1.0f : 0.0f)));
}

template <typename E, int T>
__global__ __launch_bounds__(T) void xent_fwd_kernel(XentView a, int* err) {
  __shared__ float2 tmp[T / 64];
  const int64_t i = blockIdx.x;
  const E* l = reinterpret_cast<const E*>(a.logits) + i * a.stride;
  const int target = target_of(a, i, err);
  MaxSum x;
  for (int j = threadIdx.x; j < a.vocab; j += T) {
    const float v[1] = {load1(l + j)};
    x.add(v);
  }
  const float at = target >= 0 ? load1(l + target) : 0.0f;   // before the gradient, which may be in place
  join_all<T>(x, tmp);
  if (threadIdx.x == 0) {
    const float lse = log_sum(x);
    a.lse[i] = lse;
    a.loss[i] = target < 0 ? 0.0f : at == -__builtin_inff() && lse == lse ? __builtin_inff() : lse - at;
  }
  if (a.d_logits) {
    __syncthreads();   // every lane has read the target's logit
    gradient_row<E, T>(a, i, target, reference(x.m), x.s == 0.0f ? 0.0f : 1.0f / x.s);
  }
}

template <typename E, int T>
__global__ __launch_bounds__(T) void xent_bwd_kernel(XentView a, int* err) {
  const int64_t i = blockIdx.x;
  const float lse = a.lse[i];
  gradient_row<E, T>(a, i, target_of(a, i, err), lse, lse == -__builtin_inff() ? 0.0f : 1.0f);
}

size_t xent_workspace_bytes(int64_t, int64_t) { return 0; }

hipError_t launch_xent_fwd(const XentView& v, int32_t dtype, void*, hipStream_t s, int* err) {
  const dim3 grid(static_cast<unsigned>(v.n_rows));
  if (dtype == STAPLE_BF16) xent_fwd_kernel<bf16_t, 512><<<grid, dim3(512), 0, s>>>(v, err);
  else xent_fwd_kernel<float, 512><<<grid, dim3(512), 0, s>>>(v, err);
  return hipGetLastError();
}

hipError_t launch_xent_bwd(const XentView& v, int32_t dtype, hipStream_t s, int* err) {
  const dim3 grid(static_cast<unsigned>(v.n_rows));
  if (dtype == STAPLE_BF16) xent_bwd_kernel<bf16_t, 512><<<grid, dim3(512), 0, s>>>(v, err);
  else xent_bwd_kernel<float, 512><<<grid, dim3(512), 0, s>>>(v, err);
  return hipGetLastError();
}

}  // namespace staple
