// Attention over packed sequences with a causal mask, a sliding window and
// sinks: forward and backward.
#include "attn_row.h"

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

template <typename T>
__global__ __launch_bounds__(64 * kRowWaves) void attn_fwd_row_kernel(AttnView a, int* err) {
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
  const Row2 q = load_row<T>(a.q, t, h, a.head_dim);
  RowSoftmax sm;
  for (int64_t j = 0; j <= p; ++j) {
    if (j == sink_end) j = lo;
    if (j > p) break;
    const Row2 k = load_row<T>(a.k, k0 + j, hk, a.head_dim);
    sm.add(dot(q, k) * a.scale, load_row<T>(a.v, k0 + j, hk, a.head_dim));
  }
  store_row<T>(a.o, t, h, a.head_dim, sm.value());
  if ((threadIdx.x & 63) == 0) a.lse[t * a.n_heads + h] = sm.lse();
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
  const unsigned wgs = row_wgs(a.total_q * a.n_heads);
  if (wgs == 0) return hipSuccess;
  if (dtype == STAPLE_BF16) attn_fwd_row_kernel<bf16_t><<<wgs, 64 * kRowWaves, 0, s>>>(a, err);
  else attn_fwd_row_kernel<float><<<wgs, 64 * kRowWaves, 0, s>>>(a, err);
  return hipGetLastError();
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
