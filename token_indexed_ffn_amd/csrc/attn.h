// Device views of the attention operands and the launchers of attn.hip and
// attn_decode.hip.
#pragma once

#include "kv.h"

namespace staple {

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;

// Positions and row numbers stay below this, so that 32-bit sums of a
// few of them cannot overflow.
constexpr int kMaxTokens = 1 << 29;

struct AttnView {
  int64_t n_seqs, total_q, total_k;
  int n_heads, n_kv_heads, group, head_dim;
  int window, sinks;       // window 0: every key up to the query's position
  float scale;
  const int32_t* cu_q;
  const int32_t* cu_k;
  HeadsView q, k, v, o, d_o, dq, dk, dv;
  float* lse;
};

size_t attn_bwd_workspace_bytes(const AttnView& a, int dtype);
size_t attn_fwd_workspace_bytes(const AttnView& a, int dtype);
hipError_t launch_attn_fwd(const AttnView& a, int dtype, void* ws, hipStream_t s, int* err);
hipError_t launch_attn_bwd(const AttnView& a, int dtype, void* ws, hipStream_t s, int* err);

struct DecodeView {
  int64_t n_seqs, max_len, window, sinks;
  int n_heads, group, head_dim;
  float scale;
  const int32_t* seqs;
  HeadsView q, k_new, v_new, o;
  float* lse;
};

size_t attn_decode_workspace_bytes(const KvView& kv, const DecodeView& a, int dtype);
hipError_t launch_attn_decode(const KvView& kv, const DecodeView& a, int dtype, void* ws,
                              hipStream_t s, int* err);

// Rows [begin, end) of sequence b (empty and the error word where the offsets
// are out of order or past `total`).
__device__ __forceinline__ void seq_rows(const int32_t* cu, int64_t b, int64_t total, int64_t* begin,
                                         int64_t* end, int* err) {
  const int64_t x = cu[b], y = cu[b + 1];
  const bool fine = x >= 0 && y >= x && y <= total;
  if (!fine) flag_index_error(err);
  *begin = fine ? x : 0;
  *end = fine ? y : 0;
}

// Flags every pair of offsets that seq_rows() refuses, also of sequences that
// no row leads to: called by all of a grid's threads.
__device__ __forceinline__ void check_offsets(const AttnView& a, int* err) {
  const int64_t step = static_cast<int64_t>(gridDim.x) * blockDim.x;
  for (int64_t b = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; b < a.n_seqs; b += step) {
    int64_t x, y;
    seq_rows(a.cu_q, b, a.total_q, &x, &y, err);
    seq_rows(a.cu_k, b, a.total_k, &x, &y, err);
  }
}

// The keys that a query at position p sees are [0, sink_end) and [lo, p]:
// sink_end <= lo, and both are empty for p < 0.
__device__ __forceinline__ void visible_keys(int64_t p, int64_t window, int64_t sinks,
                                             int64_t* sink_end, int64_t* lo) {
  const int64_t first = window > 0 ? p - window + 1 : 0;
  *lo = first > 0 ? first : 0;
  *sink_end = sinks < *lo ? sinks : *lo;
}

}  // namespace staple
