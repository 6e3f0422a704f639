// Launchers of the operators at a model's ends and around its blocks (embed.hip, norm.hip,
// xent.hip, sample.hip).  Arguments have been checked by the entry points.
#pragma once

#include "common.h"

namespace staple {

struct RowsView {
  char* data;
  int64_t stride;   // elements
};

hipError_t launch_embed_fwd(const void* table, int64_t vocab, int64_t d, int32_t dtype,
                            const int32_t* ids, int64_t n, float scale, RowsView y,
                            int32_t out_dtype, hipStream_t s, int* err);

struct EmbedGrad {
  RowsView dy;
  int64_t n_tokens, d;
  float scale;
  const int32_t *sorted_pos, *inv, *seg_start, *n_unique;
  int64_t max_unique;
  const int32_t* uniq;   // grad's row of unique token u: uniq[u], or u when NULL
  float* grad;
  int64_t grad_rows;
  bool accumulate;
};
size_t embed_bwd_workspace_bytes(int64_t n_tokens, int64_t d);
hipError_t launch_embed_bwd(const EmbedGrad& a, int32_t dtype, void* ws, hipStream_t s, int* err);

enum class Gate { kNone, kVector, kRows };

struct NormView {
  int64_t n_rows;
  int d;
  bool pre, post, w_bf16, r_bf16;
  Gate gate_kind;
  float scale, eps;
  RowsView x, z, gate, r, h;
  const void *w_pre, *w_post;
  float *rstd_r, *rstd_z;
  RowsView dr, dh, dx, dz, dgate;
  float *dw_pre, *dw_post, *dgate_sum;
};
constexpr int kNormMaxDim = 16384;
// The backward needs z for its own gradient through the norm, for the gate's, and where it forms r again.
__host__ __device__ inline bool norm_bwd_branch(const NormView& v) {
  return v.dz.data || v.dgate.data || v.dgate_sum || v.dw_post;
}
__host__ __device__ inline bool norm_bwd_reads_z(const NormView& v) {
  return (norm_bwd_branch(v) && v.post) || v.dgate.data || v.dgate_sum || (v.pre && !v.r.data);
}
hipError_t launch_norm_fwd(const NormView& v, int32_t r_dtype, int32_t dtype, hipStream_t s);
size_t norm_bwd_workspace_bytes(const NormView& v);
hipError_t launch_norm_bwd(const NormView& v, int32_t r_dtype, int32_t dtype, void* ws, hipStream_t s);

struct XentView {
  const char* logits;
  int64_t stride, n_rows;
  int vocab;
  const int32_t* targets;
  float *loss, *lse;
  const float* g;
  char* d_logits;
  int64_t d_stride;
};
hipError_t launch_xent_fwd(const XentView& v, int32_t dtype, hipStream_t s, int* err);
hipError_t launch_xent_bwd(const XentView& v, int32_t dtype, hipStream_t s, int* err);

struct SampleView {
  const char* logits;
  int64_t stride, n_rows;
  int vocab;
  const float *u, *temperature, *top_p, *min_p;
  const int32_t* top_k;
  int32_t* token;
  float* logprob;
};
constexpr int64_t kSampleMaxVocab = int64_t(1) << 22;
size_t sample_workspace_bytes(int64_t n_rows, int64_t vocab);
hipError_t launch_sample(const SampleView& v, int32_t dtype, void* ws, hipStream_t s);

}  // namespace staple
