// C ABI of the operators at a model's ends and around its blocks: argument validation and
// dispatch.  Nothing here allocates device memory.
#include <cmath>

#include "api_util.h"
#include "model_ops.h"

namespace staple {

constexpr int64_t kMaxRows = (int64_t(1) << 22) - 1;   // a launch has fewer than 2^32 lanes, and a row up to 1024
constexpr int64_t kMaxTokens29 = int64_t(1) << 29;
constexpr int64_t kMaxWidth = int64_t(1) << 20;

static RowsView view(const staple_rows_t& t) { return RowsView{static_cast<char*>(t.data), t.stride}; }

static bool aligned_to(const void* p, int32_t dtype) {
  return reinterpret_cast<uintptr_t>(p) % elem_bytes(dtype) == 0;
}
// Rows that are read: any stride from 0; rows that are written may not overlap.
static bool in_ok(const void* p, int64_t stride, int32_t dtype) { return p && aligned_to(p, dtype) && stride >= 0; }
static bool out_ok(const void* p, int64_t stride, int64_t n, int64_t width, int32_t dtype) {
  return p && aligned_to(p, dtype) && (stride >= width || n <= 1) && stride >= 0;
}
static bool in_ok(const staple_rows_t& t, int32_t dtype) { return in_ok(t.data, t.stride, dtype); }
static bool out_ok(const staple_rows_t& t, int64_t n, int64_t width, int32_t dtype) {
  return out_ok(t.data, t.stride, n, width, dtype);
}

// What both norm calls ask for.
static staple_status_t norm_check(const staple_norm_t* a) {
  REQUIRE(a);
  if (!valid_dtype(a->dtype) || !valid_dtype(a->r_dtype) || !valid_dtype(a->w_dtype) ||
      (a->r_dtype == STAPLE_BF16 && a->dtype == STAPLE_F32))
    return STAPLE_ERR_UNSUPPORTED;
  REQUIRE(a->n_rows >= 0 && a->d >= 1 && std::isfinite(a->scale) && std::isfinite(a->eps) && a->eps > 0.0f);
  if (a->n_rows > kMaxRows || a->d > kNormMaxDim) return STAPLE_ERR_UNSUPPORTED;
  REQUIRE(a->gate.stride >= 0);
  return STAPLE_OK;
}

static NormView view(const staple_norm_t* a) {
  NormView v{};
  v.n_rows = a->n_rows;
  v.d = static_cast<int>(a->d);
  v.pre = a->pre != 0;
  v.post = a->post != 0;
  v.w_bf16 = a->w_dtype == STAPLE_BF16;
  v.r_bf16 = a->r_dtype == STAPLE_BF16;
  v.gate_kind = !a->gate.data ? Gate::kNone : a->gate.stride == 0 ? Gate::kVector : Gate::kRows;
  v.scale = a->scale;
  v.eps = a->eps;
  v.x = view(a->x);
  v.z = view(a->z);
  v.gate = view(a->gate);
  v.r = view(a->r);
  v.h = view(a->h);
  v.w_pre = a->w_pre;
  v.w_post = a->w_post;
  v.rstd_r = a->rstd_r;
  v.rstd_z = a->rstd_z;
  return v;
}

static NormView bwd_view(const staple_norm_t* a) {
  NormView v = view(a);
  v.dr = view(a->dr);
  v.dh = view(a->dh);
  v.dx = view(a->dx);
  v.dz = view(a->dz);
  if (v.gate_kind == Gate::kRows) v.dgate = view(a->dgate);
  if (v.gate_kind == Gate::kVector) v.dgate_sum = static_cast<float*>(a->dgate.data);
  v.dw_pre = v.pre ? a->dw_pre : nullptr;
  v.dw_post = v.post ? a->dw_post : nullptr;
  return v;
}

// The gate and the weights, each NULL or readable.
static bool shared_ok(const staple_norm_t* a) {
  const bool vector = a->gate.stride == 0;
  return aligned_to(a->gate.data, vector ? a->w_dtype : a->dtype) && aligned_to(a->w_pre, a->w_dtype) &&
         aligned_to(a->w_post, a->w_dtype);
}

static staple_status_t logits_check(int64_t n, int64_t vocab, int32_t dtype, int64_t stride) {
  if (!valid_dtype(dtype)) return STAPLE_ERR_UNSUPPORTED;
  REQUIRE(n >= 0 && vocab >= 1 && stride >= 0);
  if (n > kMaxRows || vocab > kSampleMaxVocab) return STAPLE_ERR_UNSUPPORTED;
  return STAPLE_OK;
}

}  // namespace staple

using namespace staple;

#define CHECKED(expr)                          \
  do {                                         \
    const staple_status_t _st = (expr);        \
    if (_st != STAPLE_OK) return _st;          \
  } while (0)

extern "C" {

// ------------------------------------------------------------------ embedding
staple_status_t staple_embed_fwd(const void* table, int64_t vocab, int64_t d, int32_t dtype,
                                 const int32_t* ids, int64_t n_tokens, float scale, void* y,
                                 int64_t y_stride, int32_t out_dtype, void* stream) {
  if (!valid_dtype(dtype) || !valid_dtype(out_dtype)) return STAPLE_ERR_UNSUPPORTED;
  REQUIRE(n_tokens >= 0 && vocab >= 1 && d >= 1 && std::isfinite(scale));
  if (n_tokens > kMaxTokens29 || d > kMaxWidth || vocab > 0x7fffffffll) return STAPLE_ERR_UNSUPPORTED;
  if (n_tokens == 0) return STAPLE_OK;
  REQUIRE(in_ok(table, d, dtype) && ids && out_ok(y, y_stride, n_tokens, d, out_dtype));
  GET_ERR(err);
  HIPCALL(launch_embed_fwd(table, vocab, d, dtype, ids, n_tokens, scale,
                           RowsView{static_cast<char*>(y), y_stride}, out_dtype, S(stream), err));
  return STAPLE_OK;
}

size_t staple_embed_bwd_workspace_bytes(int64_t n_tokens, int64_t d) {
  return n_tokens >= 0 && n_tokens <= kMaxTokens29 && d >= 1 && d <= kMaxWidth
             ? embed_bwd_workspace_bytes(n_tokens, d) : 0;
}

staple_status_t staple_embed_bwd(const void* dy, int64_t dy_stride, int32_t dtype, int64_t n_tokens,
                                 int64_t d, float scale, const int32_t* sorted_pos,
                                 const int32_t* inv, const int32_t* seg_start,
                                 const int32_t* n_unique, int64_t max_unique, const int32_t* uniq,
                                 float* grad, int64_t grad_rows, int32_t accumulate, void* ws,
                                 size_t ws_bytes, void* stream) {
  if (!valid_dtype(dtype)) return STAPLE_ERR_UNSUPPORTED;
  REQUIRE(n_tokens >= 0 && d >= 1 && std::isfinite(scale) && max_unique >= 0 && grad_rows >= 0);
  REQUIRE(uniq || max_unique <= grad_rows);
  // workgroups of 512 lanes of a launch: one for 512 columns of 64 positions
  if (n_tokens > kMaxTokens29 || d > kMaxWidth || (n_tokens / 64 + 1) * (d / 512 + 1) >= int64_t(1) << 23)
    return STAPLE_ERR_UNSUPPORTED;
  if (n_tokens == 0) return STAPLE_OK;
  REQUIRE(in_ok(dy, dy_stride, dtype) && sorted_pos && inv && seg_start && n_unique);
  REQUIRE(grad && aligned_to(grad, STAPLE_F32));
  const size_t need = embed_bwd_workspace_bytes(n_tokens, d);
  if (ws_bytes < need) return STAPLE_ERR_WORKSPACE;
  REQUIRE(need == 0 || (ws && aligned16(ws)));
  GET_ERR(err);
  const EmbedGrad a{RowsView{static_cast<char*>(const_cast<void*>(dy)), dy_stride}, n_tokens, d, scale,
                    sorted_pos, inv, seg_start, n_unique, max_unique, uniq, grad, grad_rows, accumulate != 0};
  HIPCALL(launch_embed_bwd(a, dtype, ws, S(stream), err));
  return STAPLE_OK;
}

// ---------------------------------------------------------------------- norms
staple_status_t staple_norm_fwd(const staple_norm_t* a, void* stream) {
  CHECKED(norm_check(a));
  if (a->n_rows == 0) return STAPLE_OK;
  REQUIRE(a->x.data || a->z.data);
  REQUIRE(a->z.data || (a->pre && !a->post && !a->gate.data && !a->r.data));
  REQUIRE(!a->x.data || in_ok(a->x, a->r_dtype));
  REQUIRE(!a->z.data || (in_ok(a->z, a->dtype) && out_ok(a->r, a->n_rows, a->d, a->r_dtype)));
  REQUIRE(!a->pre || out_ok(a->h, a->n_rows, a->d, a->dtype));
  REQUIRE(shared_ok(a));
  HIPCALL(launch_norm_fwd(view(a), a->r_dtype, a->dtype, S(stream)));
  return STAPLE_OK;
}

size_t staple_norm_bwd_workspace_bytes(const staple_norm_t* a) {
  return norm_check(a) == STAPLE_OK ? norm_bwd_workspace_bytes(bwd_view(a)) : 0;
}

staple_status_t staple_norm_bwd(const staple_norm_t* a, void* ws, size_t ws_bytes, void* stream) {
  CHECKED(norm_check(a));
  REQUIRE(a->pre || a->dr.data || a->n_rows == 0);
  const NormView v = bwd_view(a);
  const int64_t n = a->n_rows, d = a->d;
  REQUIRE(!v.dr.data || in_ok(a->dr, a->r_dtype));
  if (n > 0) {
    REQUIRE(!v.pre || (a->rstd_r && in_ok(a->dh, a->dtype)));
    REQUIRE(!v.r.data || in_ok(a->r, a->r_dtype));
    REQUIRE(!v.pre || v.r.data || v.z.data);
    REQUIRE(!v.x.data || in_ok(a->x, a->r_dtype));
    const bool reads_z = norm_bwd_reads_z(v);
    REQUIRE(!reads_z || in_ok(a->z, a->dtype));
    REQUIRE(!reads_z || !v.post || a->rstd_z);
  }
  REQUIRE(!v.dx.data || out_ok(a->dx, n, d, a->r_dtype));
  REQUIRE(!v.dz.data || out_ok(a->dz, n, d, a->dtype));
  REQUIRE(!v.dgate.data || out_ok(a->dgate, n, d, a->dtype));
  REQUIRE(aligned_to(v.dgate_sum, STAPLE_F32) && aligned_to(v.dw_pre, STAPLE_F32) &&
          aligned_to(v.dw_post, STAPLE_F32) && shared_ok(a));
  const size_t need = norm_bwd_workspace_bytes(v);
  if (ws_bytes < need) return STAPLE_ERR_WORKSPACE;
  REQUIRE(need == 0 || (ws && aligned16(ws)));
  HIPCALL(launch_norm_bwd(v, a->r_dtype, a->dtype, ws, S(stream)));
  return STAPLE_OK;
}

// ----------------------------------------------------------------------- loss
staple_status_t staple_xent_fwd(const void* logits, int64_t stride, int64_t n_rows, int64_t vocab,
                                int32_t dtype, const int32_t* targets, float* loss, float* lse,
                                const float* g, void* d_logits, int64_t d_stride, void* stream) {
  CHECKED(logits_check(n_rows, vocab, dtype, stride));
  REQUIRE((g == nullptr) == (d_logits == nullptr));
  if (n_rows == 0) return STAPLE_OK;
  REQUIRE(in_ok(logits, stride, dtype) && targets && loss && lse);
  REQUIRE(!d_logits || out_ok(d_logits, d_stride, n_rows, vocab, dtype));
  GET_ERR(err);
  const XentView v{static_cast<const char*>(logits), stride, n_rows, static_cast<int>(vocab), targets,
                   loss, lse, g, static_cast<char*>(d_logits), d_stride};
  HIPCALL(launch_xent_fwd(v, dtype, S(stream), err));
  return STAPLE_OK;
}

staple_status_t staple_xent_bwd(const void* logits, int64_t stride, int64_t n_rows, int64_t vocab,
                                int32_t dtype, const int32_t* targets, const float* lse,
                                const float* g, void* d_logits, int64_t d_stride, void* stream) {
  CHECKED(logits_check(n_rows, vocab, dtype, stride));
  if (n_rows == 0) return STAPLE_OK;
  REQUIRE(in_ok(logits, stride, dtype) && targets && lse && g);
  REQUIRE(out_ok(d_logits, d_stride, n_rows, vocab, dtype));
  GET_ERR(err);
  const XentView v{static_cast<const char*>(logits), stride, n_rows, static_cast<int>(vocab), targets,
                   nullptr, const_cast<float*>(lse), g, static_cast<char*>(d_logits), d_stride};
  HIPCALL(launch_xent_bwd(v, dtype, S(stream), err));
  return STAPLE_OK;
}

// ------------------------------------------------------------------- sampling
size_t staple_sample_workspace_bytes(int64_t n_rows, int64_t vocab) {
  return n_rows >= 1 && n_rows <= kMaxRows && vocab >= 1 && vocab <= kSampleMaxVocab
             ? sample_workspace_bytes(n_rows, vocab) : 0;
}

staple_status_t staple_sample(const void* logits, int64_t stride, int64_t n_rows, int64_t vocab,
                              int32_t dtype, const float* u, const float* temperature,
                              const int32_t* top_k, const float* top_p, const float* min_p,
                              int32_t* token, float* logprob, void* ws, size_t ws_bytes,
                              void* stream) {
  CHECKED(logits_check(n_rows, vocab, dtype, stride));
  if (n_rows == 0) return STAPLE_OK;
  REQUIRE(in_ok(logits, stride, dtype) && u && token);
  const size_t need = sample_workspace_bytes(n_rows, vocab);
  if (ws_bytes < need) return STAPLE_ERR_WORKSPACE;
  REQUIRE(need == 0 || (ws && aligned16(ws)));
  const SampleView v{static_cast<const char*>(logits), stride, n_rows, static_cast<int>(vocab), u,
                     temperature, top_p, min_p, top_k, token, logprob};
  HIPCALL(launch_sample(v, dtype, ws, S(stream)));
  return STAPLE_OK;
}

}  // extern "C"
