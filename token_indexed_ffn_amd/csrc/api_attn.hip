// C ABI of the attention operators and the paged key-value cache: argument
// validation and dispatch.  Nothing here allocates device memory.
#include <cmath>

#include "api_util.h"
#include "attn.h"
#include "kv.h"

namespace staple {

constexpr int64_t kMaxCount = 0x7fffffffll;
// Rows of one launch: workgroups times threads stay below 2^32.
constexpr int64_t kMaxLaunchRows = int64_t(1) << 23;
constexpr int64_t kMaxPageBytes = int64_t(1) << 31;

static bool dims_ok(int64_t head_dim) { return head_dim >= 8 && head_dim <= 128 && head_dim % 8 == 0; }

// 16-byte aligned data and strides (read or written 16 bytes a lane).
static bool heads_ok(const staple_heads_t& t, int32_t dtype) {
  const int64_t vec = 16 / elem_bytes(dtype);
  return t.data && aligned16(t.data) && t.row_stride >= 0 && t.head_stride >= 0 &&
         t.row_stride % vec == 0 && t.head_stride % vec == 0;
}
static HeadsView view(const staple_heads_t& t) {
  return HeadsView{static_cast<char*>(t.data), t.row_stride, t.head_stride};
}

static staple_status_t attn_check(const staple_attn_t* a) {
  REQUIRE(a);
  if (!valid_dtype(a->dtype) || !dims_ok(a->head_dim)) return STAPLE_ERR_UNSUPPORTED;
  REQUIRE(a->n_seqs >= 0 && a->total_q >= 0 && a->total_k >= 0);
  REQUIRE(a->n_heads >= 1 && a->n_kv_heads >= 1 && a->n_heads % a->n_kv_heads == 0);
  REQUIRE(a->window >= 0 && a->sinks >= 0 && std::isfinite(a->scale));
  if (a->n_seqs > kMaxTokens || a->total_q > kMaxTokens || a->total_k > kMaxTokens ||
      a->n_heads > 65535 || a->total_q * a->n_heads > kMaxLaunchRows * 64 ||
      a->total_k * a->n_kv_heads > kMaxLaunchRows * 64)
    return STAPLE_ERR_UNSUPPORTED;
  // workgroups of a launch: a tile of queries (keys) and head each, and parts of
  // split tiles; a grid has less than 2^32 threads
  const bool f32 = a->dtype == STAPLE_F32;
  const int64_t tokens = a->total_q > a->total_k ? a->total_q : a->total_k;
  if ((tokens / (f32 ? 32 : 128) + a->n_seqs + 4) * a->n_heads + 4096 > kMaxLaunchRows * (f32 ? 2 : 1))
    return STAPLE_ERR_UNSUPPORTED;
  return STAPLE_OK;
}

static AttnView view(const staple_attn_t* a) {
  AttnView v{};
  v.n_seqs = a->n_seqs;
  v.total_q = a->total_q;
  v.total_k = a->total_k;
  v.n_heads = static_cast<int>(a->n_heads);
  v.n_kv_heads = static_cast<int>(a->n_kv_heads);
  v.group = static_cast<int>(a->n_heads / a->n_kv_heads);
  v.head_dim = static_cast<int>(a->head_dim);
  // a window past every position hides nothing; more sinks than positions are all of them
  v.window = a->window >= kMaxTokens ? 0 : static_cast<int>(a->window);
  v.sinks = a->sinks >= kMaxTokens ? kMaxTokens : static_cast<int>(a->sinks);
  v.scale = a->scale;
  v.cu_q = a->cu_q;
  v.cu_k = a->cu_k;
  v.q = view(a->q);
  v.k = view(a->k);
  v.v = view(a->v);
  v.o = view(a->o);
  v.d_o = view(a->d_o);
  v.dq = view(a->dq);
  v.dk = view(a->dk);
  v.dv = view(a->dv);
  v.lse = a->lse;
  return v;
}

static staple_status_t kv_check(const staple_kv_t* kv, bool pools, bool refs, bool table) {
  REQUIRE(kv);
  REQUIRE(kv->n_layers >= 1 && kv->n_pages >= 1 && kv->n_kv_heads >= 1 && kv->n_rows >= 1 &&
          kv->max_pages >= 1);
  if (!valid_dtype(kv->dtype) || !dims_ok(kv->head_dim) || kv->page_size < 16 ||
      kv->page_size > 1024 || (kv->page_size & (kv->page_size - 1)) != 0)
    return STAPLE_ERR_UNSUPPORTED;
  if (kv->n_layers > 16383 || kv->n_pages > kMaxCount || kv->n_kv_heads > 65535 ||
      kv->n_rows > kMaxCount || kv->max_pages > kMaxCount)
    return STAPLE_ERR_UNSUPPORTED;
  // a page's 16-byte pieces are numbered in 32 bits, with room for a stride of them
  if (kv->n_kv_heads * kv->page_size * kv->head_dim * elem_bytes(kv->dtype) > kMaxPageBytes)
    return STAPLE_ERR_UNSUPPORTED;
  if (pools) REQUIRE(kv->k_pages && kv->v_pages && aligned16(kv->k_pages) && aligned16(kv->v_pages));
  if (refs) REQUIRE(kv->refs);
  if (table) REQUIRE(kv->table && kv->lens);
  return STAPLE_OK;
}

static KvView view(const staple_kv_t* kv) {
  KvView v{};
  v.k_pages = static_cast<char*>(kv->k_pages);
  v.v_pages = static_cast<char*>(kv->v_pages);
  v.refs = kv->refs;
  v.table = kv->table;
  v.lens = kv->lens;
  v.refused = kv->refused;
  v.n_layers = kv->n_layers;
  v.n_pages = kv->n_pages;
  v.n_rows = kv->n_rows;
  v.max_pages = kv->max_pages;
  v.kv_heads = static_cast<int>(kv->n_kv_heads);
  v.page = static_cast<int>(kv->page_size);
  v.page_log2 = __builtin_ctzll(static_cast<unsigned long long>(kv->page_size));
  v.row_bytes = static_cast<int>(kv->head_dim) * elem_bytes(kv->dtype);
  return v;
}

static staple_status_t decode_check(const staple_kv_t* kv, const staple_attn_decode_t* a) {
  const staple_status_t st = kv_check(kv, true, false, true);
  if (st != STAPLE_OK) return st;
  REQUIRE(a && kv->n_layers == 1);
  REQUIRE(a->n_seqs >= 0 && a->n_heads >= 1 && a->n_heads % kv->n_kv_heads == 0);
  REQUIRE(a->window >= 0 && a->sinks >= 0 && std::isfinite(a->scale));
  REQUIRE(a->max_len >= 0 && a->max_len <= kv->max_pages * kv->page_size && a->max_len <= kMaxCount);
  REQUIRE(a->seqs || a->n_seqs <= kv->n_rows);
  if (a->n_heads > 65535 || a->n_seqs > kMaxLaunchRows || a->n_seqs * a->n_heads > kMaxLaunchRows)
    return STAPLE_ERR_UNSUPPORTED;
  return STAPLE_OK;
}

static DecodeView view(const staple_kv_t* kv, const staple_attn_decode_t* a) {
  DecodeView v{};
  v.n_seqs = a->n_seqs;
  v.max_len = a->max_len;
  // a window past every position hides nothing; more sinks than positions are all
  // of them: sums of the two stay far from 64 bits
  v.window = a->window >= a->max_len ? 0 : a->window;
  v.sinks = a->sinks < a->max_len ? a->sinks : a->max_len;
  v.n_heads = static_cast<int>(a->n_heads);
  v.group = static_cast<int>(a->n_heads / kv->n_kv_heads);
  v.head_dim = static_cast<int>(kv->head_dim);
  v.scale = a->scale;
  v.seqs = a->seqs;
  v.q = view(a->q);
  v.k_new = view(a->k_new);
  v.v_new = view(a->v_new);
  v.o = view(a->o);
  v.lse = a->lse;
  return v;
}

}  // namespace staple

using namespace staple;

#define CHECKED(expr)                          \
  do {                                         \
    const staple_status_t _st = (expr);        \
    if (_st != STAPLE_OK) return _st;          \
  } while (0)

extern "C" {

// ------------------------------------------------------------------ attention
size_t staple_attn_fwd_workspace_bytes(const staple_attn_t* a) {
  return attn_check(a) == STAPLE_OK ? attn_fwd_workspace_bytes(view(a), a->dtype) : 0;
}
staple_status_t staple_attn_fwd(const staple_attn_t* a, void* ws, size_t ws_bytes, void* stream) {
  CHECKED(attn_check(a));
  if (a->n_seqs == 0 || a->total_q == 0) return STAPLE_OK;
  REQUIRE(a->cu_q && a->cu_k && a->lse);
  REQUIRE(heads_ok(a->q, a->dtype) && heads_ok(a->o, a->dtype));
  REQUIRE(a->total_k == 0 || (heads_ok(a->k, a->dtype) && heads_ok(a->v, a->dtype)));
  const AttnView v = view(a);
  const size_t need = attn_fwd_workspace_bytes(v, a->dtype);
  if (ws_bytes < need) return STAPLE_ERR_WORKSPACE;
  REQUIRE(need == 0 || (ws && aligned16(ws)));
  GET_ERR(err);
  HIPCALL(launch_attn_fwd(v, a->dtype, ws, S(stream), err));
  return STAPLE_OK;
}

size_t staple_attn_bwd_workspace_bytes(const staple_attn_t* a) {
  return attn_check(a) == STAPLE_OK ? attn_bwd_workspace_bytes(view(a), a->dtype) : 0;
}

staple_status_t staple_attn_bwd(const staple_attn_t* a, void* ws, size_t ws_bytes, void* stream) {
  CHECKED(attn_check(a));
  if (a->n_seqs == 0 || (a->total_q == 0 && a->total_k == 0)) return STAPLE_OK;
  REQUIRE(a->cu_q && a->cu_k);
  REQUIRE(a->total_q == 0 || (a->lse && heads_ok(a->q, a->dtype) && heads_ok(a->o, a->dtype) &&
                              heads_ok(a->d_o, a->dtype) && heads_ok(a->dq, a->dtype)));
  REQUIRE(a->total_k == 0 || (heads_ok(a->k, a->dtype) && heads_ok(a->v, a->dtype) &&
                              heads_ok(a->dk, a->dtype) && heads_ok(a->dv, a->dtype)));
  const AttnView v = view(a);
  const size_t need = attn_bwd_workspace_bytes(v, a->dtype);
  if (ws_bytes < need) return STAPLE_ERR_WORKSPACE;
  REQUIRE(need == 0 || (ws && aligned16(ws)));
  GET_ERR(err);
  HIPCALL(launch_attn_bwd(v, a->dtype, ws, S(stream), err));
  return STAPLE_OK;
}

size_t staple_attn_decode_workspace_bytes(const staple_kv_t* kv, const staple_attn_decode_t* a) {
  return decode_check(kv, a) == STAPLE_OK ? attn_decode_workspace_bytes(view(kv), view(kv, a), kv->dtype)
                                          : 0;
}

staple_status_t staple_attn_decode_paged(const staple_kv_t* kv, const staple_attn_decode_t* a,
                                         void* ws, size_t ws_bytes, void* stream) {
  CHECKED(decode_check(kv, a));
  if (a->n_seqs == 0) return STAPLE_OK;
  REQUIRE(heads_ok(a->q, kv->dtype) && heads_ok(a->o, kv->dtype));
  REQUIRE((a->k_new.data == nullptr) == (a->v_new.data == nullptr));
  REQUIRE(a->k_new.data == nullptr || (heads_ok(a->k_new, kv->dtype) && heads_ok(a->v_new, kv->dtype)));
  const KvView kvv = view(kv);
  const DecodeView v = view(kv, a);
  const size_t need = attn_decode_workspace_bytes(kvv, v, kv->dtype);
  if (ws_bytes < need) return STAPLE_ERR_WORKSPACE;
  REQUIRE(need == 0 || (ws && aligned16(ws)));
  GET_ERR(err);
  HIPCALL(launch_attn_decode(kvv, v, kv->dtype, ws, S(stream), err));
  return STAPLE_OK;
}

// ---------------------------------------------------------------------- pages
staple_status_t staple_kv_append(const staple_kv_t* kv, const staple_heads_t* k_new,
                                 const staple_heads_t* v_new, int64_t n_new, const int32_t* seqs,
                                 int64_t n_seqs, const int32_t* cu_new, void* stream) {
  CHECKED(kv_check(kv, true, false, true));
  REQUIRE(kv->n_layers == 1 && n_new >= 0 && n_seqs >= 0 && n_seqs <= kMaxCount - 1);
  REQUIRE(cu_new || n_new == n_seqs);
  REQUIRE(seqs || n_seqs <= kv->n_rows);
  if (n_new > kMaxLaunchRows) return STAPLE_ERR_UNSUPPORTED;
  if (n_new == 0 || n_seqs == 0) return STAPLE_OK;
  REQUIRE(k_new && v_new && heads_ok(*k_new, kv->dtype) && heads_ok(*v_new, kv->dtype));
  GET_ERR(err);
  HIPCALL(launch_kv_append(view(kv), view(*k_new), view(*v_new), n_new, seqs, n_seqs, cu_new,
                           kv->dtype == STAPLE_BF16 ? 1 : 2, S(stream), err));
  return STAPLE_OK;
}

size_t staple_kv_extend_workspace_bytes(const staple_kv_t* kv, int64_t n_seqs) {
  return kv && kv->n_pages >= 1 && n_seqs >= 1 && n_seqs <= kKvMaxExtend
             ? kv_extend_workspace_bytes(kv->n_pages, n_seqs) : 0;
}

staple_status_t staple_kv_extend(const staple_kv_t* kv, const int32_t* seqs, const int32_t* n_new,
                                 int64_t n_seqs, void* ws, size_t ws_bytes, void* stream) {
  CHECKED(kv_check(kv, true, true, true));
  REQUIRE(n_seqs >= 0);
  if (n_seqs > kKvMaxExtend) return STAPLE_ERR_UNSUPPORTED;
  if (n_seqs == 0) return STAPLE_OK;
  REQUIRE(seqs);
  if (ws_bytes < kv_extend_workspace_bytes(kv->n_pages, n_seqs)) return STAPLE_ERR_WORKSPACE;
  REQUIRE(ws && aligned16(ws));
  GET_ERR(err);
  HIPCALL(launch_kv_extend(view(kv), seqs, n_new, n_seqs, ws, S(stream), err));
  return STAPLE_OK;
}

staple_status_t staple_kv_fork(const staple_kv_t* kv, const int32_t* parents,
                               const int32_t* children, int64_t n, void* stream) {
  CHECKED(kv_check(kv, false, true, true));
  REQUIRE(n >= 0);
  if (n > kMaxLaunchRows) return STAPLE_ERR_UNSUPPORTED;
  if (n == 0) return STAPLE_OK;
  REQUIRE(parents && children);
  GET_ERR(err);
  HIPCALL(launch_kv_fork(view(kv), parents, children, n, S(stream), err));
  return STAPLE_OK;
}

staple_status_t staple_kv_free(const staple_kv_t* kv, const int32_t* seqs, int64_t n, void* stream) {
  CHECKED(kv_check(kv, false, true, true));
  REQUIRE(n >= 0);
  if (n > kMaxLaunchRows) return STAPLE_ERR_UNSUPPORTED;
  if (n == 0) return STAPLE_OK;
  REQUIRE(seqs);
  GET_ERR(err);
  HIPCALL(launch_kv_free(view(kv), seqs, n, S(stream), err));
  return STAPLE_OK;
}

size_t staple_kv_compact_workspace_bytes(const staple_kv_t* kv) {
  return kv && kv->n_pages >= 1 && kv->n_pages <= kMaxCount ? kv_compact_workspace_bytes(kv->n_pages) : 0;
}

staple_status_t staple_kv_compact(const staple_kv_t* kv, int32_t* table_out, int32_t* refs_out,
                                  int32_t* n_live, void* ws, size_t ws_bytes, void* stream) {
  CHECKED(kv_check(kv, true, true, true));
  REQUIRE(table_out && refs_out && n_live);
  if (ws_bytes < kv_compact_workspace_bytes(kv->n_pages)) return STAPLE_ERR_WORKSPACE;
  REQUIRE(ws && aligned16(ws));
  GET_ERR(err);
  HIPCALL(launch_kv_compact(view(kv), table_out, refs_out, n_live, ws, S(stream), err));
  return STAPLE_OK;
}

staple_status_t staple_kv_copy_pages(const staple_kv_t* kv, const int32_t* src, const int32_t* dst,
                                     int64_t n, void* stream) {
  CHECKED(kv_check(kv, true, false, false));
  REQUIRE(n >= 0);
  if (n > kMaxLaunchRows) return STAPLE_ERR_UNSUPPORTED;
  if (n == 0) return STAPLE_OK;
  REQUIRE(src && dst);
  GET_ERR(err);
  HIPCALL(launch_kv_copy(view(kv), src, dst, n, S(stream), err));
  return STAPLE_OK;
}

}  // extern "C"
