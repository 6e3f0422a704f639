// Attention of one new token per sequence over a paged key-value cache.
#include "attn_row.h"

namespace staple {

template <typename T>
__global__ __launch_bounds__(64) void attn_decode_row_kernel(KvView kv, DecodeView a, int* err) {
  const int64_t i = blockIdx.x / a.n_heads, h = blockIdx.x % a.n_heads, hk = h / a.group;
  const int64_t s = a.seqs ? a.seqs[i] : i;
  const bool fine = s >= 0 && s < kv.n_rows;
  int64_t len = fine ? kv.lens[s] : 0;
  if (!fine || len < 0 || len > a.max_len) {
    flag_index_error(err);
    len = len < 0 ? 0 : min(len, a.max_len);
  }
  const int32_t* pages = kv.table + (fine ? s : 0) * kv.max_pages;
  const int64_t p = len - 1;
  int64_t sink_end, lo;
  visible_keys(p, a.window, a.sinks, &sink_end, &lo);
  const Row2 q = load_row<T>(a.q, i, h, a.head_dim);
  RowSoftmax sm;
  for (int64_t j = 0; j <= p; ++j) {
    if (j == sink_end) j = lo;
    if (j > p) break;
    const int64_t page = pages[j >> kv.page_log2];
    if (page < 0 || page >= kv.n_pages) {
      flag_index_error(err);
      continue;
    }
    const int64_t slot = page * kv.kv_heads * kv.page + (j & (kv.page - 1));
    HeadsView kp{kv.k_pages, a.head_dim, static_cast<int64_t>(kv.page) * a.head_dim};
    HeadsView vp{kv.v_pages, a.head_dim, static_cast<int64_t>(kv.page) * a.head_dim};
    Row2 k, v;
    if (j == p && a.k_new.data) {
      k = load_row<T>(a.k_new, i, hk, a.head_dim);
      v = load_row<T>(a.v_new, i, hk, a.head_dim);
      if (h % a.group == 0) {
        store_row<T>(kp, slot, hk, a.head_dim, k);
        store_row<T>(vp, slot, hk, a.head_dim, v);
      }
    } else {
      k = load_row<T>(kp, slot, hk, a.head_dim);
      v = load_row<T>(vp, slot, hk, a.head_dim);
    }
    sm.add(dot(q, k) * a.scale, v);
  }
  store_row<T>(a.o, i, h, a.head_dim, sm.value());
  if (a.lse && threadIdx.x == 0) a.lse[i * a.n_heads + h] = sm.lse();
}

size_t attn_decode_workspace_bytes(const KvView& kv, const DecodeView& a, int dtype) { return 0; }

hipError_t launch_attn_decode(const KvView& kv, const DecodeView& a, int dtype, void* ws,
                              hipStream_t s, int* err) {
  const unsigned wgs = static_cast<unsigned>(a.n_seqs * a.n_heads);
  if (dtype == STAPLE_BF16) attn_decode_row_kernel<bf16_t><<<wgs, 64, 0, s>>>(kv, a, err);
  else attn_decode_row_kernel<float><<<wgs, 64, 0, s>>>(kv, a, err);
  return hipGetLastError();
}

}  // namespace staple
