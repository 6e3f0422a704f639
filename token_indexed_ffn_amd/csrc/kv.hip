// Pages of the key-value cache: writing new tokens, growing, forking and
// ending sequences, and packing the pool.  All state (reference counts, page
// table, lengths) is on the device.
//
// The bookkeeping is integer work on a few kilobytes and is bound by launch
// and memory latency, so each call is one or two launches: forking and ending
// take one workgroup per sequence (the counts are integer atomics, whose
// order does not change the result); growing and packing must hand out pages
// in a fixed order and run in one workgroup, which ranks free and live pages
// with block-wide prefix sums.  Moved rows are copied by a second launch that
// spreads (page, layer, K or V) over workgroups, 16 bytes a lane: every byte
// is read once and written once, bound by HBM.
//
// Measured: 16000 new tokens of 16 heads of 128 into pages 53 us (5.0 TB/s of
// reads and writes); half a pool of 1 GB packed 217 us (4.9 TB/s) after 8 us of
// ranking 4096 pages; of 64 beams, ending 3 us, forking 3, growing by one token
// 7 (four loads that depend on each other, then a scan of 2048 counts) and 18
// for their 64 half-filled pages in 4 layers (17 MB written, scattered).
#include "common.h"
#include "kv.h"

namespace staple {

constexpr int kBookThreads = 1024;
constexpr int kBookWaves = kBookThreads / 64;

// Inclusive sum over the lanes of a wave, which V holds.
template <typename V>
__device__ __forceinline__ V wave_scan(V v) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const V o = __shfl_up(v, d);
    if (lane >= d) v += o;
  }
  return v;
}

// Exclusive sum over a workgroup of kBookThreads and the whole sum in *total.
template <typename V>
__device__ __forceinline__ int64_t block_scan(V v, int64_t* waves, int64_t* total) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const V inc = wave_scan(v);
  __syncthreads();   // the previous use of waves[] is over
  if (lane == 63) waves[w] = inc;
  __syncthreads();
  int64_t before = 0, all = 0;
#pragma unroll
  for (int i = 0; i < kBookWaves; ++i) {
    const int64_t c = waves[i];
    if (i < w) before += c;
    all += c;
  }
  *total = all;
  return before + inc - v;
}

// Pages of a row (0 and the error word where its length is impossible).
__device__ __forceinline__ int64_t pages_of_row(const KvView& kv, int len, int* err) {
  const int64_t n = (static_cast<int64_t>(len) + kv.page - 1) >> kv.page_log2;
  if (len < 0 || n > kv.max_pages) {
    flag_index_error(err);
    return 0;
  }
  return n;
}

// ---------------------------------------------------------------- free, fork
__global__ __launch_bounds__(256) void kv_free_kernel(KvView kv, const int32_t* seqs, int* err) {
  const int64_t s = seqs[blockIdx.x];
  if (s < 0 || s >= kv.n_rows) {
    if (threadIdx.x == 0) flag_index_error(err);
    return;
  }
  const int64_t n = pages_of_row(kv, kv.lens[s], err);
  int32_t* row = kv.table + s * kv.max_pages;
  for (int64_t j = threadIdx.x; j < n; j += 256) {
    const int p = row[j];
    if (p < 0 || p >= kv.n_pages) flag_index_error(err);
    else if (atomicSub(&kv.refs[p], 1) <= 0) flag_index_error(err);
    row[j] = -1;
  }
  __syncthreads();   // every thread has read the length
  if (threadIdx.x == 0) {
    kv.lens[s] = 0;
    if (kv.refused) kv.refused[s] = 0;
  }
}

__global__ __launch_bounds__(256) void kv_fork_kernel(KvView kv, const int32_t* parents,
                                                      const int32_t* children, int* err) {
  const int64_t a = parents[blockIdx.x], c = children[blockIdx.x];
  if (a < 0 || a >= kv.n_rows || c < 0 || c >= kv.n_rows || a == c || kv.lens[c] != 0) {
    if (threadIdx.x == 0) flag_index_error(err);
    return;
  }
  const int len = kv.lens[a];
  const int64_t n = pages_of_row(kv, len, err);
  const int32_t* from = kv.table + a * kv.max_pages;
  int32_t* to = kv.table + c * kv.max_pages;
  for (int64_t j = threadIdx.x; j < n; j += 256) {
    const int p = from[j];
    if (p < 0 || p >= kv.n_pages) flag_index_error(err);
    else atomicAdd(&kv.refs[p], 1);
    to[j] = p;
  }
  __syncthreads();   // every thread has read the child's length
  if (threadIdx.x == 0) {
    if (n > 0) kv.lens[c] = len;
    if (kv.refused) kv.refused[c] = 0;
  }
}

// -------------------------------------------------------------------- extend
// One workgroup.  Sequence i's pages are the ranks [first[i], first[i + 1])
// of the free list, a copy-on-write page first; rank r goes to column
// col0[i] + r - first[i] of its row (the copied page in place of the shared
// last one).
__global__ __launch_bounds__(kBookThreads) void kv_extend_kernel(KvView kv, const int32_t* seqs,
                                                                 const int32_t* n_new, int n,
                                                                 int32_t* free_list, KvCopy* copies,
                                                                 int* err) {
  constexpr int kPer = kKvMaxExtend / kBookThreads;
  __shared__ int first[kKvMaxExtend], col0[kKvMaxExtend], row[kKvMaxExtend];
  __shared__ int64_t waves[kBookWaves];
  __shared__ int refused;
  if (threadIdx.x == 0) refused = 0;
  __syncthreads();
  const int64_t max_len = min(kv.max_pages << kv.page_log2, static_cast<int64_t>(0x7fffffff));
  int old_len[kPer], new_len[kPer], need[kPer], cow_page[kPer];
  int asked[kPer];   // the row that is to grow, -1: none
  // sequence i, by thread i % kBookThreads: the loads of one depend on each other
  auto look = [&](int i, int k) {
    row[i] = -1;
    need[k] = 0;
    cow_page[k] = -1;
    old_len[k] = new_len[k] = 0;
    asked[k] = -1;
    if (i >= n) return;
    const int s = seqs[i];
    const int add = n_new ? n_new[i] : 1;
    if (s < 0 || s >= kv.n_rows) return flag_index_error(err);
    if (add != 0) asked[k] = s;
    else if (kv.refused) kv.refused[s] = 0;
    if (add < 0) return flag_index_error(err);
    const int len = kv.lens[s];
    const int64_t held = pages_of_row(kv, len, err);
    if (len < 0 || (len > 0 && held == 0)) return;
    const int64_t want = (static_cast<int64_t>(len) + add + kv.page - 1) >> kv.page_log2;
    if (static_cast<int64_t>(len) + add > max_len || want - held > kv.n_pages) {
      refused = 1;
      return;
    }
    row[i] = s;
    col0[i] = static_cast<int>(held);
    old_len[k] = len;
    new_len[k] = len + add;
    need[k] = static_cast<int>(want - held);
    if (add > 0 && (len & (kv.page - 1)) != 0) {
      const int p = kv.table[s * kv.max_pages + held - 1];
      if (p < 0 || p >= kv.n_pages) flag_index_error(err);
      else if (kv.refs[p] > 1) {
        cow_page[k] = p;
        col0[i] -= 1;
        ++need[k];
      }
    }
  };
  int64_t total = 0;
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    if (k * kBookThreads >= n) break;
    const int i = k * kBookThreads + threadIdx.x;
    look(i, k);
    int64_t all;
    first[i] = static_cast<int>(total + block_scan(static_cast<int64_t>(need[k]), waves, &all));
    total += all;
  }
  // the lowest `total` free pages
  int64_t found = 0;
  if (total <= kv.n_pages) {
    for (int64_t base = 0; base < kv.n_pages && found < total; base += 4 * kBookThreads) {
      const int64_t p0 = base + 4 * threadIdx.x;
      bool is_free[4];
      int cnt = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        is_free[e] = p0 + e < kv.n_pages && kv.refs[p0 + e] == 0;
        cnt += is_free[e];
      }
      int64_t all;
      int64_t r = found + block_scan(cnt, waves, &all);
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (is_free[e]) {
          if (r < total) free_list[r] = static_cast<int>(p0 + e);
          ++r;
        }
      found += all;
    }
  }
  __syncthreads();   // first[], col0[], row[], refused and this workgroup's free_list
  const bool refuse = refused != 0 || found < total;
  if (refuse && threadIdx.x == 0) atomicOr(err, kErrNoPages);
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int i = k * kBookThreads + threadIdx.x;
    if (i >= n) break;
    KvCopy c{-1, -1, 0};
    const bool grown = !refuse && row[i] >= 0;
    if (kv.refused && asked[k] >= 0) kv.refused[asked[k]] = grown ? 0 : 1;
    if (grown) {
      if (cow_page[k] >= 0) {
        c = KvCopy{cow_page[k], free_list[first[i]], old_len[k] & (kv.page - 1)};
        atomicSub(&kv.refs[cow_page[k]], 1);
      }
      kv.lens[row[i]] = new_len[k];
    }
    copies[i] = c;
  }
  if (refuse) return;
  for (int r = threadIdx.x; r < total; r += kBookThreads) {
    int lo = 0, hi = n;   // first[lo] <= r < first[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (first[mid] <= r) lo = mid;
      else hi = mid;
    }
    const int page = free_list[r];
    kv.refs[page] = 1;
    kv.table[static_cast<int64_t>(row[lo]) * kv.max_pages + col0[lo] + (r - first[lo])] = page;
  }
}

// ------------------------------------------------------------- page contents
// Slots [0, slots) of every head of page src to page dst, for one layer's K
// (kv_side 0) or V: `part` of `parts` workgroups.
__device__ __forceinline__ void copy_page(const KvView& kv, int64_t layer, int side, int64_t src,
                                          int64_t dst, int slots, int part, int parts) {
  char* pool = side ? kv.v_pages : kv.k_pages;
  const int64_t page_bytes = static_cast<int64_t>(kv.kv_heads) * kv.page * kv.row_bytes;
  const char* from = pool + (layer * kv.n_pages + src) * page_bytes;
  char* to = pool + (layer * kv.n_pages + dst) * page_bytes;
  const int per_head = slots * (kv.row_bytes >> 4);      // 16-byte pieces in use per head
  const int head_bytes = kv.page * kv.row_bytes;
  const int pieces = per_head * kv.kv_heads;
  constexpr int kAhead = 4;                              // loads in flight per thread
  for (int i0 = part * blockDim.x + threadIdx.x; i0 < pieces; i0 += kAhead * parts * blockDim.x) {
    uint4 v[kAhead];
    int64_t off[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int i = i0 + k * parts * blockDim.x;
      const int h = i / per_head;
      off[k] = static_cast<int64_t>(h) * head_bytes + static_cast<int64_t>(i - h * per_head) * 16;
      if (i < pieces) v[k] = *reinterpret_cast<const uint4*>(from + off[k]);
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (i0 + k * parts * blockDim.x < pieces) *reinterpret_cast<uint4*>(to + off[k]) = v[k];
  }
}

// blockIdx.z: part of a page, so that a few small copies still fill the GPU.
__global__ __launch_bounds__(256) void kv_copy_list_kernel(KvView kv, const KvCopy* copies) {
  const KvCopy c = copies[blockIdx.x];
  if (c.src < 0) return;
  copy_page(kv, blockIdx.y >> 1, blockIdx.y & 1, c.src, c.dst, c.slots, blockIdx.z, gridDim.z);
}

__global__ __launch_bounds__(256) void kv_copy_pages_kernel(KvView kv, const int32_t* src,
                                                            const int32_t* dst, int* err) {
  const int64_t a = src[blockIdx.x], b = dst[blockIdx.x];
  if (a < 0 || a >= kv.n_pages || b < 0 || b >= kv.n_pages) {
    if (threadIdx.x == 0) flag_index_error(err);
    return;
  }
  if (a != b) copy_page(kv, blockIdx.y >> 1, blockIdx.y & 1, a, b, kv.page, 0, 1);
}

// ------------------------------------------------------------------- compact
// One workgroup: n_live, to[p] (where page p's contents end up) and the moves.
__global__ __launch_bounds__(kBookThreads) void kv_rank_kernel(KvView kv, int32_t* to,
                                                               int32_t* move_src, int32_t* move_dst,
                                                               int32_t* n_moves, int32_t* n_live) {
  __shared__ int64_t waves[kBookWaves];
  int cnt = 0;
  for (int64_t p = threadIdx.x; p < kv.n_pages; p += kBookThreads) cnt += kv.refs[p] > 0;
  int64_t live;
  block_scan(cnt, waves, &live);
  int64_t holes = 0, movers = 0;   // ranks given out so far
  for (int64_t base = 0; base < kv.n_pages; base += 4 * kBookThreads) {
    const int64_t p0 = base + 4 * threadIdx.x;
    int nh = 0, nm = 0;
    bool is_live[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int64_t p = p0 + e;
      is_live[e] = p < kv.n_pages && kv.refs[p] > 0;
      nh += p < live && !is_live[e];
      nm += p >= live && is_live[e];
    }
    int64_t all_h, all_m;
    int64_t rh = holes + block_scan(nh, waves, &all_h);
    int64_t rm = movers + block_scan(nm, waves, &all_m);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int64_t p = p0 + e;
      if (p < live && !is_live[e]) move_dst[rh++] = static_cast<int>(p);
      if (p >= live && is_live[e]) move_src[rm++] = static_cast<int>(p);
      if (p < kv.n_pages) to[p] = static_cast<int>(p);
    }
    holes += all_h;
    movers += all_m;
  }
  __syncthreads();
  for (int64_t m = threadIdx.x; m < movers; m += kBookThreads) to[move_src[m]] = move_dst[m];
  if (threadIdx.x == 0) {
    *n_moves = static_cast<int>(movers);
    *n_live = static_cast<int>(live);
  }
}

// The moves' page contents (blockIdx.y: layer and K or V), and with
// blockIdx.y == 2 n_layers the table rows and the counts.
__global__ __launch_bounds__(256) void kv_move_kernel(KvView kv, const int32_t* to,
                                                      const int32_t* move_src,
                                                      const int32_t* move_dst,
                                                      const int32_t* n_moves, int32_t* table_out,
                                                      int32_t* refs_out, int* err) {
  const int moves = *n_moves;
  if (blockIdx.y < 2 * kv.n_layers) {
    for (int m = blockIdx.x; m < moves; m += gridDim.x)
      copy_page(kv, blockIdx.y >> 1, blockIdx.y & 1, move_src[m], move_dst[m], kv.page, 0, 1);
    return;
  }
  const bool moved_table = table_out != kv.table, moved_refs = refs_out != kv.refs;
  for (int64_t s = blockIdx.x; s < kv.n_rows; s += gridDim.x) {
    const int64_t n = pages_of_row(kv, kv.lens[s], err);
    const int32_t* from = kv.table + s * kv.max_pages;
    int32_t* out = table_out + s * kv.max_pages;
    for (int64_t j = threadIdx.x; j < (moved_table ? kv.max_pages : n); j += 256) {
      int p = from[j];
      if (j < n) {
        if (p < 0 || p >= kv.n_pages) flag_index_error(err);
        else p = to[p];
      }
      out[j] = p;
    }
  }
  // counts: a move's pair is written by its own thread, every other page's
  // count stays (a hole is free and below n_live; its count comes with its move)
  const int64_t step = static_cast<int64_t>(gridDim.x) * 256;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  for (int64_t m = t0; m < moves; m += step) {
    refs_out[move_dst[m]] = kv.refs[move_src[m]];
    refs_out[move_src[m]] = 0;
  }
  if (!moved_refs) return;
  const int64_t live = moves > 0 ? move_dst[moves - 1] + 1 : 0;   // no hole at or past this
  for (int64_t p = t0; p < kv.n_pages; p += step) {
    const int r = kv.refs[p];
    if (to[p] == p && !(r <= 0 && p < live)) refs_out[p] = r;
  }
}

// -------------------------------------------------------------------- append
constexpr int kAppendRows = 4;   // new rows per workgroup

__global__ __launch_bounds__(256) void kv_append_kernel(KvView kv, HeadsView kn, HeadsView vn,
                                                        int64_t n_new, const int32_t* seqs,
                                                        int64_t n_seqs, const int32_t* cu_new,
                                                        int elem_log2, int* err) {
  __shared__ int64_t dst[kAppendRows];   // byte offset of the row's slot in head 0, -1: none
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * kAppendRows;
  if (threadIdx.x < kAppendRows) {
    const int64_t t = t0 + threadIdx.x;
    int64_t at = -1;
    if (t < n_new) {
      int64_t i = t, end = t + 1;   // the sequence, and the end of its new rows
      if (cu_new) {
        int64_t lo = 0, hi = n_seqs;   // cu_new[lo] <= t < cu_new[hi]
        while (hi - lo > 1) {
          const int64_t mid = (lo + hi) >> 1;
          if (cu_new[mid] <= t) lo = mid;
          else hi = mid;
        }
        i = lo;
        end = cu_new[lo + 1];
        if (cu_new[lo] > t || end <= t) i = -1;   // in no sequence
      }
      if (i >= 0) {
        const int64_t s = seqs ? seqs[i] : i;
        bool fine = s >= 0 && s < kv.n_rows;
        const int64_t len = fine ? kv.lens[s] : 0;
        const int64_t pos = len - (end - t);
        fine = fine && pos >= 0 && (pos >> kv.page_log2) < kv.max_pages;
        const int64_t p = fine ? kv.table[s * kv.max_pages + (pos >> kv.page_log2)] : -1;
        if (p < 0 || p >= kv.n_pages) flag_index_error(err);
        else if (!was_refused(kv, s)) at = (p * kv.kv_heads * kv.page + (pos & (kv.page - 1))) * kv.row_bytes;
      }
    }
    dst[threadIdx.x] = at;
  }
  __syncthreads();
  const int vecs = kv.row_bytes >> 4;          // 16-byte pieces per head
  const int per_row = kv.kv_heads * vecs;
  for (int i = threadIdx.x; i < 2 * kAppendRows * per_row; i += 256) {
    const int side = i >= kAppendRows * per_row;
    const int r = i - side * kAppendRows * per_row;
    const int row = r / per_row, in_row = r - row * per_row;
    const int64_t at = dst[row];
    if (at < 0) continue;
    const int h = in_row / vecs, c = in_row - h * vecs;
    const HeadsView& src = side ? vn : kn;
    const uint4 v = *reinterpret_cast<const uint4*>(
        src.data + (((t0 + row) * src.row_stride + h * src.head_stride) << elem_log2) + c * 16);
    char* pool = side ? kv.v_pages : kv.k_pages;
    *reinterpret_cast<uint4*>(pool + at + static_cast<int64_t>(h) * kv.page * kv.row_bytes + c * 16) = v;
  }
}

// ------------------------------------------------------------------ launches
hipError_t launch_kv_free(const KvView& kv, const int32_t* seqs, int64_t n, hipStream_t s, int* err) {
  kv_free_kernel<<<static_cast<unsigned>(n), 256, 0, s>>>(kv, seqs, err);
  return hipGetLastError();
}

hipError_t launch_kv_fork(const KvView& kv, const int32_t* parents, const int32_t* children,
                          int64_t n, hipStream_t s, int* err) {
  kv_fork_kernel<<<static_cast<unsigned>(n), 256, 0, s>>>(kv, parents, children, err);
  return hipGetLastError();
}

size_t kv_extend_workspace_bytes(int64_t n_pages, int64_t n) {
  return align_up(static_cast<size_t>(n_pages) * sizeof(int32_t), 256) +
         align_up(static_cast<size_t>(n) * sizeof(KvCopy), 256);
}

hipError_t launch_kv_extend(const KvView& kv, const int32_t* seqs, const int32_t* n_new, int64_t n,
                            void* ws, hipStream_t s, int* err) {
  Workspace w(ws, kv_extend_workspace_bytes(kv.n_pages, n));
  int32_t* free_list = w.take<int32_t>(static_cast<size_t>(kv.n_pages) * sizeof(int32_t));
  KvCopy* copies = w.take<KvCopy>(static_cast<size_t>(n) * sizeof(KvCopy));
  kv_extend_kernel<<<1, kBookThreads, 0, s>>>(kv, seqs, n_new, static_cast<int>(n), free_list,
                                              copies, err);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  // a part has at most one round of loads: 4 x 256 x 16 bytes
  const int64_t page_bytes = static_cast<int64_t>(kv.kv_heads) * kv.page * kv.row_bytes;
  const int64_t parts = (page_bytes + 16383) / 16384;
  kv_copy_list_kernel<<<dim3(static_cast<unsigned>(n), static_cast<unsigned>(2 * kv.n_layers),
                             static_cast<unsigned>(parts < 64 ? parts : 64)), 256, 0, s>>>(kv, copies);
  return hipGetLastError();
}

hipError_t launch_kv_copy(const KvView& kv, const int32_t* src, const int32_t* dst, int64_t n,
                          hipStream_t s, int* err) {
  kv_copy_pages_kernel<<<dim3(static_cast<unsigned>(n), static_cast<unsigned>(2 * kv.n_layers)), 256,
                         0, s>>>(kv, src, dst, err);
  return hipGetLastError();
}

size_t kv_compact_workspace_bytes(int64_t n_pages) {
  return 3 * align_up(static_cast<size_t>(n_pages) * sizeof(int32_t), 256) + 256;
}

hipError_t launch_kv_compact(const KvView& kv, int32_t* table_out, int32_t* refs_out,
                             int32_t* n_live, void* ws, hipStream_t s, int* err) {
  Workspace w(ws, kv_compact_workspace_bytes(kv.n_pages));
  const size_t bytes = static_cast<size_t>(kv.n_pages) * sizeof(int32_t);
  int32_t* to = w.take<int32_t>(bytes);
  int32_t* src = w.take<int32_t>(bytes);
  int32_t* dst = w.take<int32_t>(bytes);
  int32_t* n_moves = w.take<int32_t>(sizeof(int32_t));
  kv_rank_kernel<<<1, kBookThreads, 0, s>>>(kv, to, src, dst, n_moves, n_live);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  // at most half the pages move; more workgroups than that, or than fill the
  // GPU several times over, would find nothing to do
  int64_t x = (kv.n_pages + 1) / 2;
  if (x > 2048) x = 2048;
  kv_move_kernel<<<dim3(static_cast<unsigned>(x), static_cast<unsigned>(2 * kv.n_layers + 1)), 256, 0,
                   s>>>(kv, to, src, dst, n_moves, table_out, refs_out, err);
  return hipGetLastError();
}

hipError_t launch_kv_append(const KvView& kv, const HeadsView& k_new, const HeadsView& v_new,
                            int64_t n_new, const int32_t* seqs, int64_t n_seqs,
                            const int32_t* cu_new, int elem_log2, hipStream_t s, int* err) {
  const int64_t wgs = (n_new + kAppendRows - 1) / kAppendRows;
  kv_append_kernel<<<static_cast<unsigned>(wgs), 256, 0, s>>>(kv, k_new, v_new, n_new, seqs, n_seqs,
                                                              cu_new, elem_log2, err);
  return hipGetLastError();
}

}  // namespace staple
