// Device views of the paged key-value cache and the launchers of kv.hip.
#pragma once

#include "common.h"

namespace staple {

// Bit of the device error word (beside kErrIndexRange): out of pages.
constexpr int kErrNoPages = 2;

// A [rows][heads][head_dim] operand; strides in elements.
struct HeadsView {
  char* data;
  int64_t row_stride, head_stride;
};

struct KvView {
  char* k_pages;
  char* v_pages;
  int32_t* refs;
  int32_t* table;
  int32_t* lens;
  int32_t* refused;        // or null
  int64_t n_layers, n_pages, n_rows, max_pages;
  int kv_heads, page, page_log2, row_bytes;   // row_bytes: one slot of one head
};

// Whether row s (in range) was refused its last growth: its new tokens have no place.
__device__ __forceinline__ bool was_refused(const KvView& kv, int64_t s) { return kv.refused && kv.refused[s] != 0; }

// One page copy: the first `slots` slots of every head; src -1: nothing.
struct KvCopy {
  int32_t src, dst, slots;
};

constexpr int kKvMaxExtend = 4096;

hipError_t launch_kv_free(const KvView& kv, const int32_t* seqs, int64_t n, hipStream_t s, int* err);
hipError_t launch_kv_fork(const KvView& kv, const int32_t* parents, const int32_t* children,
                          int64_t n, hipStream_t s, int* err);
size_t kv_extend_workspace_bytes(int64_t n_pages, int64_t n);
hipError_t launch_kv_extend(const KvView& kv, const int32_t* seqs, const int32_t* n_new, int64_t n,
                            void* ws, hipStream_t s, int* err);
hipError_t launch_kv_copy(const KvView& kv, const int32_t* src, const int32_t* dst, int64_t n,
                          hipStream_t s, int* err);
size_t kv_compact_workspace_bytes(int64_t n_pages);
hipError_t launch_kv_compact(const KvView& kv, int32_t* table_out, int32_t* refs_out,
                             int32_t* n_live, void* ws, hipStream_t s, int* err);
hipError_t launch_kv_append(const KvView& kv, const HeadsView& k_new, const HeadsView& v_new,
                            int64_t n_new, const int32_t* seqs, int64_t n_seqs,
                            const int32_t* cu_new, int elem_log2, hipStream_t s, int* err);

}  // namespace staple
