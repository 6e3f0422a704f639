// Attention one row at a time: a wave holds one query (or one key) across its
// lanes, two elements a lane, and walks the keys (queries) that it sees one by
// one.  A masked pair is never touched, so whatever its rows hold has no part
// in the result.
#pragma once

#include "attn.h"

namespace staple {

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int d = 32; d > 0; d /= 2) v += __shfl_xor(v, d);
  return v;
}

// Elements `lane` and `lane + 64` of a head's row (0 past head_dim).
struct Row2 {
  float x[2];
};
template <typename T>
__device__ __forceinline__ Row2 load_row(const HeadsView& t, int64_t row, int64_t head, int dim) {
  const int lane = threadIdx.x & 63;
  const T* p = reinterpret_cast<const T*>(t.data) + row * t.row_stride + head * t.head_stride;
  Row2 r;
  r.x[0] = lane < dim ? Elem<T>::load(p, lane) : 0.0f;
  r.x[1] = lane + 64 < dim ? Elem<T>::load(p, lane + 64) : 0.0f;
  return r;
}
template <typename T>
__device__ __forceinline__ void store_row(const HeadsView& t, int64_t row, int64_t head, int dim,
                                          const Row2& r) {
  const int lane = threadIdx.x & 63;
  T* p = reinterpret_cast<T*>(t.data) + row * t.row_stride + head * t.head_stride;
  if (lane < dim) Elem<T>::store(p, lane, r.x[0]);
  if (lane + 64 < dim) Elem<T>::store(p, lane + 64, r.x[1]);
}
__device__ __forceinline__ float dot(const Row2& a, const Row2& b) {
  return wave_sum(a.x[0] * b.x[0] + a.x[1] * b.x[1]);
}

// Running softmax of one query: largest score, sum of exponentials, weighted
// sum of the value rows.
struct RowSoftmax {
  float top = -INFINITY, sum = 0.0f;
  Row2 acc{{0.0f, 0.0f}};
  __device__ __forceinline__ void add(float s, const Row2& v) {
    const float t = fmaxf(top, s);
    const float base = t == -INFINITY ? 0.0f : t;
    const float keep = __expf(top - base), p = __expf(s - base);
    sum = sum * keep + p;
    acc.x[0] = acc.x[0] * keep + p * v.x[0];
    acc.x[1] = acc.x[1] * keep + p * v.x[1];
    top = t;
  }
  __device__ __forceinline__ Row2 value() const {
    const float r = sum == 0.0f ? 0.0f : 1.0f / sum;
    return Row2{{acc.x[0] * r, acc.x[1] * r}};
  }
};

}  // namespace staple
