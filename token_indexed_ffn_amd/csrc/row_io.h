// Rows of bf16 or fp32 elements read and written eight elements a lane, and sums over a
// workgroup's waves in a fixed order.
#pragma once

#include "common.h"

namespace staple {

// Eight consecutive elements, 16-byte aligned.
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const f32x4_t a = *reinterpret_cast<const f32x4_t*>(p);
  const f32x4_t b = *reinterpret_cast<const f32x4_t*>(p + 4);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[i] = a[i];
    v[i + 4] = b[i];
  }
}
__device__ __forceinline__ void load8(const bf16_t* p, float (&v)[8]) {
  const u32x4_t w = *reinterpret_cast<const u32x4_t*>(p);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  *reinterpret_cast<f32x4_t*>(p) = f32x4_t{v[0], v[1], v[2], v[3]};
  *reinterpret_cast<f32x4_t*>(p + 4) = f32x4_t{v[4], v[5], v[6], v[7]};
}
__device__ __forceinline__ void store8(bf16_t* p, const float (&v)[8]) {
  u32x4_t w;
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
  *reinterpret_cast<u32x4_t*>(p) = w;
}
__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ float load1(const bf16_t* p) { return bf16_to_f32(p->bits); }
__device__ __forceinline__ void store1(float* p, float v) { *p = v; }
__device__ __forceinline__ void store1(bf16_t* p, float v) { p->bits = f32_to_bf16(v); }

// Words that begin at any element of type E: global memory takes 16 bytes at any address.
template <typename E, int WORDS> struct LooseWords {
  typedef __attribute__((ext_vector_type(WORDS), aligned(sizeof(E)))) uint32_t type;
};

// Eight elements as they lie in memory, 16-byte aligned (load) or not (load_loose).
template <typename E> struct Raw;
template <> struct Raw<bf16_t> {
  u32x4_t a;
  __device__ __forceinline__ void load(const bf16_t* p) { a = *reinterpret_cast<const u32x4_t*>(p); }
  __device__ __forceinline__ void clear() { a = u32x4_t{0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u}; }   // -inf
  // Of data that nothing reads again soon: it is not to push other lines out of the caches.
  __device__ __forceinline__ void load_once(const bf16_t* p) { a = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(p)); }
  typedef LooseWords<bf16_t, 4>::type loose_t;
  __device__ __forceinline__ void load_loose(const bf16_t* p) { a = *reinterpret_cast<const loose_t*>(p); }
  __device__ __forceinline__ void load_loose_once(const bf16_t* p) { a = __builtin_nontemporal_load(reinterpret_cast<const loose_t*>(p)); }
  // What was made of these elements is made again after this, rather than kept in registers.
  __device__ __forceinline__ void forget() { asm volatile("" : "+v"(a)); }
  __device__ __forceinline__ void get(float (&v)[8]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(a[i] << 16);
      v[2 * i + 1] = __uint_as_float(a[i] & 0xffff0000u);
    }
  }
};
template <> struct Raw<float> {
  f32x4_t a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = *reinterpret_cast<const f32x4_t*>(p);
    b = *reinterpret_cast<const f32x4_t*>(p + 4);
  }
  __device__ __forceinline__ void clear() {
    const float x = -__builtin_inff();
    a = b = f32x4_t{x, x, x, x};
  }
  __device__ __forceinline__ void load_once(const float* p) {
    a = __builtin_nontemporal_load(reinterpret_cast<const f32x4_t*>(p));
    b = __builtin_nontemporal_load(reinterpret_cast<const f32x4_t*>(p + 4));
  }
  typedef __attribute__((ext_vector_type(4), aligned(4))) float loose_t;
  __device__ __forceinline__ void load_loose(const float* p) {
    a = *reinterpret_cast<const loose_t*>(p);
    b = *reinterpret_cast<const loose_t*>(p + 4);
  }
  __device__ __forceinline__ void load_loose_once(const float* p) {
    a = __builtin_nontemporal_load(reinterpret_cast<const loose_t*>(p));
    b = __builtin_nontemporal_load(reinterpret_cast<const loose_t*>(p + 4));
  }
  __device__ __forceinline__ void forget() { asm volatile("" : "+v"(a), "+v"(b)); }
  __device__ __forceinline__ void get(float (&v)[8]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = a[i];
      v[i + 4] = b[i];
    }
  }
};

// A row's elements in groups of eight that begin where its memory is 16-byte aligned: `shift`
// elements before the row.  The elements outside full groups are the first `head` (fewer than
// eight) and the last `tail`.
struct RowGroups {
  int n, shift, head, tail;
  template <typename E>
  __device__ __forceinline__ RowGroups(const E* p, int width)
      : n(width), shift(static_cast<int>(reinterpret_cast<uintptr_t>(p) % 16 / sizeof(E))) {
    head = shift > 0 ? min(n, 8 - shift) : 0;
    tail = n > head ? n + shift & 7 : 0;
  }
  __device__ __forceinline__ bool full(int j) const { return j >= 0 && j + 8 <= n; }
  // The element outside full groups that a lane takes (lanes 0 to 7 the first ones, 32 to 39 the last ones),
  // or -1.
  __device__ __forceinline__ int edge(int lane) const {
    if (lane < head) return lane;
    return lane >= 32 && lane - 32 < tail ? n - tail + lane - 32 : -1;
  }
};

__device__ __forceinline__ void store8_loose(float* p, const float (&v)[8]) {
  typedef Raw<float>::loose_t loose_t;
  *reinterpret_cast<loose_t*>(p) = loose_t{v[0], v[1], v[2], v[3]};
  *reinterpret_cast<loose_t*>(p + 4) = loose_t{v[4], v[5], v[6], v[7]};
}
__device__ __forceinline__ void store8_loose(bf16_t* p, const float (&v)[8]) {
  Raw<bf16_t>::loose_t w;
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
  *reinterpret_cast<Raw<bf16_t>::loose_t*>(p) = w;
}

// How rows lie: kAligned, 16-byte aligned and of whole groups of eight; kLoose, at any element and of eight
// elements or more; kSingle, narrower.
enum Layout { kSingle, kLoose, kAligned };

// The eight elements that lane t of T holds of group g of a row: (g T + t) 8 .. + 7, 16 bytes (two times 16
// in fp32) a load.  Where a loose row ends inside them a lane holds the row's last eight, of which those
// that its neighbour has too (the first `skip`) count as 0 and are not stored.  kSingle: elements (8 g + i) T + t.
// (16384 rows of 2047 in bf16 through the norms, forward and backward: 154 us, an element at a time 222.)
template <int T, Layout LAYOUT>
struct RowGroup {
  __device__ __forceinline__ static int column(int g, int t, int i) {
    return LAYOUT == kSingle ? (8 * g + i) * T + t : (g * T + t) * 8 + i;
  }
  __device__ __forceinline__ static int skip(int g, int t, int d) { return max(column(g, t, 0) - (d - 8), 0); }
  template <typename E>
  __device__ __forceinline__ static void load(const E* row, int g, int t, int d, float (&v)[8]) {
    if (LAYOUT == kAligned) {
      if (column(g, t, 0) < d) {
        load8(row + column(g, t, 0), v);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = 0.0f;
      }
    } else if (LAYOUT == kLoose) {
      Raw<E> raw;
      raw.load_loose(row + min(column(g, t, 0), d - 8));
      raw.get(v);
      const int none = skip(g, t, d);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = i >= none ? v[i] : 0.0f;
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = column(g, t, i) < d ? load1(row + column(g, t, i)) : 0.0f;
    }
  }
  template <typename E>
  __device__ __forceinline__ static void store(E* row, int g, int t, int d, const float (&v)[8]) {
    if (LAYOUT == kAligned) {
      if (column(g, t, 0) < d) store8(row + column(g, t, 0), v);
    } else if (LAYOUT == kLoose) {
      const int none = skip(g, t, d);
      if (none == 0) {
        store8_loose(row + column(g, t, 0), v);
      } else if (none < 8) {
#pragma unroll
        for (int i = 1; i < 8; ++i)
          if (i >= none) store1(row + d - 8 + i, v[i]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (column(g, t, i) < d) store1(row + column(g, t, i), v[i]);
    }
  }
};

// v of the lane that a DPP control names; `none` where there is none or the row is masked out.
template <int CONTROL, int ROWS>
__device__ __forceinline__ float from_lane(float v, float none) {
  return __uint_as_float(__builtin_amdgcn_update_dpp(__float_as_uint(none), __float_as_uint(v), CONTROL, ROWS, 0xf, false));
}
__device__ __forceinline__ float last_lane(float v) {
  return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), 63));
}

// Over a wave's lanes, in a fixed order: shifts by 1, 2, 4, 8 within rows of 16 lanes, a row's last lane
// to the next row, lane 31 to the upper half, and lane 63, which then has all, to every lane.  (In registers:
// a shuffle through LDS takes some hundred cycles a step.)
__device__ __forceinline__ float wave_sum(float v) {
  v += from_lane<0x111, 0xf>(v, 0.0f);
  v += from_lane<0x112, 0xf>(v, 0.0f);
  v += from_lane<0x114, 0xf>(v, 0.0f);
  v += from_lane<0x118, 0xf>(v, 0.0f);
  v += from_lane<0x142, 0xa>(v, 0.0f);
  v += from_lane<0x143, 0xc>(v, 0.0f);
  return last_lane(v);
}
__device__ __forceinline__ float wave_max(float v) {
  const float none = -__builtin_inff();
  v = fmaxf(v, from_lane<0x111, 0xf>(v, none));
  v = fmaxf(v, from_lane<0x112, 0xf>(v, none));
  v = fmaxf(v, from_lane<0x114, 0xf>(v, none));
  v = fmaxf(v, from_lane<0x118, 0xf>(v, none));
  v = fmaxf(v, from_lane<0x142, 0xa>(v, none));
  v = fmaxf(v, from_lane<0x143, 0xc>(v, none));
  return last_lane(v);
}

// Sum over the T lanes that share a row.  tmp: T / 64 floats of LDS that no wave still
// reads from an earlier sum (callers alternate between two).
template <int T>
__device__ __forceinline__ float row_sum(float v, float* tmp, int t) {
  if (T < 64) {   // rows of 8, 16 or 32 lanes: neighbours, pairs, and mirrors of 8 and 16, which give all lanes the same
    v += from_lane<0xb1, 0xf>(v, 0.0f);
    v += from_lane<0x4e, 0xf>(v, 0.0f);
    v += from_lane<0x141, 0xf>(v, 0.0f);
    if (T >= 16) v += from_lane<0x140, 0xf>(v, 0.0f);
    if (T == 32) v += __shfl_xor(v, 16, 64);
    return v;
  }
  v = wave_sum(v);
  if (T == 64) return v;
  if ((t & 63) == 0) tmp[t >> 6] = v;
  __syncthreads();
  float s = tmp[0];
#pragma unroll
  for (int i = 1; i < T / 64; ++i) s += tmp[i];
  return s;
}

}  // namespace staple
