// LDS tiles of the attention kernels and the matrix products over them.
//
// A tile holds rows (tokens) of one head, DP elements each (head_dim rounded
// up to 64 or 128; the rest is zeros), as they lie in memory.  Every product
// of the forward and backward pass puts a tile on the MFMA's A side (32 rows
// of v_mfma_f32_32x32x16_bf16, or of v_mfma_f32_32x32x2_f32) and keeps the B
// side in registers, one query (or key) a column:
//   - by rows:    A = 32 tile rows, contracted over head_dim;
//   - transposed: A = 32 head elements, contracted over the tile's rows.
// The result of the first kind has tile row 8 (r / 4) + 4 h + r % 4 of column
// c in register r of lane c + 32 h, which is the B operand of the second kind
// as it stands once the contraction visits the rows in that order: no score
// ever moves between lanes.
//
// 16-byte chunks of a row are XORed with a function of the row so that both
// kinds of read spread over the LDS banks: 16 consecutive rows at one chunk
// (16-byte reads) fall on 16 different chunks, and the two-chunk pieces that
// 4 consecutive rows give a transposing read fall on different banks.
#pragma once

#include "attn.h"
#include "lds_load.h"

namespace staple {

typedef short v4s_t __attribute__((ext_vector_type(4)));
typedef short v8s_t __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) v4s_t lds_v4s_t;
typedef __attribute__((address_space(3))) u32x4_t lds_u32x4;
typedef __attribute__((address_space(3))) float lds_f32;
typedef __attribute__((address_space(3))) f32x4_t lds_f32x4;

template <typename T, int DP>
struct Tile {
  static constexpr int kRow = DP * static_cast<int>(sizeof(T));   // bytes per row
  static constexpr int kChunks = kRow / 16;
  static constexpr int kSteps = kRow / 32;                        // 16-byte A reads per lane and row block
  static constexpr int kDT = DP / 32;                             // 32-element blocks of head_dim

  __device__ __forceinline__ static int spread(int row) {
    if constexpr (kChunks >= 16) return ((row & 7) << 1) | ((row >> 3) & 1);
    else return (((row >> 1) & 3) << 1) | ((row >> 3) & 1);
  }
  // By rows: the lane's 16 bytes of row `row0 + lane % 32`, step s.
  __device__ __forceinline__ static u32x4_t row_frag(const lds_char* tile, int row0, int s) {
    const int lane = threadIdx.x & 63, row = row0 + (lane & 31);
    return *reinterpret_cast<const lds_u32x4*>(tile + row * kRow + (((2 * s + (lane >> 5)) ^ spread(row)) << 4));
  }
};

__device__ __forceinline__ f32x16_t mma16(const u32x4_t& a, const u32x4_t& b, f32x16_t acc, bf16_t) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b),
                                                 acc, 0, 0, 0);
}
__device__ __forceinline__ f32x16_t mma16(const u32x4_t& a, const u32x4_t& b, f32x16_t acc, float) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    acc = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(a[i]), __uint_as_float(b[i]), acc, 0, 0, 0);
  return acc;
}

// The B operand of the transposed products: 16 (bf16) or 8 (fp32) tile rows
// of one column block, from half (bf16) or a quarter (fp32) of a result.
template <typename T> struct Column;
template <> struct Column<bf16_t> {
  u32x4_t v[2];   // rows 0-15, rows 16-31 of the block, rounded to bf16
  // times a power of two
  __device__ __forceinline__ void scale(float f) {
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        v[t][i] = pack_bf16x2(__uint_as_float(v[t][i] << 16) * f, __uint_as_float(v[t][i] & 0xffff0000u) * f);
  }
};
template <> struct Column<float> {
  f32x16_t v;
  __device__ __forceinline__ void set(const f32x16_t& x) { v = x; }
};

// The lane's LDS addresses of a 32-row block's A operands by rows, one a step;
// move() takes them to another place of the ring, `block` is a constant offset.
template <typename T, int DP>
struct RowReader {
  using TL = Tile<T, DP>;
  const lds_char* at[TL::kSteps];
  __device__ __forceinline__ explicit RowReader(const lds_char* ring) {
    const int lane = threadIdx.x & 63, row = lane & 31;
#pragma unroll
    for (int s = 0; s < TL::kSteps; ++s) at[s] = ring + row * TL::kRow + (((2 * s + (lane >> 5)) ^ TL::spread(row)) << 4);
  }
  __device__ __forceinline__ void move(int bytes) {
#pragma unroll
    for (int s = 0; s < TL::kSteps; ++s) at[s] += bytes;
  }
  __device__ __forceinline__ u32x4_t read(int s, int block) const {
    return *reinterpret_cast<const lds_u32x4*>(at[s] + block);
  }
};
// The same transposed: rows [16 t, 16 t + 16) and head elements [32 dt, 32 dt +
// 32) of the block, the rows in the order of a Column.  16 lanes read 4 rows x
// 16 elements and get 4 rows of one element each; 8 rows on, the spread
// differs, 16 rows on it does not.
// kDT: element blocks the wave reads, from block dt0 on.
template <int DP, int kDT = DP / 32>
struct ColumnReader {
  using TL = Tile<bf16_t, DP>;
  const lds_char* at[kDT][2];
  __device__ __forceinline__ explicit ColumnReader(const lds_char* ring, int dt0 = 0) {
    const int lane = threadIdx.x & 63, i16 = lane & 15;
#pragma unroll
    for (int dt = 0; dt < kDT; ++dt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int c = (dt0 + dt) * 32 + (lane & 16) + 4 * (i16 & 3), row = 8 * e + 4 * (lane >> 5) + (i16 >> 2);
        at[dt][e] = ring + row * TL::kRow + (((c >> 3) ^ TL::spread(row)) << 4) + (c & 4) * 2;
      }
  }
  __device__ __forceinline__ void move(int bytes) {
#pragma unroll
    for (int dt = 0; dt < kDT; ++dt)
#pragma unroll
      for (int e = 0; e < 2; ++e) at[dt][e] += bytes;
  }
  __device__ __forceinline__ u32x4_t read(int t, int dt, int block) const {
    v4s_t part[2];
#pragma unroll
    for (int e = 0; e < 2; ++e)
      part[e] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s_t*)(at[dt][e] + block + 16 * t * TL::kRow));
    const v8s_t a = {part[0][0], part[0][1], part[0][2], part[0][3], part[1][0], part[1][1], part[1][2], part[1][3]};
    return __builtin_bit_cast(u32x4_t, a);
  }
};
template <int DP>
__device__ __forceinline__ u32x4_t column_frag(const lds_char* tile, int row0, int t, int dt) {
  return ColumnReader<DP>(tile + row0 * Tile<bf16_t, DP>::kRow).read(t, dt, 0);
}
// acc += (rows [row0, row0 + 32) of the tile, elements [32 dt, 32 dt + 32))^T x column.
template <int DP>
__device__ __forceinline__ f32x16_t mma_transposed(const lds_char* tile, int row0, int dt,
                                                   const Column<bf16_t>& col, f32x16_t acc) {
#pragma unroll
  for (int t = 0; t < 2; ++t) acc = mma16(column_frag<DP>(tile, row0, t, dt), col.v[t], acc, bf16_t{});
  return acc;
}
template <int DP>
__device__ __forceinline__ f32x16_t mma_transposed(const lds_char* tile, int row0, int dt,
                                                   const Column<float>& col, f32x16_t acc) {
  using TL = Tile<float, DP>;
  const int lane = threadIdx.x & 63;
  const int c = dt * 32 + (lane & 31);
#pragma unroll
  for (int r = 0; r < 16; ++r) {
    const int row = row0 + 8 * (r >> 2) + 4 * (lane >> 5) + (r & 3);
    const float v = *reinterpret_cast<const lds_f32*>(tile + row * TL::kRow + (((c >> 2) ^ TL::spread(row)) << 4) + (c & 3) * 4);
    acc = __builtin_amdgcn_mfma_f32_32x32x2f32(v, col.v[r], acc, 0, 0, 0);
  }
  return acc;
}

// Zeros read in place of rows past a sequence and elements past head_dim.
__device__ const uint4 g_attn_zeros[1] = {};

// Copies R-row tiles of one head from global memory straight into LDS, 16
// bytes a lane.  Instruction i of wave w fills 1 KB of the tile; the lane's
// source is the chunk that its LDS place holds.  Rows past the sequence and
// elements past head_dim come as zeros: they lie past the end of the head's
// buffer, which is laid over the rows that exist.  kWide: row strides so large
// that a buffer could span 2^31 bytes; 64-bit addresses then take its place.
template <typename T, int DP, int R, int NW, bool kWide>
struct TileLoader {
  using TL = Tile<T, DP>;
  static constexpr int kPer = R * TL::kRow / (1024 * NW);   // instructions per wave
  static constexpr int kRowStep = 1024 * NW / TL::kRow;     // rows between them
  static_assert(kPer * 1024 * NW == R * TL::kRow, "tile shape");
  const char* base;        // row 0 of the sequence, this head
  int64_t row_bytes;
  int n, dim_bytes;
  int row, place;          // the lane's row in instruction 0, and its 16-byte place in every row
  uint32_t offset[kPer];
  u32x4_t buffer;
  uint32_t lds0;           // this wave's first byte of a tile

  // wave: the caller's number among the NW waves that load the tile.
  __device__ __forceinline__ void init(const HeadsView& t, int64_t row0, int rows, int64_t head, int dim, int wave) {
    row_bytes = t.row_stride * static_cast<int64_t>(sizeof(T));
    n = rows;
    dim_bytes = dim * static_cast<int>(sizeof(T));
    const int at = wave * 1024 + (threadIdx.x & 63) * 16;
    lds0 = wave * 1024;
    row = at / TL::kRow;
    place = at % TL::kRow / 16;
    if constexpr (!kWide) {
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int x = byte_of(i);
        offset[i] = x < dim_bytes ? static_cast<uint32_t>(row + i * kRowStep) * static_cast<uint32_t>(row_bytes) + x : 0x80000000u;
      }
    }
    set_base(t.data + row0 * row_bytes + head * t.head_stride * static_cast<int64_t>(sizeof(T)));
  }
  __device__ __forceinline__ int byte_of(int i) const { return (place ^ TL::spread(row + i * kRowStep)) * 16; }
  __device__ __forceinline__ void set_base(const char* b) {
    base = b;
    if constexpr (!kWide)
      buffer = make_buffer(base, n > 0 ? static_cast<uint32_t>((n - 1) * row_bytes) + dim_bytes : 0u);
  }
  __device__ __forceinline__ void next_head(const HeadsView& t) {
    set_base(base + t.head_stride * static_cast<int64_t>(sizeof(T)));
  }
  // Rows [row0, row0 + R) of the sequence; row0 at most R past its end.
  __device__ __forceinline__ void load(int row0, lds_char* lds) const {
    lds_char* const to = lds + lds0;
    if constexpr (!kWide) {
      const uint32_t first = static_cast<uint32_t>(row0) * static_cast<uint32_t>(row_bytes);
      u32x4_t scalar;   // wherever the compiler keeps it, the load takes it from scalar registers
#pragma unroll
      for (int i = 0; i < 4; ++i) scalar[i] = __builtin_amdgcn_readfirstlane(buffer[i]);
#pragma unroll
      for (int i = 0; i < kPer; ++i) dma16(scalar, offset[i] + first, static_cast<lds_void*>(to + i * NW * 1024));
    } else {
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int r = row0 + row + i * kRowStep;
        const int x = byte_of(i);
        dma16(r < n && x < dim_bytes ? static_cast<const void*>(base + r * row_bytes + x)
                                     : static_cast<const void*>(g_attn_zeros),
              static_cast<lds_void*>(to + i * NW * 1024));
      }
    }
  }
};

// The lane's 16 bytes of step s of row `row` (zeros where !in or past dim).
template <typename T>
__device__ __forceinline__ u32x4_t load_frag(const HeadsView& t, int64_t row, int64_t head, int dim, int s, bool in) {
  constexpr int kVec = 16 / static_cast<int>(sizeof(T));
  const int e = (2 * s + ((threadIdx.x & 63) >> 5)) * kVec;
  if (!in || e >= dim) return u32x4_t{0, 0, 0, 0};
  return *reinterpret_cast<const u32x4_t*>(t.data + (row * t.row_stride + head * t.head_stride + e) * static_cast<int64_t>(sizeof(T)));
}
// Sum of the products of two such pieces.
__device__ __forceinline__ float dot_frag(const u32x4_t& a, const u32x4_t& b, bf16_t) {
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    s += __uint_as_float(a[i] << 16) * __uint_as_float(b[i] << 16);
    s += __uint_as_float(a[i] & 0xffff0000u) * __uint_as_float(b[i] & 0xffff0000u);
  }
  return s;
}
__device__ __forceinline__ float dot_frag(const u32x4_t& a, const u32x4_t& b, float) {
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) s += __uint_as_float(a[i]) * __uint_as_float(b[i]);
  return s;
}
// The operand negated (sign bits flipped, exactly).
template <typename T>
__device__ __forceinline__ u32x4_t flip_sign(u32x4_t v) {
  const uint32_t m = sizeof(T) == 2 ? 0x80008000u : 0x80000000u;
  return v ^ u32x4_t{m, m, m, m};
}

// Keeps a value's computation where it stands in the program, between the
// products around it, instead of where it is used.
__device__ __forceinline__ void pin(uint32_t& v) { asm volatile("" : "+v"(v)); }

// The other half-wave's value of the same column.
__device__ __forceinline__ float other_half(float x) { return __shfl_xor(x, 32); }

// Stores a transposed result's column (head elements 32 dt + 8 (r / 4) + 4 h +
// r % 4 of one row) times `mul` as 16-byte pieces: the half-waves trade 4-element
// groups first, so that each lane holds 8 consecutive elements (fp32: 4).
template <typename T>
__device__ __forceinline__ void store_column(const HeadsView& t, int64_t row, int64_t head, int dim, int dt,
                                             const f32x16_t& x, float mul, bool in);
template <>
__device__ __forceinline__ void store_column<bf16_t>(const HeadsView& t, int64_t row, int64_t head, int dim, int dt,
                                                     const f32x16_t& x, float mul, bool in) {
  const int h = (threadIdx.x & 63) >> 5;
  char* p = t.data + (row * t.row_stride + head * t.head_stride) * 2;
#pragma unroll
  for (int g = 0; g < 2; ++g) {
    uint32_t a[2], b[2];   // groups 2 g and 2 g + 1
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      a[i] = pack_bf16x2(x[8 * g + 2 * i] * mul, x[8 * g + 2 * i + 1] * mul);
      b[i] = pack_bf16x2(x[8 * g + 4 + 2 * i] * mul, x[8 * g + 4 + 2 * i + 1] * mul);
    }
    // lower lanes keep group 2 g and take the upper lanes' half of it
    const uint32_t s0 = h ? a[0] : b[0], s1 = h ? a[1] : b[1];
    const uint32_t o0 = __shfl_xor(s0, 32), o1 = __shfl_xor(s1, 32);
    const u32x4_t v = h ? u32x4_t{o0, o1, b[0], b[1]} : u32x4_t{a[0], a[1], o0, o1};
    const int e = dt * 32 + 16 * g + 8 * h;
    if (in && e < dim) *reinterpret_cast<u32x4_t*>(p + e * 2) = v;
  }
}
template <>
__device__ __forceinline__ void store_column<float>(const HeadsView& t, int64_t row, int64_t head, int dim, int dt,
                                                    const f32x16_t& x, float mul, bool in) {
  const int h = (threadIdx.x & 63) >> 5;
  char* p = t.data + (row * t.row_stride + head * t.head_stride) * 4;
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    const int e = dt * 32 + 8 * g + 4 * h;
    if (in && e < dim)
      *reinterpret_cast<f32x4_t*>(p + e * 4) = f32x4_t{x[4 * g] * mul, x[4 * g + 1] * mul, x[4 * g + 2] * mul, x[4 * g + 3] * mul};
  }
}

}  // namespace staple
