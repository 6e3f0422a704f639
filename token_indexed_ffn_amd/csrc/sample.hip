// Sampling of a row's token from given random numbers, with temperature, top-k, top-p and min-p.
//
// The weights are whole numbers: w_j = round(unit exp((l_j - max l) / T)), from an exponential in
// 64 bits, with unit a power of two: 2^62 by the number of logits, at most 2^50 (2^45 for 100352).
// Their sums are exact in 64-bit integers, so that no order of adding, and no atomic one, changes a
// token, and a sum is off by half a unit's inverse a logit at most, where sums in 32 bits would be
// off by some 1e-7.
#include "model_ops.h"
#include "row_io.h"

namespace staple {

constexpr int kSampleThreads = 1024;
typedef unsigned long long u64;

// Order of the logits: larger logits have larger keys; NaN counts as -inf, -0 as 0.
__device__ __forceinline__ uint32_t key_of(float l) {
  if (!(l == l)) l = -__builtin_inff();
  const uint32_t b = __float_as_uint(l + 0.0f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float logit_of(uint32_t key) {
  return __uint_as_float(key & 0x80000000u ? key & 0x7fffffffu : ~key);
}

// The weights of a row.
struct Weights {
  uint32_t top;   // key of the largest logit
  double rate;    // 1 / T
  double unit;
  __device__ __forceinline__ u64 operator()(uint32_t key) const {
    if (key == top) return static_cast<u64>(unit);
    const double l = logit_of(key), m = logit_of(top);
    if (l == -__builtin_inf() || m == __builtin_inf()) return 0;
    return static_cast<u64>(rint(exp((l - m) * rate) * unit));
  }
};

// The whole part of share total, and whether there is a rest: exact, so that sums of equal weights
// that meet a border are told from those that pass it.  share is in [0, 1).
__device__ __forceinline__ u64 part_of(float share, u64 total, bool& rest) {
  int e;
  const float m = frexpf(share, &e);                                // share = m 2^e, e <= 0
  const auto x = static_cast<unsigned __int128>(total) * static_cast<uint32_t>(m * 16777216.0f);
  const int shift = 24 - e;                                         // of a product below 2^87
  if (shift >= 88) {
    rest = x != 0;
    return 0;
  }
  const auto whole = x >> shift;
  rest = (whole << shift) != x;
  return static_cast<u64>(whole);
}

struct RowSums {
  u64 wave[kSampleThreads / 64];
  uint32_t key[kSampleThreads / 64];
  u64 weights[256];
  uint32_t counts[256];
  u64 found[4];
};

__device__ __forceinline__ u64 sum_all(u64 v, RowSums& s) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o, 64);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) s.wave[threadIdx.x >> 6] = v;
  __syncthreads();
  u64 r = 0;
  for (int i = 0; i < kSampleThreads / 64; ++i) r += s.wave[i];
  return r;
}

// Sum over the lanes before this one, and over all.
__device__ __forceinline__ u64 sum_before(u64 v, RowSums& s, u64& total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  u64 x = v;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const u64 y = __shfl_up(x, o, 64);
    if (lane >= o) x += y;
  }
  __syncthreads();
  if (lane == 63) s.wave[wave] = x;
  __syncthreads();
  u64 before = 0;
  total = 0;
  for (int i = 0; i < kSampleThreads / 64; ++i) {
    if (i < wave) before += s.wave[i];
    total += s.wave[i];
  }
  return before + x - v;
}

// The kept tokens: keys above `key`, and of those equal to it the first `ties` in the row.
struct Cut {
  uint32_t key;
  uint32_t ties;
};

// In the order of falling keys, ties by rising index, the shortest run of tokens whose counts
// (BY_COUNT) or weights reach `want` (at least 1), found digit by digit of the key.
template <typename E, bool BY_COUNT>
__device__ Cut find_cut(const E* l, int n, const Weights& weight, u64 want, RowSums& s) {
  uint32_t prefix = 0;
  uint32_t ties = 0;
  for (int shift = 24; shift >= 0; shift -= 8) {
    __syncthreads();
    for (int b = threadIdx.x; b < 256; b += kSampleThreads) {
      s.counts[b] = 0;
      s.weights[b] = 0;
    }
    __syncthreads();
    for (int j = threadIdx.x; j < n; j += kSampleThreads) {
      const uint32_t key = key_of(load1(l + j));
      if (shift < 24 && (key >> (shift + 8)) != (prefix >> (shift + 8))) continue;
      const int b = (key >> shift) & 255;
      atomicAdd(&s.counts[b], 1u);
      if (!BY_COUNT) atomicAdd(&s.weights[b], weight(key));
    }
    __syncthreads();
    if (threadIdx.x == 0) {
      u64 left = want;
      int b = 255, last = 255;
      for (; b >= 0; --b) {
        if (s.counts[b] == 0) continue;
        last = b;
        const u64 here = BY_COUNT ? s.counts[b] : s.weights[b];
        if (here >= left) break;
        left -= here;
      }
      if (b < 0) {   // all of them: the last one is reached
        b = last;
        left += BY_COUNT ? s.counts[b] : s.weights[b];
      }
      s.found[0] = b;
      s.found[1] = left;
      s.found[2] = s.counts[b];
    }
    __syncthreads();
    prefix |= static_cast<uint32_t>(s.found[0]) << shift;
    want = s.found[1];
    ties = static_cast<uint32_t>(s.found[2]);
  }
  // `want` is left to the tokens with this key
  if (BY_COUNT) return Cut{prefix, static_cast<uint32_t>(want < ties ? want : ties)};
  const u64 w = weight(prefix);
  const u64 need = w == 0 ? 1 : (want + w - 1) / w;
  return Cut{prefix, static_cast<uint32_t>(need < ties ? (need > 0 ? need : 1) : ties)};
}

// Sum of the kept weights.
template <typename E>
__device__ u64 kept_sum(const E* l, int n, const Weights& weight, Cut cut, RowSums& s) {
  u64 w = 0;
  for (int j = threadIdx.x; j < n; j += kSampleThreads) {
    const uint32_t key = key_of(load1(l + j));
    if (key > cut.key) w += weight(key);
  }
  return sum_all(w, s) + cut.ties * weight(cut.key);
}

template <typename E>
__global__ __launch_bounds__(kSampleThreads) void sample_kernel(SampleView a) {
  __shared__ RowSums s;
  const int64_t row = blockIdx.x;
  const E* l = reinterpret_cast<const E*>(a.logits) + row * a.stride;
  const int n = a.vocab;
  // the largest logit, and the first place of it
  u64 best = 0;
  for (int j = threadIdx.x; j < n; j += kSampleThreads) {
    const u64 x = static_cast<u64>(key_of(load1(l + j))) << 32 | (0xffffffffu - static_cast<uint32_t>(j));
    best = x > best ? x : best;
  }
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) {
    const u64 x = __shfl_xor(best, o, 64);
    best = x > best ? x : best;
  }
  if ((threadIdx.x & 63) == 0) s.wave[threadIdx.x >> 6] = best;
  __syncthreads();
  for (int i = 0; i < kSampleThreads / 64; ++i) best = s.wave[i] > best ? s.wave[i] : best;
  const uint32_t top = static_cast<uint32_t>(best >> 32);
  const float t = a.temperature ? a.temperature[row] : 1.0f;
  const bool empty = logit_of(top) == -__builtin_inff();
  if (empty || !(t > 0.0f)) {
    if (threadIdx.x == 0) {
      a.token[row] = empty ? -1 : static_cast<int32_t>(0xffffffffu - static_cast<uint32_t>(best));
      if (a.logprob) a.logprob[row] = empty ? -__builtin_inff() : 0.0f;
    }
    return;
  }
  const int bits = 62 - (32 - __clz(n));
  const Weights weight{top, 1.0 / static_cast<double>(t), static_cast<double>(u64(1) << (bits < 50 ? bits : 50))};
  Cut cut{0u, 0u};   // nothing has the key 0: all are kept
  const int k = a.top_k ? a.top_k[row] : 0;
  if (k > 0 && k < n) cut = find_cut<E, true>(l, n, weight, k, s);
  u64 total = kept_sum(l, n, weight, cut, s);
  const float p = a.top_p ? a.top_p[row] : 1.0f;
  if (p < 1.0f) {
    bool rest = false;
    u64 want = p > 0.0f ? part_of(p, total, rest) : 0;
    want += rest || want == 0;
    const Cut by_p = find_cut<E, false>(l, n, weight, want, s);
    if (by_p.key > cut.key || (by_p.key == cut.key && by_p.ties < cut.ties)) cut = by_p;
    total = kept_sum(l, n, weight, cut, s);
  }
  double least = a.min_p && a.min_p[row] > 0.0f ? static_cast<double>(a.min_p[row]) : 0.0;
  if (least > 1.0) least = 1.0;
  const u64 floor_w = static_cast<u64>(ceil(least * weight.unit));
  if (floor_w > 0) {
    u64 w = 0;
    for (int j = threadIdx.x; j < n; j += kSampleThreads) {
      const uint32_t key = key_of(load1(l + j));
      const u64 x = key > cut.key ? weight(key) : 0;
      if (x >= floor_w) w += x;
    }
    const u64 tie = weight(cut.key);
    total = sum_all(w, s) + (cut.ties > 0 && tie >= floor_w ? cut.ties * tie : 0);
  }
  // the first token at which the sum passes u total
  const float u = a.u[row];
  bool rest;
  const u64 target = !(u > 0.0f) ? 0 : u < 1.0f ? part_of(u, total, rest) : total - 1;
  u64 before = 0;
  uint32_t ties = 0;
  for (int j0 = 0; j0 < n; j0 += kSampleThreads) {
    const int j = j0 + threadIdx.x;
    const uint32_t key = j < n ? key_of(load1(l + j)) : 0u;
    u64 tied_here;
    const bool tied = j < n && key == cut.key;
    const uint32_t rank = ties + static_cast<uint32_t>(sum_before(tied, s, tied_here));
    ties += static_cast<uint32_t>(tied_here);
    u64 w = 0;
    if (j < n && (key > cut.key || (tied && rank < cut.ties))) w = weight(key);
    if (w < floor_w) w = 0;
    u64 here;
    const u64 mine = before + sum_before(w, s, here);
    if (w > 0 && mine <= target && target < mine + w) {
      a.token[row] = j;
      if (a.logprob) {
        const double d = key == top ? 0.0 : (static_cast<double>(logit_of(key)) - logit_of(top)) * weight.rate;
        a.logprob[row] = static_cast<float>(d - log(static_cast<double>(total) / weight.unit));
      }
    }
    before += here;
    if (before > target) break;
  }
}

size_t sample_workspace_bytes(int64_t, int64_t) { return 0; }

hipError_t launch_sample(const SampleView& v, int32_t dtype, void*, hipStream_t s) {
  const dim3 grid(static_cast<unsigned>(v.n_rows)), threads(kSampleThreads);
  if (dtype == STAPLE_BF16) sample_kernel<bf16_t><<<grid, threads, 0, s>>>(v);
  else sample_kernel<float><<<grid, threads, 0, s>>>(v);
  return hipGetLastError();
}

}  // namespace staple
