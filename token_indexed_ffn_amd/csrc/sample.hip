// Sampling of a row's token from given random numbers, with temperature, top-k, top-p and min-p.
//
// The weights are whole numbers: w_j = round(unit exp((l_j - max l) / T)), from an exponential in
// 64 bits, with unit a power of two: 2^62 by the number of logits, at most 2^50 (2^45 for 100352).
// Their sums are exact in 64-bit integers, so that no order of adding, and no atomic one, changes a
// token.  A weight is off by half a unit's inverse from its rounding, by 2^-48 of itself from the exponential's
// terms, and by |ln w| 2^-51 of itself from its argument, which is rounded four times: by 2^-47 of itself and one unit's
// inverse in all, where sums in 32 bits would be off by some 1e-7.
//
// The kept tokens are a first part of the order of falling logits (ties: rising index), so one
// pass finds the largest logit, a second one counts and weighs the tokens in kBins intervals of
// the logit, which tells the interval that the cut falls into, and a third one lists that
// interval's tokens and sums the weights above it, by blocks of the row.  The list gives the
// cut, the blocks' sums the block of the drawn token.  Without top-k and top-p the second pass sums the
// blocks and the third is not needed.  A long row among few is dealt out to several workgroups, a launch for each
// pass, and the last of them to arrive goes on with the row; otherwise a workgroup takes a row through
// all passes.
//
// What bounds it: of one row of 100352, whose bytes are nothing, latency: three launches of 5, 8 and 15 us,
// in which a wave has three or four steps of some 0.6 us, and the row's last workgroup sorts, sums and draws
// alone.  64 such rows in fp32: 10 us for the read, 17 and 23 for the others (26 MB, 5 us at a copy's
// rate).  509 rows of 50021 in bf16 with a temperature alone: 39 us, of which the 64-bit exponentials are some 15.
#include "model_ops.h"
#include "row_io.h"

namespace staple {

typedef unsigned long long u64;

constexpr int kSampleThreads = 256;
constexpr int kWaves = kSampleThreads / 64;
constexpr int kBins = 512;          // two a lane of four waves
constexpr int kList = 2048;         // listed tokens
constexpr int kMostBlocks = 2049;   // blocks of a row: 512 elements each, 1024 or 2048 past 2^20 logits
constexpr int kMostChunks = 16;     // workgroups of a row: the last one has all intervals' loads in flight at once

// --------------------------------------------------------------------------- logits and weights
// NaN as -inf, +inf as the largest finite number.
__device__ __forceinline__ float plain(float l) { return fminf(fmaxf(l, -__builtin_inff()), 3.402823466e38f); }

// Order of the logits: larger logits have larger keys, -0 that of 0.
__device__ __forceinline__ uint32_t key_of(float l) {
  const uint32_t b = __float_as_uint(l + 0.0f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float logit_of(uint32_t key) {
  return __uint_as_float(key & 0x80000000u ? key & 0x7fffffffu : ~key);
}

// Order of a row's tokens: falling logits, ties by rising index.  No two are the same.
constexpr int kIndexBits = 22;
constexpr uint32_t kIndexMask = (1u << kIndexBits) - 1;
static_assert(kSampleMaxVocab <= int64_t(1) << kIndexBits, "an index fits");
__device__ __forceinline__ u64 place_of(float l, int j) {
  return static_cast<u64>(key_of(l)) << kIndexBits | (kIndexMask - static_cast<uint32_t>(j));
}
__device__ __forceinline__ float logit_at(u64 place) { return logit_of(static_cast<uint32_t>(place >> kIndexBits)); }
__device__ __forceinline__ int index_at(u64 place) {
  return static_cast<int>(kIndexMask - (static_cast<uint32_t>(place) & kIndexMask));
}

// 2^(i / 32), i < 32.
__device__ const double kSteps[32] = {
    1.0, 1.0218971486541166, 1.0442737824274138, 1.0671404006768237,
    1.0905077326652577, 1.1143867425958924, 1.1387886347566916, 1.1637248587775775,
    1.189207115002721, 1.215247359980469, 1.241857812073484, 1.2690509571917332,
    1.2968395546510096, 1.3252366431597413, 1.3542555469368927, 1.383909881963832,
    1.4142135623730951, 1.4451808069770467, 1.4768261459394993, 1.5091644275934228,
    1.5422108254079407, 1.5759808451078865, 1.6104903319492543, 1.645755478153965,
    1.681792830507429, 1.718619298122478, 1.7562521603732995, 1.7947090750031072,
    1.8340080864093424, 1.8741676341103, 1.9152065613971474, 1.9571441241754002,
};

// A row's weights.
struct Weights {
  double top;       // the largest logit
  double rate;      // 32 log2(e) / T
  double lowest;    // exponents from here on are rounded to a weight of 0
  int unit_log2;
  const double* step;
  __device__ __forceinline__ u64 unit() const { return u64(1) << unit_log2; }
  // 2^(y / 32) with y = n + r: the step of n's last five bits, its other bits added to the exponent, and
  // five terms of exp(r ln 2 / 32) (|r| <= 1/2: off by 2^-48).  Some 22 instructions, 14 of them in 64 bits.
  __device__ __forceinline__ u64 operator()(float l) const {
    const double far = fmax((static_cast<double>(l) - top) * rate, lowest);
    const double magic = 6755399441055744.0;   // 3 2^51: a sum with it is rounded to a whole number
    const double big = far + magic;
    const int n = static_cast<int>(__double_as_longlong(big));
    const double r = far - (big - magic);
    constexpr double c = 0.693147180559945309417 / 32;
    double p = c * c * c * c * c / 120;
    p = fma(p, r, c * c * c * c / 24);
    p = fma(p, r, c * c * c / 6);
    p = fma(p, r, c * c / 2);
    p = fma(p, r, c);
    p = fma(p, r, 1.0);
    const u64 bits = __double_as_longlong(p * step[n & 31]) + (static_cast<u64>((n >> 5) + unit_log2) << 52);
    return __double_as_longlong(__longlong_as_double(bits) + 4503599627370496.0) & ((u64(1) << 52) - 1);
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

// ------------------------------------------------------------------------------- a row's layout
// The row is cut into blocks of 2^log_size elements that begin where its memory is 16-byte aligned
// (`shift` elements before its first one); consecutive blocks make a workgroup's chunk.
struct SampleGrid {
  int chunks, blocks, blocks_a_chunk, log_size;
  int64_t row_bytes;
  __host__ __device__ int size() const { return 1 << log_size; }
};

enum { kDone, kListed, kSearch };   // the token is known; lo to hi are listed; too many for the list
struct Border {
  u64 total;             // of all weights
  u64 weight_before;     // of the tokens above interval `lo`
  uint32_t count_before;
  int lo, hi;            // intervals whose tokens are listed: the cut is among them
  int mode;
};

struct RowState {
  Border border;
  uint32_t arrived[2];
};

struct RowSpace {
  RowState* state;
  u64* best;        // [chunks]: place of the largest logit
  float* least;     // [chunks]: the smallest logit
  u64* sums;        // [blocks]: kept weights, those of listed tokens aside
  u64* list;        // [chunks][kList]: places
  uint32_t* listed; // [chunks]
  u64* weights;     // [chunks][kBins]
  uint32_t* counts; // [chunks][kBins]
  __host__ __device__ RowSpace(char* p, int64_t row, const SampleGrid& g) {
    p += row * g.row_bytes;
    state = reinterpret_cast<RowState*>(p);
    best = reinterpret_cast<u64*>(p + 64);
    sums = best + kMostChunks;
    list = sums + kMostBlocks + 7;
    weights = list + static_cast<int64_t>(g.chunks) * kList;
    counts = reinterpret_cast<uint32_t*>(weights + static_cast<int64_t>(g.chunks) * kBins);
    least = reinterpret_cast<float*>(counts + static_cast<int64_t>(g.chunks) * kBins);
    listed = reinterpret_cast<uint32_t*>(least + kMostChunks);
  }
};
static_assert(sizeof(RowState) <= 64, "before best");

template <typename E>
struct Row {
  const E* p;
  int n, shift;
  __device__ __forceinline__ Row(const SampleView& a, int64_t row)
      : p(reinterpret_cast<const E*>(a.logits) + row * a.stride), n(a.vocab),
        shift(static_cast<int>(reinterpret_cast<uintptr_t>(p) % 16 / sizeof(E))) {}
  __device__ __forceinline__ float at(int j) const { return plain(load1(p + j)); }
  // The elements outside full groups of eight are held one a lane (lanes 0 to 7 the row's first
  // ones, 32 to 39 its last ones), in the blocks that they belong to; -1: none.
  __device__ __forceinline__ bool has_edge(const SampleGrid& g, int block) const {
    return (block == 0 && shift > 0) || (block == n - 1 + shift >> g.log_size && (n + shift & 7) != 0);
  }
  __device__ __forceinline__ int edge(const SampleGrid& g, int block, int lane) const {
    const int head = shift > 0 ? min(n, 8 - shift) : 0, tail = n > head ? n + shift & 7 : 0;
    if (block == 0 && lane < head) return lane;
    if (block == n - 1 + shift >> g.log_size && lane >= 32 && lane - 32 < tail) return n - tail + lane - 32;
    return -1;
  }
};

// Blocks begin, begin + stride, ... of a row before `end`, eight elements a lane at a time, with the
// next kAhead loads in flight, from the walk's making on.  One copy of the body, and loops that are not
// unrolled, here and below: these kernels run for a few microseconds, and 60 KB of code took longer to
// fetch than to run.
constexpr int kAhead = 3;
template <typename E>
struct Walk {
  const Row<E>& r;
  const SampleGrid& g;
  int lane, begin, stride, steps, log_its;
  Raw<E> raw[kAhead];
  __device__ __forceinline__ Walk(const Row<E>& row, const SampleGrid& grid, int first_block, int end, int each)
      : r(row), g(grid), lane(threadIdx.x & 63), begin(first_block), stride(each) {
    log_its = g.log_size - 9;
    steps = begin < end ? (end - begin + stride - 1) / stride << log_its : 0;
#pragma unroll
    for (int i = 0; i < kAhead; ++i) load(i, raw[i]);
  }
  __device__ __forceinline__ int block(int s) const { return begin + (s >> log_its) * stride; }
  __device__ __forceinline__ int first(int s) const {
    return (block(s) << g.log_size) + (s & ((1 << log_its) - 1)) * 512 + lane * 8 - r.shift;
  }
  __device__ __forceinline__ void load(int s, Raw<E>& to) const {
    const int j = first(s);
    if (s < steps && j >= 0 && j + 8 <= r.n) to.load(r.p + j);
    else to.clear();
  }
  // f(j, v, full): elements from j on, -inf for those that there are not; full: there are all eight.
  // done(block): after a block's last ones.
  template <typename F, typename Done>
  __device__ __forceinline__ void run(F f, Done done) {
#pragma unroll 1
    for (int s = 0; s < steps; ++s) {
      float v[8];
      raw[0].get(v);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = plain(v[i]);
      int j = first(s);
      bool full = j >= 0 && j + 8 <= r.n;
#pragma unroll
      for (int i = 0; i + 1 < kAhead; ++i) raw[i] = raw[i + 1];
      load(s + kAhead, raw[kAhead - 1]);
      const bool last = (s + 1 & ((1 << log_its) - 1)) == 0;
      bool edge = last && r.has_edge(g, block(s));
#pragma unroll 1
      for (;;) {
        f(j, v, full);
        if (!edge) break;
        edge = false;
        full = false;
        j = r.edge(g, block(s), lane);
        v[0] = j >= 0 ? r.at(j) : -__builtin_inff();
#pragma unroll
        for (int i = 1; i < 8; ++i) v[i] = -__builtin_inff();
      }
      if (last) done(block(s));
    }
  }
};

// A wave's part of chunk c, of a workgroup of T lanes.
template <int T = kSampleThreads, typename E>
__device__ __forceinline__ Walk<E> walk_of(const Row<E>& r, const SampleGrid& g, int c) {
  return Walk<E>(r, g, c * g.blocks_a_chunk + (threadIdx.x >> 6), min((c + 1) * g.blocks_a_chunk, g.blocks), T / 64);
}

// A row's limits and weights, from its largest logit.
struct Limits {
  float top, temperature;
  int first;             // of the largest logits
  Weights weight;
  u64 least_weight;      // of min-p
  int k;                 // 0: no limit
  float p;               // 1: no limit
  float bin_rate;
  bool greedy, empty;
  // Interval of a logit, rising as it falls.
  __device__ __forceinline__ int bin(float l) const {
    return l == top ? 0 : static_cast<int>(fminf((top - l) * bin_rate, kBins - 1));
  }
};

// A row's arguments.  Every load before the first use, none behind a branch: u stands in for what is not given.
struct Arguments {
  float temperature, p, low;
  int k;
  double step;
  __device__ __forceinline__ Arguments(const SampleView& a, int64_t row) {
    step = kSteps[threadIdx.x & 31];
    temperature = (a.temperature ? a.temperature : a.u)[row];
    p = (a.top_p ? a.top_p : a.u)[row];
    low = (a.min_p ? a.min_p : a.u)[row];
    k = (a.top_k ? a.top_k : reinterpret_cast<const int32_t*>(a.u))[row];
  }
};

// best: the place of the largest logit; least: the smallest logit, or one that is near it.
__device__ __forceinline__ Limits limits_of(const SampleView& a, const Arguments& given, u64 best, float least, double* step) {
  Limits m;
  m.top = logit_at(best);
  m.first = index_at(best);
  m.empty = m.top == -__builtin_inff();
  m.temperature = a.temperature ? given.temperature : 1.0f;
  m.greedy = !(m.temperature > 0.0f);
  const int bits = 62 - (32 - __clz(a.vocab));
  const int unit = bits < 50 ? bits : 50;
  m.weight = Weights{m.top, 46.1662413084468290355 / static_cast<double>(m.temperature), -32.0 * (unit + 2), unit, step};
  const int k = a.top_k ? given.k : 0;
  m.k = k > 0 && k < a.vocab ? k : 0;
  const float p = a.top_p ? given.p : 1.0f;
  m.p = p < 1.0f ? fmaxf(p, 0.0f) : 1.0f;
  const float low = a.min_p ? given.low : 0.0f;
  m.least_weight = low > 0.0f ? static_cast<u64>(ceil(static_cast<double>(fminf(low, 1.0f)) * m.weight.unit())) : 0;
  // Weights past this distance are rounded to zero.  With top-p alone also: all weights below
  // (1 - p) / vocab, of the largest one, make less than 1 - p of the whole, so that the cut lies above them.
  float reach = 0.6932f * (m.weight.unit_log2 + 2);
  if (m.k == 0 && m.p < 1.0f) reach = fminf(reach, logf(static_cast<float>(a.vocab) / (1.0f - m.p)) + 0.01f);
  reach = fminf(m.temperature * reach, m.top - least);
  m.bin_rate = reach > 0.0f ? kBins / reach : 0.0f;
  if (threadIdx.x < 32) step[threadIdx.x] = given.step;
  __syncthreads();
  return m;
}

__device__ __forceinline__ Limits limits_of(const SampleView& a, int64_t row, const SampleGrid& g, const RowSpace& s,
                                            double* step) {
  const Arguments given(a, row);
  u64 best = 0;
  float least = __builtin_inff();
  const int lane = threadIdx.x & 63;
  if (lane < g.chunks) {
    best = s.best[lane];
    least = s.least[lane];
  }
  static_assert(kMostChunks <= 16, "one row of lanes");
#pragma unroll
  for (int o = 8; o >= 1; o >>= 1) {
    const u64 x = __shfl_xor(best, o, 64);
    best = x > best ? x : best;
    least = fminf(least, __shfl_xor(least, o, 64));
  }
  best = __shfl(best, 0, 64);
  least = __shfl(least, 0, 64);
  return limits_of(a, given, best, least, step);
}

// ------------------------------------------------------------------------------ workgroup sums
// v of the lane that a DPP control names, 0 where there is none or the row is masked out.
template <int CONTROL, int ROWS>
__device__ __forceinline__ u64 from_lane(u64 v) {
  const uint32_t lo = __builtin_amdgcn_update_dpp(0, static_cast<int>(v), CONTROL, ROWS, 0xf, false);
  const uint32_t hi = __builtin_amdgcn_update_dpp(0, static_cast<int>(v >> 32), CONTROL, ROWS, 0xf, false);
  return static_cast<u64>(hi) << 32 | lo;
}

// Sum over a wave's lanes up to this one: shifts by 1, 2, 4, 8 within rows of 16 lanes, then a row's
// last lane to the next row, and lane 31 to the upper half.  (In registers: a shuffle through LDS takes some
// hundred cycles a step.)
__device__ __forceinline__ u64 sum_up_to(u64 v) {
  v += from_lane<0x111, 0xf>(v);
  v += from_lane<0x112, 0xf>(v);
  v += from_lane<0x114, 0xf>(v);
  v += from_lane<0x118, 0xf>(v);
  v += from_lane<0x142, 0xa>(v);
  v += from_lane<0x143, 0xc>(v);
  return v;
}
// Lane 63 has the wave's sum.

// Sum over the lanes before this one, of W waves; total over all.
template <int W = kWaves>
__device__ __forceinline__ u64 sum_before(u64 v, u64* wave_sums, u64& total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const u64 x = sum_up_to(v);
  __syncthreads();
  if (lane == 63) wave_sums[wave] = x;
  __syncthreads();
  u64 before = 0;
  total = 0;
#pragma unroll
  for (int i = 0; i < W; ++i) {
    if (i < wave) before += wave_sums[i];
    total += wave_sums[i];
  }
  return before + x - v;
}

// What workgroups of a row tell each other in one launch goes past the caches of an XCD: written and
// read with relaxed atomic accesses of the device's scope.  (Fences of that scope write back and drop a
// whole L2: a fence in every workgroup made each of the two passes over 64 rows take
// 110 us in place of 25.)
template <typename T>
__device__ __forceinline__ void tell(T* p, T v) {
  __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
template <typename T>
__device__ __forceinline__ T told(const T* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// Whether this workgroup is the last of its row's to get here: what the others told is there then.
__device__ __forceinline__ bool last_of_row(uint32_t* arrived, int chunks, uint32_t* shared) {
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
  wait_vmcnt<0>();   // this wave's stores have reached the device's memory
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
  __syncthreads();
  if (chunks == 1) return true;
  if (threadIdx.x == 0) *shared = __hip_atomic_fetch_add(arrived, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  __syncthreads();
  return *shared == static_cast<uint32_t>(chunks - 1);
}

constexpr int kRowThreads = 512;   // of a workgroup that has a row to itself
struct Shared {
  double step[32];
  u64 wave[kRowThreads / 64];
  u64 found[4];
  uint32_t arrived, listed;
};

// ------------------------------------------------------------------------------------- the draw
// The token at which the sum of the kept weights passes u times their total.  sum(b): of block
// b; kept(l, j): whether token j, with its weight not below min-p, is kept.
template <typename E, int T = kSampleThreads, typename Sum, typename Kept>
__device__ __forceinline__ void draw(const SampleView& a, int64_t row, const SampleGrid& g, const Limits& m, Shared& s, Sum sum, Kept kept) {
  const Row<E> r(a, row);
  const int each = (g.blocks + T - 1) / T;   // consecutive blocks a lane
  const int b0 = threadIdx.x * each, b1 = min(b0 + each, g.blocks);
  u64 all = 0;
  for (int b = b0; b < b1; ++b) all += sum(b);
  u64 total;
  u64 before = sum_before<T / 64>(all, s.wave, total);
  const float u = a.u[row];
  bool rest;
  const u64 target = !(u > 0.0f) ? 0 : u < 1.0f ? part_of(u, total, rest) : total - 1;
  if (before <= target && target < before + all)
    for (int b = b0; b < b1; ++b) {
      const u64 here = sum(b);
      if (target < before + here) {
        s.found[0] = b;
        s.found[1] = before;
        break;
      }
      before += here;
    }
  __syncthreads();
  const int block = static_cast<int>(s.found[0]);
  before = s.found[1];
#pragma unroll 1
  for (int i = threadIdx.x; i < g.size(); i += T) {
    const int j = (block << g.log_size) - r.shift + i;
    u64 w = 0;
    float l = 0.0f;
    if (j >= 0 && j < r.n) {
      l = r.at(j);
      w = m.weight(l);
      if (w < m.least_weight || !kept(l, j)) w = 0;
    }
    u64 here;
    const u64 mine_before = before + sum_before<T / 64>(w, s.wave, here);
    if (w > 0 && mine_before <= target && target < mine_before + w) {
      a.token[row] = j;
      if (a.logprob) {
        const double d = l == m.top ? 0.0 : (static_cast<double>(l) - m.top) / static_cast<double>(m.temperature);
        a.logprob[row] = static_cast<float>(d - log(static_cast<double>(total) / static_cast<double>(m.weight.unit())));
      }
    }
    before += here;
    if (before > target) break;
  }
}

// -------------------------------------------------------------------------------------- pass one
struct Top {
  u64 place;     // of the largest logit
  float least;   // the smallest logit of full groups
};

// Of a workgroup's part of a row; lane 0 of the workgroup has it, or (ALL) every lane.
template <int T, bool ALL, typename E>
__device__ __forceinline__ Top find_top(const Row<E>& r, Walk<E> walk, u64* place_of_wave, float* least_of_wave) {
  // a lane's largest logit and its group, later the group's first element that has it
  float best = -__builtin_inff(), least = __builtin_inff();
  int at = 0;
  walk.run([&](int j, const float (&v)[8], bool full) {
    float top = v[0], low = v[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) {
      top = fmaxf(top, v[i]);
      low = fminf(low, v[i]);
    }
    if (full) least = fminf(least, low);
    // a row's first elements come after the rest of its first block
    if (top > best || (top == best && j < at)) {
      best = top;
      at = j;
    }
  }, [](int) {});
  int first = 0;   // a row of -inf has no token: any will do
  if (best != -__builtin_inff()) {
    float v[8];   // all loads before the first comparison: none behind a branch
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = r.at(min(max(at + i, 0), r.n - 1));
#pragma unroll
    for (int i = 7; i >= 0; --i)
      if (v[i] == best) first = min(max(at + i, 0), r.n - 1);
  }
  Top x{place_of(best, first), least};
  const auto join = [&](u64 place, float low) {
    x.place = place > x.place ? place : x.place;
    x.least = fminf(x.least, low);
  };
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) join(__shfl_xor(x.place, o, 64), __shfl_xor(x.least, o, 64));
  if ((threadIdx.x & 63) == 0) {
    place_of_wave[threadIdx.x >> 6] = x.place;
    least_of_wave[threadIdx.x >> 6] = x.least;
  }
  __syncthreads();
  if (ALL || threadIdx.x == 0)
    for (int i = 0; i < T / 64; ++i) join(place_of_wave[i], least_of_wave[i]);
  return x;
}

template <typename E>
__global__ __launch_bounds__(kSampleThreads) void sample_top_kernel(SampleView a, SampleGrid g, char* ws) {
  __shared__ u64 places[kWaves];
  __shared__ float leasts[kWaves];
  const int64_t row = blockIdx.y;
  const int c = blockIdx.x;
  const Row<E> r(a, row);
  const RowSpace s(ws, row, g);
  if (c == 0 && threadIdx.x == 0) s.state->arrived[0] = s.state->arrived[1] = 0;
  const Top top = find_top<kSampleThreads, false>(r, walk_of(r, g, c), places, leasts);
  if (threadIdx.x == 0) {
    s.best[c] = top.place;
    s.least[c] = top.least;
  }
}

// -------------------------------------------------------------------------------------- pass two
// Whether a row needs no sums; then its token is written by the workgroup that is told to.
__device__ __forceinline__ bool plain_row(const SampleView& a, int64_t row, const Limits& m, bool write) {
  if (!m.empty && !m.greedy) return false;
  if (write && threadIdx.x == 0) {
    a.token[row] = m.empty ? -1 : m.first;
    if (a.logprob) a.logprob[row] = m.empty ? -__builtin_inff() : 0.0f;
  }
  return true;
}

// The blocks' sums of the weights not below min-p: put(block, sum) by lane 63.
template <typename E, typename Put>
__device__ __forceinline__ void sum_blocks(const Limits& m, Walk<E> walk, Put put) {
  u64 sum = 0;
  walk.run([&](int, const float (&v)[8], bool) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const u64 w = m.weight(v[i]);
      sum += w >= m.least_weight ? w : 0;
    }
  }, [&](int block) {
    sum = sum_up_to(sum);
    if ((threadIdx.x & 63) == 63) put(block, sum);
    sum = 0;
  });
}

// A row without top-k and top-p: the blocks' sums, and the draw.
template <typename E>
__device__ __forceinline__ void free_row(const SampleView& a, int64_t row, const SampleGrid& g, const Limits& m,
                                         const RowSpace& s, Shared& sh, const Walk<E>& walk) {
  sum_blocks(m, walk, [&](int b, u64 sum) { tell(&s.sums[b], sum); });
  if (!last_of_row(&s.state->arrived[0], g.chunks, &sh.arrived)) return;
  if (threadIdx.x == 0) s.state->border.mode = kDone;
  draw<E>(a, row, g, m, sh, [&](int b) { return told(&s.sums[b]); }, [](float, int) { return true; });
}

template <typename E>
__global__ __launch_bounds__(kSampleThreads) void sample_free_kernel(SampleView a, SampleGrid g, char* ws) {
  __shared__ Shared sh;
  const int64_t row = blockIdx.y;
  const RowSpace s(ws, row, g);
  const Row<E> r(a, row);
  const auto walk = walk_of(r, g, blockIdx.x);
  const Limits m = limits_of(a, row, g, s, sh.step);
  if (plain_row(a, row, m, blockIdx.x == 0)) return;
  free_row(a, row, g, m, s, sh, walk);
}

// The same in one pass: the row stays in registers, as it lies in memory, between its largest logit and its
// weights; G groups of eight elements a lane.
template <typename E, int G>
__global__ __launch_bounds__(kRowThreads) void sample_row_kernel(SampleView a) {
  constexpr int T = kRowThreads, kRowWaves = T / 64;
  __shared__ Shared sh;
  __shared__ u64 sums[G * kRowWaves];   // of blocks of 512 elements
  __shared__ u64 best_of[kRowWaves];
  const int64_t row = blockIdx.x;
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  const Row<E> r(a, row);
  const E* l = r.p;
  const RowGroups groups(l, r.n);
  Raw<E> raw[G];
#pragma unroll
  for (int q = 0; q < G; ++q) {
    const int j = (q * T + t) * 8 - groups.shift;
    if (groups.full(j)) raw[q].load(l + j);
    else raw[q].clear();
  }
  const int edge = wave == 0 ? groups.edge(lane) : -1;
  const float at_edge = edge >= 0 ? r.at(edge) : -__builtin_inff();
  const Arguments given(a, row);
  // a lane's largest logit and its group
  float best = -__builtin_inff();
  int at = 0;
#pragma unroll
  for (int q = 0; q < G; ++q) {
    float v[8], top = -__builtin_inff();
    raw[q].get(v);
#pragma unroll
    for (int i = 0; i < 8; ++i) top = fmaxf(top, v[i]);   // passes over NaN
    top = plain(top);
    if (top > best) {
      best = top;
      at = (q * T + t) * 8 - groups.shift;
    }
  }
  int first = 0;
  if (best != -__builtin_inff())
    for (int i = 7; i >= 0; --i)
      if (r.at(at + i) == best) first = at + i;
  u64 place = place_of(best, first);
  if (edge >= 0) {
    const u64 x = place_of(at_edge, edge);
    place = x > place ? x : place;
  }
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) {
    const u64 x = __shfl_xor(place, o, 64);
    place = x > place ? x : place;
  }
  if (lane == 0) best_of[wave] = place;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kRowWaves; ++i) place = best_of[i] > place ? best_of[i] : place;
  const Limits m = limits_of(a, given, place, 0.0f, sh.step);
  if (plain_row(a, row, m, true)) return;
#pragma unroll
  for (int q = 0; q < G; ++q) {
    float v[8];
    raw[q].forget();
    raw[q].get(v);
    u64 sum = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const u64 w = m.weight(plain(v[i]));
      sum += w >= m.least_weight ? w : 0;
    }
    sum = sum_up_to(sum);
    if (lane == 63) sums[q * kRowWaves + wave] = sum;
  }
  __syncthreads();
  if (edge >= 0) {
    const u64 w = m.weight(at_edge);
    if (w >= m.least_weight) atomicAdd(&sums[(edge + groups.shift) / 512], w);
  }
  __syncthreads();
  const SampleGrid g{1, G * kRowWaves, G * kRowWaves, 9, 0};
  draw<E, T>(a, row, g, m, sh, [&](int b) { return sums[b]; }, [](float, int) { return true; });
}

// Tokens (with top-k) or weights of the intervals.
struct Bins {
  u64 weights[kBins];
  uint32_t counts[kBins];
  __device__ __forceinline__ void clear(int threads) {
    for (int i = threadIdx.x; i < kBins; i += threads) {
      weights[i] = 0;
      counts[i] = 0;
    }
  }
};

template <typename E>
__device__ __forceinline__ void fill_bins(const Limits& m, Walk<E> walk, Bins& bins) {
  if (m.k > 0) {
    walk.run([&](int, const float (&v)[8], bool) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (v[i] != -__builtin_inff()) atomicAdd(&bins.counts[m.bin(v[i])], 1u);
    }, [](int) {});
    return;
  }
  u64 rest = 0;   // of the last interval, which half of the tokens fall into and more
  walk.run([&](int, const float (&v)[8], bool) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const u64 w = m.weight(v[i]);
      const int bin = v[i] == -__builtin_inff() ? kBins - 1 : m.bin(v[i]);
      if (bin < kBins - 1) atomicAdd(&bins.weights[bin], w);
      else rest += w;
    }
  }, [](int) {});
  rest = sum_up_to(rest);
  if ((threadIdx.x & 63) == 63) atomicAdd(&bins.weights[kBins - 1], rest);
}

// The intervals that the cut lies in, from the consecutive ones that each of T lanes has: one lane writes them.
template <int T>
__device__ __forceinline__ void find_border(const Limits& m, const u64 (&w)[kBins / T], const uint32_t (&n)[kBins / T],
                                            Shared& sh, Border* out) {
  constexpr int kEach = kBins / T;
  const int t = threadIdx.x;
  u64 all_w = 0, all_n = 0, total, count;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    all_w += w[i];
    all_n += n[i];
  }
  u64 before_w = sum_before<T / 64>(all_w, sh.wave, total), before_n = sum_before<T / 64>(all_n, sh.wave, count);
  // with top-k the interval of the k-th token, and all before it where the list holds them; top-p
  // alone: the interval in which the sum reaches p
  const bool by_k = m.k > 0;
  if (by_k && static_cast<u64>(m.k) >= count) {   // no more than k tokens: top-k limits nothing
    if (t == 0) *out = Border{0, 0, 0, kBins, kBins, m.p < 1.0f ? kSearch : kListed};
    return;
  }
  bool rest = false;
  u64 want = by_k ? 0 : part_of(m.p, total, rest);
  want += rest || want == 0;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const bool here = by_k ? before_n < static_cast<u64>(m.k) && static_cast<u64>(m.k) <= before_n + n[i]
                           : before_w < want && want <= before_w + w[i];
    if (here) {
      const bool all = by_k && before_n + n[i] <= kList;
      const int hi = t * kEach + i;
      // top-p may cut anywhere above the k-th token; how many tokens a weight's interval holds is
      // seen when they are listed
      *out = Border{total, all ? 0 : before_w, all ? 0 : static_cast<uint32_t>(before_n), all ? 0 : hi, hi,
                    all || (n[i] <= kList && !(by_k && m.p < 1.0f)) ? kListed : kSearch};
    }
    before_w += w[i];
    before_n += n[i];
  }
}

template <typename E>
__global__ __launch_bounds__(kSampleThreads) void sample_bins_kernel(SampleView a, SampleGrid g, char* ws) {
  __shared__ Shared sh;
  __shared__ Bins bins;
  const int64_t row = blockIdx.y;
  const RowSpace s(ws, row, g);
  const int c = blockIdx.x, t = threadIdx.x;
  const Row<E> r(a, row);
  const auto walk = walk_of(r, g, c);
  bins.clear(kSampleThreads);
  const Limits m = limits_of(a, row, g, s, sh.step);
  if (plain_row(a, row, m, c == 0)) {
    if (c == 0 && t == 0) s.state->border.mode = kDone;
    return;
  }
  if (m.k == 0 && m.p == 1.0f) {
    free_row(a, row, g, m, s, sh, walk);
    return;
  }
  fill_bins(m, walk, bins);
  __syncthreads();
  if (g.chunks > 1) {
    for (int i = t; i < kBins; i += kSampleThreads) {
      if (m.k == 0) tell(&s.weights[c * kBins + i], bins.weights[i]);
      else tell(&s.counts[c * kBins + i], bins.counts[i]);
    }
  }
  if (!last_of_row(&s.state->arrived[0], g.chunks, &sh.arrived)) return;
  constexpr int kEach = kBins / kSampleThreads;
  u64 w[kEach];
  uint32_t n[kEach];
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    w[i] = g.chunks > 1 ? 0 : bins.weights[t * kEach + i];
    n[i] = g.chunks > 1 ? 0 : bins.counts[t * kEach + i];
  }
  if (g.chunks > 1) {
    // all chunks' loads before the first sum
    static_assert(kEach == 2, "a lane's two counts are read as one word");
    u64 part[kMostChunks][kEach];
    if (m.k == 0) {
#pragma unroll
      for (int k = 0; k < kMostChunks; ++k)
#pragma unroll
        for (int i = 0; i < kEach; ++i) part[k][i] = told(&s.weights[min(k, g.chunks - 1) * kBins + t * kEach + i]);
#pragma unroll
      for (int k = 0; k < kMostChunks; ++k)
#pragma unroll
        for (int i = 0; i < kEach; ++i) w[i] += k < g.chunks ? part[k][i] : 0;
    } else {
#pragma unroll
      for (int k = 0; k < kMostChunks; ++k)
        part[k][0] = told(reinterpret_cast<const u64*>(s.counts) + (min(k, g.chunks - 1) * kBins / 2 + t));
#pragma unroll
      for (int k = 0; k < kMostChunks; ++k) {
        n[0] += k < g.chunks ? static_cast<uint32_t>(part[k][0]) : 0;
        n[1] += k < g.chunks ? static_cast<uint32_t>(part[k][0] >> 32) : 0;
      }
    }
  }
  find_border<kSampleThreads>(m, w, n, sh, &s.state->border);
}

// ------------------------------------------------------------------------------------ pass three
struct ListSpace {
  alignas(16) u64 place[kList];
  u64 bin_weights[256];
  uint32_t bin_counts[256];
};

// The lowest place that is kept: in falling order, the first one at which the count (by_count) or
// the sum of the weights reaches want >= 1, and 0 where none does.  Digit by digit, of what `each` calls
// its argument with: (place, weight) of every token.  The places have the bits of `base` but for the
// last `bits`.
template <int T, typename Each>
__device__ __forceinline__ u64 find_cut(bool by_count, u64 want, u64 base, int bits, Shared& s, ListSpace& list, Each each) {
  const int t = threadIdx.x;
  u64 prefix = base >> bits << bits;
  __syncthreads();
  if (t < 256) {
    list.bin_weights[t] = 0;
    list.bin_counts[t] = 0;
  }
  if (t == 0) s.found[2] = 0;
  __syncthreads();
  for (int known = bits; known > 0;) {
    const int shift = known > 8 ? known - 8 : 0;
    each([&](u64 place, u64 w) {
      if (w == 0 || place >> known != prefix >> known) return;
      const int b = 255 - static_cast<int>(place >> shift & 255);
      atomicAdd(&list.bin_counts[b], 1u);
      if (!by_count) atomicAdd(&list.bin_weights[b], w);
    });
    __syncthreads();
    uint32_t count = 0;
    u64 here = 0;
    if (t < 256) {
      count = list.bin_counts[t];
      here = by_count ? count : list.bin_weights[t];
      list.bin_counts[t] = 0;
      list.bin_weights[t] = 0;
    }
    u64 total;
    const u64 before = sum_before<T / 64>(here, s.wave, total);
    if (before < want && want <= before + here) {
      s.found[0] = 255 - t;
      s.found[1] = want - before;
      s.found[2] = count;
    }
    __syncthreads();
    if (s.found[2] == 0) return 0;
    prefix |= s.found[0] << shift;
    want = s.found[1];
    known = shift;
    if (s.found[2] > 1) continue;
    // one token is left.  Its own place is told from those that `each` does not go through
    each([&](u64 place, u64 w) {
      if (w > 0 && place >> known == prefix >> known) s.found[3] = place;
    });
    __syncthreads();
    return s.found[3];
  }
  return prefix;
}

// The cut of a row's top-k and top-p, from the tokens that `each` goes through; what lies before
// them counts and weighs as given.
template <int T, typename Each>
__device__ __forceinline__ u64 cut_of(const Limits& m, u64 total, u64 weight_before, u64 count_before, u64 base, int bits,
                                      Shared& s, ListSpace& list, Each each) {
  u64 cut = 0;
#pragma unroll 1
  for (int by_k = m.k > 0; by_k >= (m.p < 1.0f ? 0 : 1); --by_k) {
    u64 want = m.k - count_before;
    if (!by_k) {
      if (m.k > 0) {   // p of the first k
        u64 sum = 0;
        each([&](u64 place, u64 w) { sum += place >= cut ? w : 0; });
        sum_before<T / 64>(sum, s.wave, total);
        total += weight_before;
      }
      bool rest;
      want = part_of(m.p, total, rest);
      want += rest || want == 0;
      want -= weight_before;
    }
    const u64 found = find_cut<T>(by_k != 0, want, base, bits, s, list, each);
    cut = found > cut ? found : cut;
  }
  return cut;
}

// The same for n <= T listed tokens, which are sorted: a lane counts the places before its own, in reads that all
// lanes share and that do not wait for each other, where exchanges wait for each other up to 45 times.  (As
// positive numbers in floating point, places are in the same order.)
template <int T>
__device__ __forceinline__ u64 cut_of_few(const Limits& m, u64 total, u64 weight_before, u64 count_before, int n, Shared& s,
                                          ListSpace& list) {
  const int t = threadIdx.x;
  constexpr int kAtOnce = 16;
  static_assert(2 * T + kAtOnce <= kList, "beside each other");
  u64* sorted = list.place + T + kAtOnce;
  u64 place = t < n ? list.place[t] : 0;
  if (t < kAtOnce) list.place[n + t] = 0;
  __syncthreads();
  int rank = 0;
#pragma unroll 1
  for (int i = 0; i < n; i += kAtOnce) {
    double2 x[kAtOnce / 2];
#pragma unroll
    for (int k = 0; k < kAtOnce / 2; ++k) x[k] = reinterpret_cast<const double2*>(list.place + i)[k];
#pragma unroll
    for (int k = 0; k < kAtOnce / 2; ++k)
      rank += (x[k].x > __longlong_as_double(place)) + (x[k].y > __longlong_as_double(place));
  }
  if (t < n) sorted[rank] = place;
  __syncthreads();
  if (t < n) place = sorted[t];
  const u64 w = t < n ? m.weight(logit_at(place)) : 0;
  bool keep = t < n;
  if (m.k > 0) {
    keep = keep && t + count_before < static_cast<u64>(m.k);
    if (m.p < 1.0f) {
      sum_before<T / 64>(keep ? w : 0, s.wave, total);
      total += weight_before;
    }
  }
  if (m.p < 1.0f) {
    bool rest;
    u64 want = part_of(m.p, total, rest);
    want += rest || want == 0;
    u64 all;
    const u64 before = sum_before<T / 64>(w, s.wave, all);   // by every lane: it has barriers
    keep = keep && before + weight_before < want;
  }
  // the kept ones are the first ones: the last of them is the cut
  const u64 kept = __ballot(keep);
  __syncthreads();
  if ((t & 63) == 0) s.wave[t >> 6] = __popcll(kept);
  __syncthreads();
  int count = 0;
#pragma unroll
  for (int i = 0; i < T / 64; ++i) count += static_cast<int>(s.wave[i]);
  return count > 0 ? sorted[count - 1] : ~u64(0);
}

// v[i], by selections: an array that is indexed by a register leaves the registers.
__device__ __forceinline__ float pick(const float (&v)[8], int i) {
  const bool one = i & 1, two = i & 2;
  const float a = one ? v[1] : v[0], b = one ? v[3] : v[2], c = one ? v[5] : v[4], d = one ? v[7] : v[6];
  const float low = two ? b : a, high = two ? d : c;
  return i & 4 ? high : low;
}

// The tokens of the border's intervals into list.place, as far as it goes (sh.listed: their number), and the
// sums of what lies above them: put(block, sum) by lane 63.
template <typename E, typename Put>
__device__ __forceinline__ void list_tokens(const Limits& m, const Border& x, Walk<E> walk, Shared& sh, ListSpace& list,
                                            Put put) {
  u64 sum = 0;
  walk.run([&](int j, const float (&v)[8], bool) {
    // first what each of the eight is, without a branch, then the few that count one by one
    unsigned above = 0, listed = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int bin = v[i] == -__builtin_inff() ? kBins : m.bin(v[i]);
      above |= static_cast<unsigned>(bin < x.lo) << i;
      listed |= static_cast<unsigned>(bin >= x.lo && bin <= x.hi && bin < kBins) << i;
    }
#pragma unroll 1
    for (; above; above &= above - 1) {
      const u64 w = m.weight(pick(v, __ffs(above) - 1));
      sum += w >= m.least_weight ? w : 0;
    }
    if (listed == 0) return;
    uint32_t at = atomicAdd(&sh.listed, static_cast<uint32_t>(__popc(listed)));
#pragma unroll 1
    for (; listed && at < kList; listed &= listed - 1, ++at) {
      const int i = __ffs(listed) - 1;
      list.place[at] = place_of(pick(v, i), j + i);
    }
  }, [&](int block) {
    if (x.lo > 0) sum = sum_up_to(sum);
    if ((threadIdx.x & 63) == 63) put(block, sum);
    sum = 0;
  });
}

// The cut and the draw, by one workgroup: from the n listed tokens, or where they are more than the list holds
// the whole row.  sums: of the blocks, the listed tokens aside.
template <typename E, int T>
__device__ __forceinline__ void finish_row(const SampleView& a, int64_t row, const SampleGrid& g, const Limits& m,
                                           const Border& x, int n, const Row<E>& r, Shared& sh, ListSpace& list, u64* sums) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, t = threadIdx.x;
  const bool in_list = x.mode == kListed && n <= kList;
  u64 cut = 0;
  if (!in_list) {
    for (int b = t; b < g.blocks; b += T) sums[b] = 0;
    __syncthreads();
  }
  const auto each = [&](auto f) {
    if (in_list) {
#pragma unroll 1
      for (int i = t; i < n; i += T) f(list.place[i], m.weight(logit_at(list.place[i])));
    } else {
#pragma unroll 1
      for (int j = t; j < r.n; j += T) {
        const float l = r.at(j);
        f(place_of(l, j), m.weight(l));
      }
    }
  };
  if (in_list && n <= T) {
    if (x.lo < kBins) cut = cut_of_few<T>(m, x.total, x.weight_before, x.count_before, n, sh, list);
  } else if (!in_list || x.lo < kBins) {
    u64 base = 0;   // what the listed tokens' places have in common
    int bits = 32 + kIndexBits;
    if (in_list) {
      base = list.place[0];
      u64 other = 0;
      for (int i = t; i < n; i += T) other |= list.place[i] ^ base;
#pragma unroll
      for (int o = 32; o >= 1; o >>= 1) other |= __shfl_xor(other, o, 64);
      if (lane == 0) sh.wave[wave] = other;
      __syncthreads();
      other = 0;
#pragma unroll
      for (int i = 0; i < T / 64; ++i) other |= sh.wave[i];
      bits = 64 - __clzll(other);
    }
    cut = cut_of<T>(m, x.total, in_list ? x.weight_before : 0, in_list ? x.count_before : 0, base, bits, sh, list, each);
  }
  __syncthreads();
  each([&](u64 place, u64 w) {
    if (w > 0 && place >= cut && w >= m.least_weight) atomicAdd(&sums[index_at(place) + r.shift >> g.log_size], w);
  });
  __syncthreads();
  draw<E, T>(a, row, g, m, sh, [&](int b) { return sums[b]; }, [&](float l, int j) { return place_of(l, j) >= cut; });
}

template <typename E>
__global__ __launch_bounds__(kSampleThreads) void sample_cut_kernel(SampleView a, SampleGrid g, char* ws) {
  __shared__ Shared sh;
  __shared__ ListSpace list;
  __shared__ u64 sums[kMostBlocks];
  const int64_t row = blockIdx.y;
  const RowSpace s(ws, row, g);
  const int lane = threadIdx.x & 63, c = blockIdx.x, t = threadIdx.x;
  const Row<E> r(a, row);
  const auto walk = walk_of(r, g, c);
  const Border x = s.state->border;
  if (t == 0) sh.listed = 0;
  const Limits m = limits_of(a, row, g, s, sh.step);
  if (x.mode == kDone) return;
  if (x.mode == kListed) {
    list_tokens(m, x, walk, sh, list, [&](int b, u64 sum) { tell(&s.sums[b], sum); });
    if (g.chunks > 1) {
      __syncthreads();
      const uint32_t mine = sh.listed;
      for (uint32_t i = t; i < min(mine, static_cast<uint32_t>(kList)); i += kSampleThreads)
        tell(&s.list[c * kList + i], list.place[i]);
      if (t == 0) tell(&s.listed[c], mine);
    }
  }
  if (!last_of_row(&s.state->arrived[1], g.chunks, &sh.arrived)) return;
  int n = 0, before = 0;
  const int part = t / 16;   // sixteen lanes for a chunk's list
  static_assert(kMostChunks * 16 <= kSampleThreads, "a row of lanes a chunk");
  if (x.mode == kListed) {
    uint32_t count = g.chunks > 1 ? (lane < g.chunks ? told(&s.listed[lane]) : 0) : (lane == 0 ? sh.listed : 0);
#pragma unroll
    for (int i = 0; i < kMostChunks; ++i) {
      const int here = min(__shfl(static_cast<int>(count), i, 64), kList + 1);
      if (i < part) before += here;
      n += here;
    }
    count = __shfl(count, part, 64);
    if (g.chunks > 1 && n <= kList && part < g.chunks)
      for (uint32_t i = t % 16; i < count; i += 16) list.place[before + i] = told(&s.list[part * kList + i]);
    for (int b = t; b < g.blocks; b += kSampleThreads) sums[b] = told(&s.sums[b]);
    __syncthreads();
  }
  finish_row<E, kSampleThreads>(a, row, g, m, x, n, r, sh, list, sums);
}

// ----------------------------------------------------------------------------- a row a workgroup
// All passes in one launch, the later ones from the caches.
template <typename E, int T>
__global__ __launch_bounds__(T) void sample_whole_kernel(SampleView a, SampleGrid g) {
  __shared__ Shared sh;
  __shared__ Bins bins;
  __shared__ ListSpace list;
  __shared__ u64 sums[kMostBlocks], places[T / 64];
  __shared__ float leasts[T / 64];
  __shared__ Border border;
  const int64_t row = blockIdx.x;
  const int t = threadIdx.x;
  const Row<E> r(a, row);
  const auto walk = walk_of<T>(r, g, 0);
  const Arguments given(a, row);
  bins.clear(T);
  if (t == 0) sh.listed = 0;
  const Top top = find_top<T, true>(r, walk, places, leasts);
  const Limits m = limits_of(a, given, top.place, top.least, sh.step);
  if (plain_row(a, row, m, true)) return;
  const auto put = [&](int b, u64 sum) { sums[b] = sum; };
  if (m.k == 0 && m.p == 1.0f) {
    sum_blocks(m, walk, put);
    __syncthreads();
    draw<E, T>(a, row, g, m, sh, [&](int b) { return sums[b]; }, [](float, int) { return true; });
    return;
  }
  fill_bins(m, walk, bins);
  __syncthreads();
  constexpr int kEach = kBins / T;
  u64 w[kEach];
  uint32_t n[kEach];
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    w[i] = bins.weights[t * kEach + i];
    n[i] = bins.counts[t * kEach + i];
  }
  find_border<T>(m, w, n, sh, &border);
  __syncthreads();
  const Border x = border;
  if (x.mode == kListed) list_tokens(m, x, walk, sh, list, put);
  __syncthreads();
  finish_row<E, T>(a, row, g, m, x, static_cast<int>(sh.listed), r, sh, list, sums);
}

// ------------------------------------------------------------------------------------------ host
static SampleGrid whole_row(int64_t vocab) {
  SampleGrid g;
  g.log_size = vocab <= (1 << 20) ? 9 : vocab <= (1 << 21) ? 10 : 11;
  g.blocks = static_cast<int>((vocab + 7 + g.size() - 1) / g.size());   // wherever the row begins
  g.chunks = 1;
  g.blocks_a_chunk = g.blocks;
  g.row_bytes = 0;
  return g;
}

static SampleGrid sample_grid(int64_t n_rows, int64_t vocab) {
  SampleGrid g = whole_row(vocab);
  // about four workgroups a CU, and a block at least for each of their waves
  int64_t chunks = 4 * device_cus() / n_rows;
  if (chunks > (g.blocks + kWaves - 1) / kWaves) chunks = (g.blocks + kWaves - 1) / kWaves;
  if (chunks > kMostChunks) chunks = kMostChunks;
  if (chunks < 1) chunks = 1;
  g.blocks_a_chunk = static_cast<int>((g.blocks + chunks - 1) / chunks);
  g.chunks = (g.blocks + g.blocks_a_chunk - 1) / g.blocks_a_chunk;
  g.row_bytes = static_cast<int64_t>(align_up(
      64 + 8 * (kMostChunks + kMostBlocks + 7) + static_cast<size_t>(g.chunks) * (8 * kList + 12 * kBins) + 8 * kMostChunks, 256));
  return g;
}

// A row gets one workgroup where there are rows for all CUs, or where it is short.  bf16, us with one and with
// several workgroups a row: top-k and top-p, 64 rows of 2000: 15, 20; of 16000: 23, 25; of 32000: 32, 30; of
// 100352: 66, 36; 256 rows of 32000: 33, 41; of 100352: 69, 71; 512 rows: 45, 57; 95, 110.
constexpr int kShortBlocks = 33;
static bool one_workgroup(int64_t n_rows, const SampleGrid& g) { return n_rows >= device_cus() || g.blocks <= kShortBlocks; }

size_t sample_workspace_bytes(int64_t n_rows, int64_t vocab) {
  const SampleGrid g = sample_grid(n_rows, vocab);
  return one_workgroup(n_rows, g) ? 0 : static_cast<size_t>(n_rows) * g.row_bytes;
}

// Groups of eight elements a lane with which rows of temperature and min-p alone are worked off in registers, or
// 0: long rows too few to occupy half of the CUs are faster in parts.  bf16, us in registers and
// otherwise: 64 rows of 16000: 9, 12; of 50021: 20, 16; 128 rows: 21, 23; 512 rows: 41, 52; 512 rows of
// 100352: 68, 86.  25 groups are the most: in 32 (201 registers) and otherwise 128 rows of 102400 take 38, 32, 512 rows 81,
// 75; of 128256 128 rows take 37, 35, 256 rows 43, 57, 512 rows 85, 91.
template <typename E>
static int row_groups(const SampleView& v) {
  const int64_t w = v.vocab + 7;
  if (v.top_k || v.top_p || (v.n_rows < device_cus() / 2 && w > kRowThreads * 8 * 4)) return 0;
  for (int g : {2, 4, 8, 16})
    if (w <= int64_t(kRowThreads) * 8 * g) return g;
  return sizeof(E) == 2 && w <= int64_t(kRowThreads) * 8 * 25 ? 25 : 0;
}

template <typename E>
static bool sample_rows(const SampleView& v, hipStream_t s) {
  const dim3 grid(static_cast<unsigned>(v.n_rows)), threads(kRowThreads);
  switch (row_groups<E>(v)) {
    case 2: sample_row_kernel<E, 2><<<grid, threads, 0, s>>>(v); return true;
    case 4: sample_row_kernel<E, 4><<<grid, threads, 0, s>>>(v); return true;
    case 8: sample_row_kernel<E, 8><<<grid, threads, 0, s>>>(v); return true;
    case 16: sample_row_kernel<E, 16><<<grid, threads, 0, s>>>(v); return true;
    case 25:
      if constexpr (sizeof(E) == 2) sample_row_kernel<E, 25><<<grid, threads, 0, s>>>(v);
      return true;
    default: return false;
  }
}

template <typename E>
static void sample(const SampleView& a, char* ws, hipStream_t s) {
  if (sample_rows<E>(a, s)) return;
  SampleGrid g = sample_grid(a.n_rows, a.vocab);
  if (one_workgroup(a.n_rows, g)) {
    g = whole_row(a.vocab);
    const dim3 grid(static_cast<unsigned>(a.n_rows));
    // four waves where a row has no more than two blocks for each: with eight 2048 rows of 500 take 72 us
    if (g.blocks <= 9) sample_whole_kernel<E, 256><<<grid, dim3(256), 0, s>>>(a, g);
    else sample_whole_kernel<E, 512><<<grid, dim3(512), 0, s>>>(a, g);
    return;
  }
  const dim3 grid(g.chunks, static_cast<unsigned>(a.n_rows)), threads(kSampleThreads);
  sample_top_kernel<E><<<grid, threads, 0, s>>>(a, g, ws);
  if (!a.top_k && !a.top_p) {
    sample_free_kernel<E><<<grid, threads, 0, s>>>(a, g, ws);
  } else {
    sample_bins_kernel<E><<<grid, threads, 0, s>>>(a, g, ws);
    sample_cut_kernel<E><<<grid, threads, 0, s>>>(a, g, ws);
  }
}

hipError_t launch_sample(const SampleView& v, int32_t dtype, void* ws, hipStream_t s) {
  if (dtype == STAPLE_BF16) sample<bf16_t>(v, static_cast<char*>(ws), s);
  else sample<float>(v, static_cast<char*>(ws), s);
  return hipGetLastError();
}

}  // namespace staple
