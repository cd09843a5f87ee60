// Sampling from stored logits with temperature, top-k, top-p and min-p, from one given uniform
// number per row.  Nothing is sorted, and all sums are integers.
//
// The weight of logit l is W = floor(2^40 * exp((l - max) / T)), the float32 exponential as an
// integer (exact from 2^-16 up, cut at 2^-40 of the largest weight).  n <= 2^22, so a row's
// sum is at most 2^62.  Integer sums do not depend on their order, so the result is the same
// for every split of the row over threads and workgroups, atomics included.
//
// Sorting is not needed because 16-bit logits have at most 2^16 values: what top-k and top-p
// keep is "every key above t, and the first c columns with key t" for an order key t.  t is
// found with two histograms: the keys' high 11 bits (count and weight per bin), then the low
// 5 bits inside the bin where the k-th column, or the top-p share of the weight, falls.
// The draw runs over the kept columns in index order: u times their sum, located by sums over
// ever shorter ranges.
//
// Four kernels, because the weights need the row's maximum and the threshold needs the whole
// row: (1) each chunk's largest key and its first column; (2) each chunk's weights, into the
// row's histogram or, for a row without top-k and top-p, as the chunk's sum; (3) the
// threshold's bin, and each chunk's columns from that bin up, the candidates; (4) one
// workgroup per row, with the candidates in its LDS, finds the threshold and draws.  Where
// there are more candidates than that pays for, (3) has left each chunk's weight above the bin and
// its columns of each key in the bin, from which (4) finds the threshold and the chunk to draw
// from.  What touches every column is spread over the chunks' workgroups: one workgroup takes
// about 10 us for 10 instructions on each of 150000 columns.  (Two kernels with one workgroup
// per row for all that follows the maximum: 74 us for a row, 132 us for 32.)
//
// What bounds it: for one row the chain of four launches (2.3 us each at least) and, inside
// them, of loads, scans and barriers; a row's columns are loaded before its settings, maximum
// and threshold arrive.  For many rows (2) is bound by its vector instructions, about 70 per
// column, most of them the exponential, the division by T (a product with 1/T and a correction
// changed nothing measurable) and the conversion to an integer.  Measured, 151936 columns: one
// row with top-k and top-p 25 us; 32 rows with mixed settings 40 us (5 + 11 + 10 + 14 us).
#include "device_common.hpp"
#include "sample.hpp"

namespace qmm {
namespace sampling {
namespace {

typedef unsigned long long u64;

constexpr int kChunkThreads = 256;
constexpr int kRowThreads = 1024;
constexpr int kRowWaves = kRowThreads / 64;
constexpr int kLow = 32;             // keys per bin
constexpr int kShift = 5;
// Candidates that one wave draws from, and that a row draws from at all; beyond, the chunks'
// sums are faster (3707 candidates: 31 us a call instead of 40).  Only a top-p inside a top-k
// needs up to kCandidates, since the chunks do not know its bin.
constexpr uint32_t kFew = 256, kHeld = 1024;
constexpr int kUnitBits = 24;        // u and top_p count in units of 2^-24
constexpr int kRun = 8;              // consecutive columns per lane and step
constexpr int kStep = 64 * kRun;     // columns per wave and step
constexpr int kCols = kRun * kChunkThreads;   // columns per workgroup and step of the chunk kernels

// Order key of a 16-bit logit: larger logits have larger keys, NaN and -inf (never drawn) 0.
template <bool FP16>
__device__ inline uint32_t key_of(uint32_t b) {
  constexpr uint32_t kInf = FP16 ? 0x7C00u : 0x7F80u, kLeast = 0xFFFFu - (0x8000u | kInf) + 1u;   // of the lowest finite
  uint32_t k = b ^ (0x8000u | (uint32_t)-(int32_t)(b >> 15)) & 0xFFFFu;
  k = k == 0x7FFFu ? 0x8000u : k;    // -0 draws like +0
  return k - kLeast <= (0x8000u | kInf) - kLeast ? k : 0u;
}

template <class T>
__device__ inline float key_value(uint32_t key) {
  return T::to_f32((key & 0x8000u) ? (key & 0x7FFFu) : (~key & 0xFFFFu));
}

// A row's settings.
struct Row {
  float t, min_p;
  uint32_t k;            // 0: no top-k
  uint32_t units;        // top_p in units of 2^-24; 2^24: no top-p
  bool greedy;           // the first maximum, whatever u is
  __device__ bool threshold() const { return k || units < (1u << kUnitBits); }   // top-k or top-p cuts the row
};

__device__ inline uint32_t units_of(float x) {   // floor(clamp(x, 0, 1) * 2^24), 0 for NaN
  return x >= 1.0f ? 1u << kUnitBits : (x > 0.0f ? (uint32_t)(x * 16777216.0f) : 0u);
}

__device__ inline Row row_settings(const SampleArgs& a, int64_t row) {
  Row r;
  r.t = a.temperature.get(row);
  r.min_p = a.min_p.get(row);
  const int32_t k = a.top_k.get(row);
  r.k = k > 0 && k < a.n ? (uint32_t)k : 0u;
  r.units = units_of(a.top_p.get(row));
  // a share of nothing, one column, and weights of more than the largest all leave the first
  // maximum alone
  r.greedy = !(r.t > 0.0f) || r.units == 0u || k == 1 || !(r.min_p <= 1.0f);
  return r;
}

// Relative weight (1 for the maximum) and its integer.
template <class T>
__device__ inline float weight(uint32_t key, uint32_t top_key, float top, float t) {
  return key == top_key ? 1.0f : expf((key_value<T>(key) - top) / t);
}
__device__ inline u64 weight_int(float w) { return (u64)(w * 1099511627776.0f); }

// floor(total * units / 2^24); total <= 2^62, units <= 2^24
__device__ inline u64 share(u64 total, uint32_t units) {
  const u64 mask = (1ull << kUnitBits) - 1;
  return (total >> kUnitBits) * units + (((total & mask) * units) >> kUnitBits);
}

// Keys of columns [i, i + 8) of a row of n columns, 0 past its end.
template <bool FP16>
__device__ inline void load_keys(const uint16_t* row, int64_t i, int64_t end, bool vec, uint32_t (&k)[kRun]) {
  if (vec && i + kRun <= end) {
    const u32x4 v = *(const u32x4*)(row + i);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      k[2 * e] = key_of<FP16>(v[e] & 0xFFFFu);
      k[2 * e + 1] = key_of<FP16>(v[e] >> 16);
    }
  } else {
#pragma unroll
    for (int e = 0; e < kRun; ++e) k[e] = i + e < end ? key_of<FP16>(row[i + e]) : 0u;
  }
}

// The same columns as they are, four runs `step` apart: what a kernel loads before it knows the
// row's settings.  Past the end NaN, whose key is 0.
constexpr int kAhead = 4;
struct Ahead {
  u32x4 w[kAhead];
  template <bool FP16>
  __device__ uint32_t key(int j, int e) const {
    return key_of<FP16>((w[j][e >> 1] >> (16 * (e & 1))) & 0xFFFFu);
  }
};
__device__ inline void load_ahead(const uint16_t* row, int64_t i, int64_t end, int64_t step, bool vec, Ahead& r) {
#pragma unroll
  for (int j = 0; j < kAhead; ++j) {
    const int64_t c = i + j * step;
    r.w[j] = u32x4{~0u, ~0u, ~0u, ~0u};
    if (c >= end) continue;
    if (vec && c + kRun <= end) {
      r.w[j] = *(const u32x4*)(row + c);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        r.w[j][e] = (c + 2 * e < end ? (uint32_t)row[c + 2 * e] : 0xFFFFu) |
                    (c + 2 * e + 1 < end ? (uint32_t)row[c + 2 * e + 1] : 0xFFFFu) << 16;
    }
  }
}

// f(key) for the runs of columns at i, i + step, .. below end (key 0 past it); four runs are
// loaded before the first is used.
template <bool FP16, class F>
__device__ inline void each_key(const uint16_t* row, int64_t i, int64_t end, int64_t step, bool vec, F&& f) {
  for (; i < end; i += kAhead * step) {
    Ahead a;
    load_ahead(row, i, end, step, vec, a);
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
#pragma unroll
      for (int e = 0; e < kRun; ++e) f(a.template key<FP16>(j, e));
  }
}

__device__ inline u64 shfl_xor64(u64 v, int d) {
  const uint32_t lo = __shfl_xor((uint32_t)v, d), hi = __shfl_xor((uint32_t)(v >> 32), d);
  return ((u64)hi << 32) | lo;
}
__device__ inline u64 shfl_up64(u64 v, int d) {
  const uint32_t lo = __shfl_up((uint32_t)v, d), hi = __shfl_up((uint32_t)(v >> 32), d);
  return ((u64)hi << 32) | lo;
}
__device__ inline u64 wave_max64(u64 v) {
  for (int d = 1; d < 64; d <<= 1) {
    const u64 o = shfl_xor64(v, d);
    v = o > v ? o : v;
  }
  return v;
}
__device__ inline u64 wave_sum64(u64 v) {
  for (int d = 1; d < 64; d <<= 1) v += shfl_xor64(v, d);
  return v;
}

// Largest (key, first column) word of the row, from its chunks' words.  Every lane gets it.
__device__ inline u64 row_top(const RowSpace& s, int chunks, int lane) {
  u64 top = 0;
  for (int c = lane; c < chunks; c += 64) top = s.top[c] > top ? s.top[c] : top;
  return wave_max64(top);
}

template <bool FP16>
__global__ __launch_bounds__(kChunkThreads) void chunk_top_kernel(const SampleArgs a) {
  __shared__ u64 wave_top[kChunkThreads / 64];
  const int64_t row = blockIdx.y;
  const int chunk = blockIdx.x;
  RowSpace& s = a.space[row];
  // clear this chunk's share of the histogram (the next kernel adds to it)
  for (int i = chunk * kChunkThreads + threadIdx.x; i < kBins; i += a.chunks * kChunkThreads) {
    s.mass[i] = 0ull;
    s.count[i] = 0u;
  }
  if (chunk == 0 && threadIdx.x == 0) s.found = 0u;
  const uint16_t* x = (const uint16_t*)a.logits + row * a.row_stride;
  const bool vec = ((uintptr_t)x & 15u) == 0u;
  const int64_t begin = chunk * a.chunk, end = min(a.n, begin + a.chunk);
  uint32_t key = 0u, column = 0u;    // the thread's largest, and its first column (columns ascend)
  for (int64_t i = begin + kRun * threadIdx.x; i < end; i += kAhead * kCols) {
    Ahead v;
    load_ahead(x, i, end, kCols, vec, v);
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      if (i + j * kCols >= end) break;
#pragma unroll
      for (int e = 0; e < kRun; ++e) {
        const uint32_t k = v.template key<FP16>(j, e);
        column = k > key ? (uint32_t)(i + j * kCols) + e : column;
        key = k > key ? k : key;
      }
    }
  }
  u64 top = wave_max64(key ? ((u64)key << 32) | (0xFFFFFFFFu - column) : 0ull);
  if ((threadIdx.x & 63) == 0) wave_top[threadIdx.x >> 6] = top;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < kChunkThreads / 64; ++w) top = wave_top[w] > top ? wave_top[w] : top;
    s.top[chunk] = top;
  }
}

template <class T>
__global__ __launch_bounds__(kChunkThreads) void chunk_weights_kernel(const SampleArgs a) {
  constexpr bool FP16 = T::kDtype == 2;
  __shared__ u64 mass[kBins];
  __shared__ uint32_t count[kBins];
  __shared__ u64 wave_mass[kChunkThreads / 64];
  const int64_t row = blockIdx.y;
  const int chunk = blockIdx.x, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  RowSpace& s = a.space[row];
  const uint16_t* x = (const uint16_t*)a.logits + row * a.row_stride;
  const bool vec = ((uintptr_t)x & 15u) == 0u;
  const int64_t begin = chunk * a.chunk, end = min(a.n, begin + a.chunk);
  Ahead v;                                    // (in flight while the settings and the maximum arrive)
  load_ahead(x, begin + kRun * threadIdx.x, end, kCols, vec, v);
  const Row r = row_settings(a, row);
  const u64 top_word = row_top(s, a.chunks, lane);
  const uint32_t top_key = (uint32_t)(top_word >> 32);
  if (r.greedy || top_key == 0u) return;      // the same in the whole workgroup
  const float top = key_value<T>(top_key);
  const bool threshold = r.threshold();
  if (threshold) {
    for (int i = threadIdx.x; i < kBins; i += kChunkThreads) {
      mass[i] = 0ull;
      count[i] = 0u;
    }
    __syncthreads();
  }
  u64 sum = 0;
  for (int64_t i = begin + kRun * threadIdx.x; i < end;) {
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      if (i + j * kCols >= end) break;
#pragma unroll
      for (int e = 0; e < kRun; ++e) {
        const uint32_t k = v.template key<FP16>(j, e);
        if (k == 0u) continue;
        const float w = weight<T>(k, top_key, top, r.t);
        if (threshold) {
          atomicAdd(&mass[k >> kShift], weight_int(w));
          atomicAdd(&count[k >> kShift], 1u);
        } else if (w >= r.min_p) {
          sum += weight_int(w);
        }
      }
    }
    i += kAhead * kCols;
    if (i < end) load_ahead(x, i, end, kCols, vec, v);
  }
  if (threshold) {
    __syncthreads();
    for (int i = threadIdx.x; i < kBins; i += kChunkThreads)
      if (count[i]) {
        atomicAdd(&s.mass[i], mass[i]);
        atomicAdd(&s.count[i], count[i]);
      }
  } else {
    sum = wave_sum64(sum);
    if (lane == 0) wave_mass[wave] = sum;
    __syncthreads();
    if (threadIdx.x == 0) {
      for (int w = 1; w < kChunkThreads / 64; ++w) sum += wave_mass[w];
      s.chunk_mass[chunk] = sum;
    }
  }
}

// Candidates of a row from which it is drawn.
__device__ inline uint32_t held_limit(int32_t mode, const Row& r) {
  return mode == kByCount && r.units < (1u << kUnitBits) ? (uint32_t)kCandidates : kHeld;
}

// What a row keeps: keys above t, and the first c columns with key t.
struct Cut {
  uint32_t t;
  uint32_t c;
};

// Shared state of a bin search.
template <int THREADS>
struct BinSearch {
  u64 mass[THREADS / 64];
  uint32_t count[THREADS / 64];
  int bin;
  u64 above_mass, total_mass;
  uint32_t above_count;
};

// The bin (from the top) in which the running count reaches `want_count` or, when that is 0,
// the running mass reaches want_mass(total mass); with the count and mass of the bins above
// it.  Each thread owns consecutive bins, thread order being descending.  bin = -1: not
// reached.
template <int THREADS, class W>
__device__ inline void find_bin(const RowSpace& s, uint32_t want_count, W&& want_mass, BinSearch<THREADS>& sh) {
  constexpr int kPer = kBins / THREADS;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  u64 m[kPer], mt = 0;
  uint32_t n[kPer], nt = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    m[i] = s.mass[kBins - 1 - (kPer * threadIdx.x + i)];
    n[i] = s.count[kBins - 1 - (kPer * threadIdx.x + i)];
    mt += m[i];
    nt += n[i];
  }
  u64 mi = mt;
  uint32_t ni = nt;
  for (int d = 1; d < 64; d <<= 1) {
    const u64 mo = shfl_up64(mi, d);
    const uint32_t no = __shfl_up(ni, d);
    if (lane >= d) {
      mi += mo;
      ni += no;
    }
  }
  if (threadIdx.x == 0) sh.bin = -1;
  if (lane == 63) {
    sh.mass[wave] = mi;
    sh.count[wave] = ni;
  }
  __syncthreads();
  u64 mb = mi - mt, total = 0;
  uint32_t nb = ni - nt;
#pragma unroll
  for (int w = 0; w < THREADS / 64; ++w) {
    if (w < wave) {
      mb += sh.mass[w];
      nb += sh.count[w];
    }
    total += sh.mass[w];
  }
  const u64 need = want_mass(total);
  if (threadIdx.x == 0) sh.total_mass = total;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const bool crosses = want_count ? nb < want_count && nb + n[i] >= want_count : mb < need && mb + m[i] >= need;
    if (crosses) {
      sh.bin = kBins - 1 - (kPer * (int)threadIdx.x + i);
      sh.above_mass = mb;
      sh.above_count = nb;
    }
    mb += m[i];
    nb += n[i];
  }
  __syncthreads();
}

// Smallest key whose relative weight reaches min_p (keys' weights rise with the key), found by
// one wave, 64 keys at a time.  Keys without a weight of their own (-inf and below) count as 0.
template <class T>
__device__ inline uint32_t smallest_key(uint32_t top_key, float top, float t, float min_p, int lane) {
  constexpr uint32_t kLeast = 0x10000u - (T::kDtype == 2 ? 0xFC00u : 0xFF80u);   // key of the lowest finite value
  if (!(min_p > 0.0f)) return 1u;
  uint32_t lo = 0u;      // keys up to lo fail
  for (int shift = 10; shift >= 0; shift = shift > 4 ? shift - 6 : (shift > 0 ? 0 : -1)) {
    const uint32_t key = lo + ((uint32_t)(lane + 1) << shift);
    const bool ok = key >= top_key || (key >= kLeast && weight<T>(key, top_key, top, t) >= min_p);
    const u64 fails = __ballot(!ok);
    const int n = fails == ~0ull ? 64 : __ffsll(~fails) - 1;   // leading lanes that fail
    lo += (uint32_t)n << shift;
  }
  return lo + 1u;
}

// Chunk-parallel: the row's threshold bin (the same in every workgroup of the row), and the
// chunk's columns that can lie above the threshold.
template <class T>
__global__ __launch_bounds__(kChunkThreads) void collect_kernel(const SampleArgs a) {
  constexpr bool FP16 = T::kDtype == 2;
  __shared__ BinSearch<kChunkThreads> sh;
  __shared__ uint32_t wave_n[kChunkThreads / 64], first, low[kLow];
  __shared__ u64 wave_mass[kChunkThreads / 64];
  const int64_t row = blockIdx.y;
  const int chunk = blockIdx.x, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  RowSpace& s = a.space[row];
  const uint16_t* x = (const uint16_t*)a.logits + row * a.row_stride;
  const bool vec = ((uintptr_t)x & 15u) == 0u;
  const int64_t begin = chunk * a.chunk, end = min(a.n, begin + a.chunk);
  Ahead v;                                 // (in flight while the threshold's bin is found)
  load_ahead(x, begin + kRun * threadIdx.x, end, kCols, vec, v);
  const Row r = row_settings(a, row);
  const u64 top_word = row_top(s, a.chunks, lane);
  const uint32_t top_key = (uint32_t)(top_word >> 32);
  const bool settled = top_key == 0u || r.greedy || !r.threshold();
  if (settled) {
    if (chunk == 0 && threadIdx.x == 0) {
      s.plan.top = top_word;
      s.plan.mode = top_key == 0u ? kNothing : (r.greedy ? kGreedy : kFree);
    }
    return;
  }
  const float top = key_value<T>(top_key);
  int32_t mode = kAll, bin = 0;
  if (r.k) {
    find_bin(s, r.k, [](u64) { return 0ull; }, sh);
    if (sh.bin >= 0) {
      mode = kByCount;
      bin = sh.bin;
    }
    __syncthreads();                       // sh is used again
  }
  if (mode == kAll && r.units < (1u << kUnitBits)) {
    find_bin(s, 0u, [&](u64 total) { return max(1ull, share(total, r.units)); }, sh);
    mode = kByMass;
    bin = sh.bin;
  }
  const uint32_t min_key = smallest_key<T>(top_key, top, r.t, r.min_p, lane);
  uint32_t edge = max(1u, (uint32_t)bin << kShift);
  int32_t low_bin = bin;
  // (min-p; but a top-p's share inside a top-k is of the weights below min_p too)
  if (mode != kByCount || r.units == (1u << kUnitBits)) {
    edge = max(edge, min_key);
    low_bin = max(bin, (int32_t)(min_key >> kShift));
  }
  // more columns above the bin than the last kernel draws from: none are stored
  const uint32_t limit = held_limit(mode, r);
  const bool store = mode == kAll || low_bin != bin || sh.above_count <= limit;
  if (threadIdx.x < kLow) low[threadIdx.x] = 0u;
  __syncthreads();
  if (chunk == 0 && threadIdx.x == 0) {
    RowPlan p;
    p.top = top_word;
    p.above_mass = sh.above_mass;          // (not used in mode kAll)
    p.total_mass = sh.total_mass;
    p.above_count = sh.above_count;
    p.mode = mode;
    p.bin = bin;
    p.low_bin = low_bin;
    p.min_key = min_key;
    s.plan = p;
    if (!store) s.found = limit + 1;
  }
  u64 mass = 0;
  for (int64_t base = begin; base < end; base += kAhead * kCols) {
    const int64_t i = base + kRun * threadIdx.x;
    uint32_t take = 0u;             // the thread's candidates, bit 8 j + e
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      if (base + j * kCols >= end) break;
#pragma unroll
      for (int e = 0; e < kRun; ++e) {
        const uint32_t k = v.template key<FP16>(j, e);
        if ((int)(k >> kShift) > low_bin) mass += weight_int(weight<T>(k, top_key, top, r.t));
        if (k && (int)(k >> kShift) == low_bin) atomicAdd(&low[k & (kLow - 1)], 1u);
        take |= k >= edge ? 1u << (kRun * j + e) : 0u;
      }
    }
    if (store) {
      const uint32_t n = __popc(take);
      uint32_t at = n;
      for (int d = 1; d < 64; d <<= 1) {
        const uint32_t o = __shfl_up(at, d);
        if (lane >= d) at += o;
      }
      if (lane == 63) wave_n[wave] = at;
      at -= n;
      __syncthreads();
      if (threadIdx.x == 0) {
        uint32_t all = 0;
        for (int g = 0; g < kChunkThreads / 64; ++g) all += wave_n[g];
        first = all ? atomicAdd(&s.found, all) : 0u;   // n <= 2^22: no wrap
      }
      __syncthreads();
      at += first;
      for (int g = 0; g < wave; ++g) at += wave_n[g];
      for (; take; take &= take - 1u, ++at) {          // few: their logits are read again
        const int bit = __ffs(take) - 1;
        const int64_t c = i + (bit / kRun) * kCols + bit % kRun;
        if (at >= limit) break;
        const uint32_t k = key_of<FP16>(x[c]);
        s.candidate[at] = ((u64)k << 32) | (uint32_t)c;
        s.weight[at] = weight<T>(k, top_key, top, r.t);
      }
      __syncthreads();                     // wave_n and first are used again
    }
    if (base + kAhead * kCols < end) load_ahead(x, i + kAhead * kCols, end, kCols, vec, v);
  }
  mass = wave_sum64(mass);
  if (lane == 0) wave_mass[wave] = mass;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int v = 1; v < kChunkThreads / 64; ++v) mass += wave_mass[v];
    s.chunk_mass[chunk] = mass;
  }
  if (threadIdx.x < kLow) s.chunk_low[chunk][threadIdx.x] = low[threadIdx.x];
}

// Shared state of the row kernel.
struct RowShared {
  BinSearch<kRowThreads> search;
  uint32_t low[kLow];
  u64 part_mass[kRowWaves];
  uint32_t part_ties[kRowWaves];
  u64 slot_mass[64];
  uint32_t slot_count[64];
  Cut cut;
  u64 kept_mass;
  int64_t begin, end;
  u64 target, before_mass, total;
  uint32_t before_ties;
  u64 low_weight[kLow];
  u64 chunk_mass[kMaxChunks];
  uint32_t chunk_ties[kMaxChunks];
};

// Columns of each key of one bin, into sh.low, from the whole row.
template <bool FP16>
__device__ inline void count_low(const uint16_t* x, int64_t n, bool vec, int bin, RowShared& sh) {
  if (threadIdx.x < kLow) sh.low[threadIdx.x] = 0u;
  __syncthreads();
  each_key<FP16>(x, kRun * threadIdx.x, n, kRun * kRowThreads, vec, [&](uint32_t key) {
    if (key && (int)(key >> kShift) == bin) atomicAdd(&sh.low[key & (kLow - 1)], 1u);
  });
  __syncthreads();
}

// The cut inside a bin, by the first wave: lane i takes the bin's i-th key from the top, of
// which sh.low columns exist (`have` of them under the cut `within`).  By count: where `left`
// columns are reached; by mass: where the weight `left` is reached.  Nothing changes if it is
// not reached.  *kept: weight of the bin's columns inside a cut by count.
template <class T, class IW>
__device__ inline void cut_bin(int bin, bool by_count, u64 left, Cut within, IW&& int_weight, RowShared& sh,
                               u64 above_mass) {
  if (threadIdx.x >= 64) return;
  const int lane = threadIdx.x;
  const uint32_t key = ((uint32_t)bin << kShift) + (uint32_t)(kLow - 1 - (lane & (kLow - 1)));
  uint32_t have = lane < kLow ? sh.low[key & (kLow - 1)] : 0u;
  have = key < within.t ? 0u : (key == within.t ? min(within.c, have) : have);
  const u64 w = have ? int_weight(key) : 0ull;
  const u64 step = by_count ? (u64)have : have * w;
  u64 incl = step, mass = have * w;
  for (int d = 1; d < 64; d <<= 1) {
    const u64 o = shfl_up64(incl, d), mo = shfl_up64(mass, d);
    if (lane >= d) {
      incl += o;
      mass += mo;
    }
  }
  const u64 before = incl - step;
  if (before < left && incl >= left) {     // one lane at most
    const uint32_t c = by_count ? (uint32_t)(left - before) : (uint32_t)((left - before + w - 1) / w);
    sh.cut = Cut{key, c};
    if (by_count) sh.kept_mass = above_mass + mass - (have - c) * w;
  }
}

template <class T>
__global__ __launch_bounds__(kRowThreads) void row_kernel(const SampleArgs a) {
  constexpr bool FP16 = T::kDtype == 2;
  __shared__ RowShared sh;
  extern __shared__ u64 cand[];            // [kCandidates], then their weights
  float* const rel = (float*)(cand + kCandidates);
  const int64_t row = blockIdx.x;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const RowSpace& s = a.space[row];
  const Row r = row_settings(a, row);
  const RowPlan plan = s.plan;
  const uint32_t found = s.found;
  const uint32_t top_key = (uint32_t)(plan.top >> 32);
  const int mode = plan.mode;
  if (mode == kNothing || mode == kGreedy) {
    if (threadIdx.x == 0) {
      a.out_index[row] = top_key ? (int32_t)(0xFFFFFFFFu - (uint32_t)plan.top) : -1;
      if (a.out_prob) a.out_prob[row] = top_key ? 1.0f : 0.0f;
    }
    return;
  }
  const float top = key_value<T>(top_key);
  const uint16_t* x = (const uint16_t*)a.logits + row * a.row_stride;
  const bool vec = ((uintptr_t)x & 15u) == 0u;
  const bool threshold = mode != kFree;
  const auto int_weight = [&](uint32_t key) { return weight_int(weight<T>(key, top_key, top, r.t)); };
  const uint32_t u_units = min(units_of(a.u[row]), (1u << kUnitBits) - 1u);

  // ---- candidates in LDS: every column that can be drawn, when they fit
  const bool held = threshold && found <= held_limit(mode, r);
  if (held) {
    for (uint32_t i = threadIdx.x; i < found; i += kRowThreads) {
      cand[i] = s.candidate[i];
      rel[i] = s.weight[i];
    }
  }
  // f(key, column, relative weight) for this thread's candidates (at first those that it wrote)
  uint32_t stride = kRowThreads;           // threads that share them
  const auto each_candidate = [&](auto&& f) {
    for (uint32_t i = threadIdx.x; i < found; i += stride) {
      const u64 c = cand[i];
      f((uint32_t)(c >> 32), (uint32_t)c, rel[i]);
    }
  };
  // otherwise the chunks' sums lead to the chunk; only a top-k too wide to be held with a top-p
  // inside it, whose bin the chunks do not know, is drawn from the whole row
  const bool whole = threshold && !held && mode == kByCount && r.units < (1u << kUnitBits);
  const auto low_of = [&](int bin) {
    if (threshold && !held && !whole) {
      if (threadIdx.x < kLow) sh.low[threadIdx.x] = 0u;
      __syncthreads();
      if (bin == plan.low_bin) {           // else min-p cuts above this bin
        for (int c = threadIdx.x / kLow; c < a.chunks; c += kRowThreads / kLow) {
          const uint32_t n = s.chunk_low[c][threadIdx.x % kLow];
          if (n) atomicAdd(&sh.low[threadIdx.x % kLow], n);
        }
      }
      __syncthreads();
      return;
    }
    if (!held) {
      count_low<FP16>(x, a.n, vec, bin, sh);
      return;
    }
    if (threadIdx.x < kLow) sh.low[threadIdx.x] = 0u;
    __syncthreads();
    each_candidate([&](uint32_t key, uint32_t, float) {
      if ((int)(key >> kShift) == bin) atomicAdd(&sh.low[key & (kLow - 1)], 1u);
    });
    __syncthreads();
  };

  // ---- the cut
  Cut cut = {0u, 0u};                      // every key above 0: everything that can be drawn
  if (threshold) {
    if (threadIdx.x == 0) sh.cut = cut;
    if (mode != kAll) {
      low_of(plan.bin);                    // (and a barrier)
      if (mode == kByCount)
        cut_bin<T>(plan.bin, true, r.k - plan.above_count, cut, int_weight, sh, plan.above_mass);
      else
        cut_bin<T>(plan.bin, false, max(1ull, share(plan.total_mass, r.units)) - plan.above_mass, cut, int_weight, sh,
                   0ull);
      __syncthreads();
      cut = sh.cut;
    }
    if (mode == kByCount && r.units < (1u << kUnitBits)) {
      const u64 need = max(1ull, share(sh.kept_mass, r.units));
      int bin = plan.bin;
      u64 above = plan.above_mass;
      __syncthreads();                     // every thread has the cut by count
      if (need <= above) {
        find_bin(s, 0u, [&](u64) { return need; }, sh.search);
        bin = sh.search.bin;
        above = sh.search.above_mass;
        low_of(bin);
      }
      cut_bin<T>(bin, false, need - above, cut, int_weight, sh, 0ull);
      __syncthreads();
      cut = sh.cut;
    }
    if (cut.t < plan.min_key) cut = Cut{plan.min_key - 1u, 0u};   // min-p cuts higher
  }
  const u64 tie_w = cut.c ? int_weight(cut.t) : 0ull;

  if (held) {
    // ---- the draw among the candidates: few of them by one wave, whose barriers wait for
    // nobody (waves that have ended do not count)
    if (found <= kFew) {
      __syncthreads();
      if (wave != 0) return;
      stride = 64u;
    }
    u64 mass = 0;
    uint32_t ties = 0;
    each_candidate([&](uint32_t key, uint32_t, float w) {
      if (key > cut.t) mass += weight_int(w);
      ties += key == cut.t ? 1u : 0u;
    });
    mass = wave_sum64(mass);
    for (int d = 1; d < 64; d <<= 1) ties += __shfl_xor(ties, d);
    if (lane == 0) {
      sh.part_mass[wave] = mass;
      sh.part_ties[wave] = ties;
    }
    __syncthreads();
    mass = 0;
    ties = 0;
    for (uint32_t w = 0; w < stride / 64; ++w) {
      mass += sh.part_mass[w];
      ties += sh.part_ties[w];
    }
    const u64 total = mass + cut.c * tie_w;      // c is at most the number of ties
    u64 target = share(total, u_units);
    // Columns are located six bits of their index at a time, from the highest that n needs.
    int shift0 = 0;
    while ((a.n - 1) >> (shift0 + 6)) shift0 += 6;
    // The last column among the first c ties:
    uint32_t limit = 0xFFFFFFFFu;
    if (cut.c && cut.c < ties) {
      uint32_t left = cut.c;
      limit = 0u;
      for (int shift = shift0; shift >= 0; shift -= 6) {
        if (threadIdx.x < 64) sh.slot_count[threadIdx.x] = 0u;
        __syncthreads();
        each_candidate([&](uint32_t key, uint32_t col, float) {
          if (key == cut.t && (col >> shift >> 6) == limit) atomicAdd(&sh.slot_count[(col >> shift) & 63u], 1u);
        });
        __syncthreads();
        uint32_t incl = sh.slot_count[lane];
        const uint32_t own = incl;
        for (int d = 1; d < 64; d <<= 1) {
          const uint32_t o = __shfl_up(incl, d);
          if (lane >= d) incl += o;
        }
        const int at = __ffsll(__ballot(incl >= left)) - 1;
        left -= __shfl(incl, at) - __shfl(own, at);
        limit = (limit << 6) | (uint32_t)at;
        __syncthreads();
      }
    }
    // The column at which the running sum passes the target:
    uint32_t prefix = 0u;
    u64 last = 0;
    for (int shift = shift0; shift >= 0; shift -= 6) {
      if (threadIdx.x < 64) sh.slot_mass[threadIdx.x] = 0ull;
      __syncthreads();
      each_candidate([&](uint32_t key, uint32_t col, float w) {
        const bool kept = key > cut.t || (key == cut.t && cut.c && col <= limit);
        if (kept && (col >> shift >> 6) == prefix) atomicAdd(&sh.slot_mass[(col >> shift) & 63u], weight_int(w));
      });
      __syncthreads();
      u64 incl = sh.slot_mass[lane];
      const u64 own = incl;
      for (int d = 1; d < 64; d <<= 1) {
        const u64 o = shfl_up64(incl, d);
        if (lane >= d) incl += o;
      }
      const int at = __ffsll(__ballot(incl > target)) - 1;
      const u64 before = incl - own;
      target -= ((u64)__shfl((uint32_t)(before >> 32), at) << 32) | __shfl((uint32_t)before, at);
      last = ((u64)__shfl((uint32_t)(own >> 32), at) << 32) | __shfl((uint32_t)own, at);
      prefix = (prefix << 6) | (uint32_t)at;
      __syncthreads();
    }
    if (threadIdx.x == 0) {
      a.out_index[row] = (int32_t)prefix;
      if (a.out_prob) a.out_prob[row] = (float)((double)last / (double)total);
    }
    return;
  }

  // ---- the draw from the row itself: sums over 16 equal parts of a range, then of the part
  // that holds the target
  const auto above_weight = [&](uint32_t key) -> u64 {
    if (key <= cut.t) return 0ull;
    const float w = weight<T>(key, top_key, top, r.t);
    return threshold || w >= r.min_p ? weight_int(w) : 0ull;   // a cut includes min_p
  };
  bool first = whole;
  if (whole) {
    if (threadIdx.x == 0) {
      sh.begin = 0;
      sh.end = a.n;
      sh.before_mass = 0ull;
      sh.before_ties = 0u;
    }
  } else {
    // each chunk's kept weight but for its ties, and its ties: eight threads per chunk
    if (threadIdx.x == 0) sh.begin = sh.end = 0;
    if (threadIdx.x < kLow) {
      const uint32_t key = ((uint32_t)plan.low_bin << kShift) + threadIdx.x;
      sh.low_weight[threadIdx.x] = threshold && key > cut.t && key <= top_key ? int_weight(key) : 0ull;
    }
    __syncthreads();
    const bool tied = threshold && cut.c && (int)(cut.t >> kShift) == plan.low_bin;
    for (int c = threadIdx.x / 8; c < a.chunks; c += kRowThreads / 8) {
      u64 m = 0;
      if (threshold)
        for (int i = threadIdx.x % 8; i < kLow; i += 8) m += s.chunk_low[c][i] * sh.low_weight[i];
      for (int d = 1; d < 8; d <<= 1) m += shfl_xor64(m, d);
      if (threadIdx.x % 8 == 0) {
        sh.chunk_mass[c] = m + s.chunk_mass[c];
        sh.chunk_ties[c] = tied ? s.chunk_low[c][cut.t & (kLow - 1)] : 0u;
      }
    }
    __syncthreads();
    if (wave == 0) {                       // two chunks per lane
      const int c0 = 2 * lane, c1 = c0 + 1;
      const uint32_t t0 = c0 < a.chunks ? sh.chunk_ties[c0] : 0u, t1 = c1 < a.chunks ? sh.chunk_ties[c1] : 0u;
      uint32_t ti = t0 + t1;
      for (int d = 1; d < 64; d <<= 1) {
        const uint32_t o = __shfl_up(ti, d);
        if (lane >= d) ti += o;
      }
      const uint32_t tb = ti - t0 - t1;    // ties before the lane's chunks
      const auto ties_kept = [&](uint32_t before, uint32_t n) { return min(n, cut.c > before ? cut.c - before : 0u); };
      const u64 m0 = c0 < a.chunks ? sh.chunk_mass[c0] + ties_kept(tb, t0) * tie_w : 0ull;
      const u64 m1 = c1 < a.chunks ? sh.chunk_mass[c1] + ties_kept(tb + t0, t1) * tie_w : 0ull;
      u64 incl = m0 + m1;
      for (int d = 1; d < 64; d <<= 1) {
        const u64 o = shfl_up64(incl, d);
        if (lane >= d) incl += o;
      }
      const u64 total = ((u64)__shfl((uint32_t)(incl >> 32), 63) << 32) | __shfl((uint32_t)incl, 63);
      const u64 target = share(total, u_units), before = incl - m0 - m1;
      if (before <= target && incl > target) {       // one lane
        const bool second = before + m0 <= target;
        sh.begin = (c0 + (second ? 1 : 0)) * a.chunk;
        sh.end = min(a.n, sh.begin + a.chunk);
        sh.before_mass = before + (second ? m0 : 0ull);
        sh.before_ties = tb + (second ? t0 : 0u);
      }
      if (lane == 0) {
        sh.total = total;
        sh.target = target;
      }
    }
  }
  __syncthreads();
  while (first || sh.end - sh.begin > kStep) {
    const int64_t begin = sh.begin, end = sh.end;
    const int64_t part = ((end - begin + kRowWaves - 1) / kRowWaves + kStep - 1) / kStep * kStep;
    const int64_t p0 = begin + wave * part, p1 = min(end, p0 + part);
    u64 mass = 0;
    uint32_t ties = 0;
    each_key<FP16>(x, p0 + kRun * lane, p1, kStep, vec, [&](uint32_t key) {
      if (key == 0u || key < cut.t) return;
      if (key == cut.t)
        ++ties;
      else
        mass += above_weight(key);
    });
    mass = wave_sum64(mass);
    for (int d = 1; d < 64; d <<= 1) ties += __shfl_xor(ties, d);
    if (lane == 0) {
      sh.part_mass[wave] = mass;
      sh.part_ties[wave] = ties;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
      // ties kept in a part: what is left of c after the ties before it
      const auto part_sum = [&](int w, uint32_t before) {
        const uint32_t room = cut.c > before ? cut.c - before : 0u;
        return sh.part_mass[w] + (u64)min(room, sh.part_ties[w]) * tie_w;
      };
      if (first) {
        u64 total = 0;
        uint32_t t = 0;
        for (int w = 0; w < kRowWaves; ++w) {
          total += part_sum(w, t);
          t += sh.part_ties[w];
        }
        sh.total = total;
        sh.target = share(total, u_units);
      }
      u64 before = sh.before_mass;
      uint32_t t = sh.before_ties;
      for (int w = 0; w < kRowWaves; ++w) {
        const u64 m = part_sum(w, t);
        if (before + m > sh.target || w == kRowWaves - 1) {   // (the range shrinks in any case)
          sh.begin = begin + w * part;
          sh.end = min(end, sh.begin + part);
          break;
        }
        before += m;
        t += sh.part_ties[w];
      }
      sh.before_mass = before;
      sh.before_ties = t;
    }
    first = false;
    __syncthreads();
  }

  // ---- one step of columns left: a prefix sum over the lanes of one wave, 8 columns each
  if (wave != 0) return;
  const int64_t i = sh.begin + kRun * lane;
  uint32_t k[kRun], ties = 0;
  load_keys<FP16>(x, i, sh.end, vec, k);
#pragma unroll
  for (int e = 0; e < kRun; ++e) ties += cut.t && k[e] == cut.t ? 1u : 0u;
  uint32_t t = ties;
  for (int d = 1; d < 64; d <<= 1) {
    const uint32_t o = __shfl_up(t, d);
    if (lane >= d) t += o;
  }
  t += sh.before_ties - ties;              // ties before this lane's columns
  u64 w[kRun], mass = 0;
#pragma unroll
  for (int e = 0; e < kRun; ++e) {
    w[e] = 0ull;
    if (k[e] != 0u && k[e] >= cut.t) {
      if (k[e] == cut.t)
        w[e] = t++ < cut.c ? tie_w : 0ull;
      else
        w[e] = above_weight(k[e]);
    }
    mass += w[e];
  }
  u64 incl = mass;
  for (int d = 1; d < 64; d <<= 1) {
    const u64 o = shfl_up64(incl, d);
    if (lane >= d) incl += o;
  }
  u64 before = sh.before_mass + incl - mass;
  if (before > sh.target || before + mass <= sh.target) return;
#pragma unroll
  for (int e = 0; e < kRun; ++e) {
    if (before <= sh.target && before + w[e] > sh.target) {
      a.out_index[row] = (int32_t)(i + e);
      if (a.out_prob) a.out_prob[row] = (float)((double)w[e] / (double)sh.total);
    }
    before += w[e];
  }
}

template <class T>
hipError_t launch(const SampleArgs& a, hipStream_t stream) {
  const dim3 chunks((unsigned)a.chunks, (unsigned)a.rows);
  hipLaunchKernelGGL((chunk_top_kernel<T::kDtype == 2>), chunks, dim3(kChunkThreads), 0, stream, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((chunk_weights_kernel<T>), chunks, dim3(kChunkThreads), 0, stream, a);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((collect_kernel<T>), chunks, dim3(kChunkThreads), 0, stream, a);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  constexpr int kLds = kCandidates * 12;
  e = hipFuncSetAttribute((const void*)row_kernel<T>, hipFuncAttributeMaxDynamicSharedMemorySize, kLds);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((row_kernel<T>), dim3((unsigned)a.rows), dim3(kRowThreads), kLds, stream, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_sample(SampleArgs a, hipStream_t stream) {
  // at most 2048 chunks in all, each of whole 2048-column steps of its workgroup (32 rows of
  // 151936: 1024 chunks leave some CUs four workgroups and others three, 45 us; 2048 40 us;
  // 4096, whose histograms are cleared and joined more often, 49 us)
  const int64_t want = a.rows >= 2048 ? 1 : (2048 / a.rows < kMaxChunks ? 2048 / a.rows : kMaxChunks);
  const int64_t steps = (a.n + kCols - 1) / kCols;
  a.chunk = (steps + want - 1) / want * kCols;
  a.chunks = (int32_t)((a.n + a.chunk - 1) / a.chunk);
  return a.dtype == 1 ? launch<Bf16>(a, stream) : launch<Fp16>(a, stream);
}

}  // namespace sampling
}  // namespace qmm
