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
// Three kernels, because the weights need the row's maximum and the histogram needs the whole
// row: (1) each chunk's largest key and its first column; (2) each chunk's weights, into the
// row's histogram or, for a row without top-k and top-p, as the chunk's sum; (3) one workgroup
// per row finds the threshold and draws.
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
constexpr int kUnitBits = 24;        // u and top_p count in units of 2^-24
constexpr int kRun = 8;              // consecutive columns per lane and step
constexpr int kStep = 64 * kRun;     // columns per wave and step

// Order key of a 16-bit logit: larger logits have larger keys, NaN and -inf (never drawn) 0.
template <bool FP16>
__device__ inline uint32_t key_of(uint32_t b) {
  constexpr uint32_t kInf = FP16 ? 0x7C00u : 0x7F80u;
  if ((b & 0x7FFFu) > kInf || b == (0x8000u | kInf)) return 0u;
  if (b == 0x8000u) b = 0u;          // -0 draws like +0
  return (b & 0x8000u) ? (~b & 0xFFFFu) : (b | 0x8000u);
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
  const uint16_t* x = (const uint16_t*)a.logits + row * a.row_stride;
  const bool vec = ((uintptr_t)x & 15u) == 0u;
  const int64_t begin = chunk * a.chunk, end = min(a.n, begin + a.chunk);
  u64 top = 0;
  for (int64_t i = begin + kRun * threadIdx.x; i < end; i += kRun * kChunkThreads) {
    uint32_t k[kRun];
    load_keys<FP16>(x, i, end, vec, k);
#pragma unroll
    for (int e = 0; e < kRun; ++e) {
      const u64 w = k[e] ? ((u64)k[e] << 32) | (0xFFFFFFFFu - (uint32_t)(i + e)) : 0ull;
      top = w > top ? w : top;
    }
  }
  top = wave_max64(top);
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
  const uint16_t* x = (const uint16_t*)a.logits + row * a.row_stride;
  const bool vec = ((uintptr_t)x & 15u) == 0u;
  const int64_t begin = chunk * a.chunk, end = min(a.n, begin + a.chunk);
  u64 sum = 0;
  for (int64_t i = begin + kRun * threadIdx.x; i < end; i += kRun * kChunkThreads) {
    uint32_t k[kRun];
    load_keys<FP16>(x, i, end, vec, k);
#pragma unroll
    for (int e = 0; e < kRun; ++e) {
      if (k[e] == 0u) continue;
      const float w = weight<T>(k[e], top_key, top, r.t);
      if (threshold) {
        atomicAdd(&mass[k[e] >> kShift], weight_int(w));
        atomicAdd(&count[k[e] >> kShift], 1u);
      } else if (w >= r.min_p) {
        sum += weight_int(w);
      }
    }
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

// What a row keeps: keys above t, and the first c columns with key t.
struct Cut {
  uint32_t t;
  uint32_t c;
};

// Shared state of the row kernel.
struct RowShared {
  u64 scan_mass[kRowWaves];
  uint32_t scan_count[kRowWaves];
  uint32_t low[kLow];
  u64 part_mass[kRowWaves];
  uint32_t part_ties[kRowWaves];
  // results that one thread finds and all read
  int bin;
  u64 above_mass;
  uint32_t above_count;
  Cut cut;
  u64 kept_mass;
  int64_t begin, end;
  u64 target, before_mass, total;
  uint32_t before_ties;
};

// The bin (from the top) in which the running count reaches `want_count` or, when that is 0,
// the running mass reaches `want_mass`; with the count and mass of the bins above it.  Thread
// i owns bins 2047 - 2i and 2046 - 2i, so thread order is descending.  bin = -1: not reached.
__device__ inline void find_bin(const RowSpace& s, uint32_t want_count, u64 want_mass, RowShared& sh) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int b0 = kBins - 1 - 2 * threadIdx.x;
  const u64 m0 = s.mass[b0], m1 = s.mass[b0 - 1];
  const uint32_t n0 = s.count[b0], n1 = s.count[b0 - 1];
  u64 m = m0 + m1;
  uint32_t n = n0 + n1;
  for (int d = 1; d < 64; d <<= 1) {
    const u64 mo = shfl_up64(m, d);
    const uint32_t no = __shfl_up(n, d);
    if (lane >= d) {
      m += mo;
      n += no;
    }
  }
  if (threadIdx.x == 0) sh.bin = -1;
  if (lane == 63) {
    sh.scan_mass[wave] = m;
    sh.scan_count[wave] = n;
  }
  __syncthreads();
  u64 mb = m - m0 - m1;
  uint32_t nb = n - n0 - n1;
  for (int w = 0; w < wave; ++w) {
    mb += sh.scan_mass[w];
    nb += sh.scan_count[w];
  }
  const auto crosses = [&](u64 mass_b, uint32_t count_b, u64 mm, uint32_t nn) {
    return want_count ? (count_b < want_count && count_b + nn >= want_count)
                      : (mass_b < want_mass && mass_b + mm >= want_mass);
  };
  if (crosses(mb, nb, m0, n0)) {
    sh.bin = b0;
    sh.above_mass = mb;
    sh.above_count = nb;
  } else if (crosses(mb + m0, nb + n0, m1, n1)) {
    sh.bin = b0 - 1;
    sh.above_mass = mb + m0;
    sh.above_count = nb + n0;
  }
  __syncthreads();
}

// Columns of each key of one bin, into sh.low.
template <bool FP16>
__device__ inline void count_low(const uint16_t* x, int64_t n, bool vec, int bin, RowShared& sh) {
  if (threadIdx.x < kLow) sh.low[threadIdx.x] = 0u;
  __syncthreads();
  for (int64_t i = kRun * threadIdx.x; i < n; i += kRun * kRowThreads) {
    uint32_t k[kRun];
    load_keys<FP16>(x, i, n, vec, k);
#pragma unroll
    for (int e = 0; e < kRun; ++e)
      if (k[e] && (int)(k[e] >> kShift) == bin) atomicAdd(&sh.low[k[e] & (kLow - 1)], 1u);
  }
  __syncthreads();
}

template <class T>
__global__ __launch_bounds__(kRowThreads) void row_kernel(const SampleArgs a) {
  constexpr bool FP16 = T::kDtype == 2;
  __shared__ RowShared sh;
  const int64_t row = blockIdx.x;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const RowSpace& s = a.space[row];
  const Row r = row_settings(a, row);
  const u64 top_word = row_top(s, a.chunks, lane);
  const uint32_t top_key = (uint32_t)(top_word >> 32);
  if (top_key == 0u || r.greedy) {
    if (threadIdx.x == 0) {
      a.out_index[row] = top_key ? (int32_t)(0xFFFFFFFFu - (uint32_t)top_word) : -1;
      if (a.out_prob) a.out_prob[row] = top_key ? 1.0f : 0.0f;
    }
    return;
  }
  const float top = key_value<T>(top_key);
  const uint16_t* x = (const uint16_t*)a.logits + row * a.row_stride;
  const bool vec = ((uintptr_t)x & 15u) == 0u;
  const auto int_weight = [&](uint32_t key) { return weight_int(weight<T>(key, top_key, top, r.t)); };

  // ---- the cut
  const bool threshold = r.threshold();
  Cut cut = {0u, 0u};                      // every key above 0: everything that can be drawn
  if (threshold) {
    int k_bin = -1;
    u64 k_above = 0;
    if (r.k) {
      find_bin(s, r.k, 0ull, sh);
      k_bin = sh.bin;                      // -1: fewer than k columns can be drawn
      k_above = sh.above_mass;
    }
    if (k_bin >= 0) {
      count_low<FP16>(x, a.n, vec, k_bin, sh);
      if (threadIdx.x == 0) {
        uint32_t left = r.k - sh.above_count;
        u64 kept = sh.above_mass;
        for (int i = kLow - 1; i >= 0; --i) {
          const uint32_t key = (uint32_t)(k_bin << kShift) + i, have = min(left, sh.low[i]);
          if (have == 0u) continue;
          kept += have * int_weight(key);
          left -= have;
          if (left == 0u) {
            sh.cut = Cut{key, have};
            break;
          }
        }
        sh.kept_mass = kept;
      }
    } else {
      u64 m = 0;
      for (int i = threadIdx.x; i < kBins; i += kRowThreads) m += s.mass[i];
      m = wave_sum64(m);
      if (lane == 0) sh.part_mass[wave] = m;
      __syncthreads();
      if (threadIdx.x == 0) {
        m = 0;
        for (int w = 0; w < kRowWaves; ++w) m += sh.part_mass[w];
        sh.kept_mass = m;
        sh.cut = cut;
      }
    }
    __syncthreads();
    cut = sh.cut;
    const u64 kept = sh.kept_mass;
    __syncthreads();                       // every thread has them before sh.cut changes
    if (r.units < (1u << kUnitBits)) {
      u64 need = share(kept, r.units);
      need = need ? need : 1ull;           // the first column always stays
      int bin = k_bin;
      u64 above = k_above;
      if (k_bin < 0 || need <= k_above) {
        find_bin(s, 0u, need, sh);
        bin = sh.bin;
        above = sh.above_mass;
        count_low<FP16>(x, a.n, vec, bin, sh);
      }
      if (threadIdx.x == 0) {
        u64 left = need - above;
        for (int i = kLow - 1; i >= 0; --i) {
          const uint32_t key = (uint32_t)(bin << kShift) + i;
          const uint32_t have = key < cut.t ? 0u : (key == cut.t ? min(cut.c, sh.low[i]) : sh.low[i]);
          const u64 w = have ? int_weight(key) : 0ull;
          if (w == 0ull) continue;
          if (left <= have * w) {
            sh.cut = Cut{key, (uint32_t)((left + w - 1) / w)};
            break;
          }
          left -= have * w;
        }
      }
      __syncthreads();
      cut = sh.cut;
    }
  }

  // ---- the draw: sums over 16 equal parts of a range, then of the part that holds the target
  const float tie_rel = cut.t ? weight<T>(cut.t, top_key, top, r.t) : 0.0f;
  const u64 tie_w = tie_rel >= r.min_p ? weight_int(tie_rel) : 0ull;
  const auto above_weight = [&](uint32_t key) -> u64 {
    if (key <= cut.t) return 0ull;
    const float w = weight<T>(key, top_key, top, r.t);
    return w >= r.min_p ? weight_int(w) : 0ull;
  };
  bool first = true;
  if (threadIdx.x == 0) {
    sh.begin = 0;
    sh.end = a.n;
    sh.before_mass = 0ull;
    sh.before_ties = 0u;
    if (!threshold) {                      // the chunks' sums are there already
      u64 total = 0;
      for (int c = 0; c < a.chunks; ++c) total += s.chunk_mass[c];
      sh.total = total;
      sh.target = share(total, min(units_of(a.u[row]), (1u << kUnitBits) - 1u));
      u64 before = 0;
      for (int c = 0; c < a.chunks; ++c) {
        const u64 m = s.chunk_mass[c];
        if (before + m > sh.target) {
          sh.begin = c * a.chunk;
          sh.end = min(a.n, sh.begin + a.chunk);
          break;
        }
        before += m;
      }
      sh.before_mass = before;
    }
  }
  if (!threshold) first = false;
  __syncthreads();
  while (first || sh.end - sh.begin > kStep) {
    const int64_t begin = sh.begin, end = sh.end;
    const int64_t part = ((end - begin + kRowWaves - 1) / kRowWaves + kStep - 1) / kStep * kStep;
    const int64_t p0 = begin + wave * part, p1 = min(end, p0 + part);
    u64 mass = 0;
    uint32_t ties = 0;
    for (int64_t i = p0 + kRun * lane; i < p1; i += kStep) {
      uint32_t k[kRun];
      load_keys<FP16>(x, i, p1, vec, k);
#pragma unroll
      for (int e = 0; e < kRun; ++e) {
        if (k[e] == 0u || k[e] < cut.t) continue;
        if (k[e] == cut.t)
          ++ties;
        else
          mass += above_weight(k[e]);
      }
    }
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
        sh.target = share(total, min(units_of(a.u[row]), (1u << kUnitBits) - 1u));
      }
      u64 before = sh.before_mass;
      uint32_t t = sh.before_ties;
      for (int w = 0; w < kRowWaves; ++w) {
        const u64 m = part_sum(w, t);
        if (before + m > sh.target) {
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
  hipLaunchKernelGGL((row_kernel<T>), dim3((unsigned)a.rows), dim3(kRowThreads), 0, stream, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_sample(SampleArgs a, hipStream_t stream) {
  // about 1024 chunks in all, each of whole 2048-column steps of its workgroup
  constexpr int64_t kCols = kRun * kChunkThreads;
  const int64_t want = a.rows >= 1024 ? 1 : (1024 / a.rows < kMaxChunks ? 1024 / a.rows : kMaxChunks);
  const int64_t steps = (a.n + kCols - 1) / kCols;
  a.chunk = (steps + want - 1) / want * kCols;
  a.chunks = (int32_t)((a.n + a.chunk - 1) / a.chunk);
  return a.dtype == 1 ? launch<Bf16>(a, stream) : launch<Fp16>(a, stream);
}

}  // namespace sampling
}  // namespace qmm
