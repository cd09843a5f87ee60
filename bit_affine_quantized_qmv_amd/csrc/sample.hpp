// Launch interface of sampling from stored logits.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace qmm {
namespace sampling {

constexpr int kBins = 2048;         // values of an order key's high 11 bits
constexpr int kMaxChunks = 128;     // column chunks per row

constexpr int kCandidates = 12288;  // columns of a row that the last kernel holds in LDS, at most

// How a row's column is drawn.
enum RowMode : int32_t {
  kNothing,    // no column can be drawn
  kGreedy,     // the first largest
  kFree,       // any column, by the chunks' sums (no threshold but min-p)
  kAll,        // any column above min-p (a top-k that reaches every column)
  kByCount,    // top-k, then top-p inside it
  kByMass      // top-p
};

// What is known of a row before its draw.
struct RowPlan {
  unsigned long long top;                    // (largest key << 32 | ~its first column)
  unsigned long long above_mass, total_mass; // weight above the threshold's bin, of all columns
  uint32_t above_count;
  int32_t mode, bin;
  int32_t low_bin;                           // bin, or the bin of min_key where that is higher (not with top-p inside top-k)
  uint32_t min_key;                          // smallest key whose weight reaches min_p
  uint32_t pad;
};

// Workspace of one row.  Every word is written by the call before it is read.
struct RowSpace {
  unsigned long long mass[kBins];            // sum of the weights of each bin
  unsigned long long chunk_mass[kMaxChunks]; // sum of each chunk's weights (kFree), of those above low_bin (others)
  uint32_t chunk_low[kMaxChunks][1 << (16 - 11)];   // each chunk's columns of each key of low_bin (not kFree)
  unsigned long long top[kMaxChunks];        // each chunk's largest (key << 32 | ~column), 0: nothing to draw
  uint32_t count[kBins];
  RowPlan plan;
  uint32_t found;                            // candidates; more than the row is drawn from: they are incomplete
  uint32_t pad;
  unsigned long long candidate[kCandidates]; // key << 32 | column, in any order
  float weight[kCandidates];                 // their relative weights
};

// One value per row: an array, or the same number for every row.
template <class V>
struct PerRow {
  const V* array;
  V value;
  __device__ V get(int64_t row) const { return array ? array[row] : value; }
};

struct SampleArgs {
  const void* logits;   // [rows, row_stride] of dtype
  int64_t rows;
  int64_t n;
  int64_t row_stride;
  int32_t dtype;
  const float* u;
  PerRow<float> temperature, top_p, min_p;
  PerRow<int32_t> top_k;
  int32_t* out_index;
  float* out_prob;      // or null
  RowSpace* space;
  int64_t chunk;        // columns per chunk
  int32_t chunks;
};

hipError_t launch_sample(SampleArgs a, hipStream_t stream);

}  // namespace sampling
}  // namespace qmm
