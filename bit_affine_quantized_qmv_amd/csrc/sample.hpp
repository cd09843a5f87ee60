// Launch interface of sampling from stored logits.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace qmm {
namespace sampling {

constexpr int kBins = 2048;         // values of an order key's high 11 bits
constexpr int kMaxChunks = 128;     // column chunks per row

// Workspace of one row.  Every word is written by the call before it is read.
struct RowSpace {
  unsigned long long mass[kBins];            // sum of the weights of each bin
  unsigned long long chunk_mass[kMaxChunks]; // sum of the weights of each chunk (rows without a threshold)
  unsigned long long top[kMaxChunks];        // each chunk's largest (key << 32 | ~column), 0: nothing to draw
  uint32_t count[kBins];
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
