// Launch interface of the mixture-of-experts layer for a few tokens.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/qmm.h"

namespace qmm {
namespace moe {

constexpr int kMaxTokens = 32;
constexpr int kMaxExperts = 512;
constexpr int kMaxTopK = 32;
constexpr int kWaves = 4;             // per workgroup
constexpr int kMaxSplits = 16;
constexpr int kXBytes = 40 * 1024;    // LDS of the staged activations: three workgroups per CU fit (with 48 KB, two)

// How a row of K is walked, in slots (spans of K that one round of loads covers).  A workgroup's
// walk starts at an even slot and goes on in chunks, what LDS holds of the activations; in a
// chunk each of the `parts` waves of a tile takes a stretch, in rounds of its ring of loads.
// Starts, chunks, stretches and rounds are all even: a round's scales are one load, which has
// to start on a word also where a slot has one scale of two bytes.

// Slots of a chunk: whole rounds of all parts where LDS holds them, else what it holds.
// slot_entries: 16-byte entries of a slot per row, of all operand planes; 2^xrl rows; round: parts
// times the ring's slots.
__host__ __device__ constexpr int chunk_of(int slot_entries, int xrl, int round) {
  const int fit = kXBytes / 16 / (slot_entries << xrl);
  return fit >= round ? fit / round * round : fit & ~1;
}
// Slots of one part of n.
__host__ __device__ constexpr int stretch_of(int n, int parts) { return ((n + parts - 1) / parts + 1) & ~1; }

// A stack of quantized weights, [experts][N][K].
struct Stack {
  const uint32_t* w;
  int64_t w_row_stride;      // words
  int64_t w_expert_stride;
  const uint16_t* s;
  const uint16_t* b;
  int64_t sb_row_stride;     // elements
  int64_t sb_expert_stride;
  int32_t bits;
  int32_t group_size;
};

struct MoeArgs {
  const uint16_t* x;         // [tokens, x_stride]
  int64_t x_stride;
  const uint16_t* router;    // [tokens, router_stride]
  int64_t router_stride;
  int32_t tokens;
  int32_t experts;
  int32_t top_k;
  int32_t renormalize;
  int32_t hidden;
  int32_t inter;
  int32_t dtype;
  Stack gate, up, down;
  uint16_t* y;               // [tokens, y_stride]
  int64_t y_stride;
  // workspace
  int32_t* pair_expert;      // [tokens * top_k]: pair t * top_k + i is token t's i-th largest router logit
  float* pair_share;         // [tokens * top_k]: its unnormalised weight
  uint16_t* h;               // [tokens * top_k][2][inter]: silu(gate) * up in bfloat16, leading bits and the rest
  float* out;                // [tokens * top_k][splits][hidden]: each pair's product with down
  // waves that share one tile, each a part of K, and workgroups per expert, in the first and
  // the second kernel; stretches of K that different workgroups of the second kernel take
  int32_t parts, down_parts, blocks, down_blocks, splits;
};

// Validate one stack of an expert layer (host only): [n, cols] per expert, of dtype.
int32_t check_stack(const char* name, const qmm_expert_stack_t* k, int64_t n, int64_t cols, int32_t experts, int32_t dtype,
                    Stack* out);

hipError_t launch_b4(const MoeArgs& a, hipStream_t stream, bool down);
hipError_t launch_b8(const MoeArgs& a, hipStream_t stream, bool down);
hipError_t launch_bn(const MoeArgs& a, hipStream_t stream, bool down);
hipError_t launch_sum(const MoeArgs& a, hipStream_t stream);

}  // namespace moe
}  // namespace qmm
