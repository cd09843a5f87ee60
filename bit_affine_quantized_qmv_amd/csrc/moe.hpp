// Launch interface of the mixture-of-experts layer for a few tokens.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace qmm {
namespace moe {

constexpr int kMaxTokens = 32;
constexpr int kMaxExperts = 512;
constexpr int kMaxTopK = 32;
constexpr int kWaves = 4;             // per workgroup
constexpr int kMaxSplits = 16;

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

hipError_t launch_b4(const MoeArgs& a, hipStream_t stream, bool down);
hipError_t launch_b8(const MoeArgs& a, hipStream_t stream, bool down);
hipError_t launch_bn(const MoeArgs& a, hipStream_t stream, bool down);
hipError_t launch_sum(const MoeArgs& a, hipStream_t stream);

}  // namespace moe
}  // namespace qmm
