// Launch interface of the mixture-of-experts layer for a few tokens.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace qmm {
namespace moe {

constexpr int kMaxTokens = 32;
constexpr int kMaxExperts = 512;
constexpr int kMaxTopK = 32;

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
  int32_t* active;           // [1 + experts]: number of experts in use, then their indices, ascending
  int16_t* row_of;           // [experts in use][kMaxTokens]: row of h of the token with this expert, or -1
  uint16_t* h;               // [tokens * top_k][inter]: w * silu(gate) * up
  float* part;               // [splits][tokens][hidden] sums of the second kernel's splits
  // launch shape
  int32_t parts;             // waves that share one tile of the first kernel, each a part of K
  int32_t splits;            // workgroups that share one tile of the second kernel
  int32_t cuts;              // pieces of each expert's K in the second kernel
};

hipError_t launch_b4(const MoeArgs& a, hipStream_t stream, bool down);
hipError_t launch_b8(const MoeArgs& a, hipStream_t stream, bool down);
hipError_t launch_bn(const MoeArgs& a, hipStream_t stream, bool down);
hipError_t launch_join(const MoeArgs& a, hipStream_t stream);

}  // namespace moe
}  // namespace qmm
