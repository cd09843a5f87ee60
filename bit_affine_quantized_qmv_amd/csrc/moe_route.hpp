// Order of router logits, shared by the expert layers.
#pragma once

#include "device_common.hpp"
#include "moe.hpp"

namespace qmm {
namespace moe {

// Order key of a 16-bit float: larger values have larger keys, NaN the largest.
template <class T>
__device__ inline uint32_t order_key(uint32_t b) {
  constexpr uint32_t kInf = T::kDtype == 2 ? 0x7C00u : 0x7F80u;
  if ((b & 0x7FFFu) > kInf) return 0xFFFFu;
  if (b == 0x8000u) b = 0u;                     // -0 and +0 are equal
  return (b & 0x8000u) ? (~b & 0xFFFFu) : (b | 0x8000u);
}

// Largest v of the wave, in every lane: row-local steps, then the row broadcasts.
__device__ inline uint32_t wave_max(uint32_t v) {
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, false));    // quad_perm [1,0,3,2]
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, false));    // quad_perm [2,3,0,1]
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x141, 0xF, 0xF, false));   // row_half_mirror
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x140, 0xF, 0xF, false));   // row_mirror
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x142, 0xA, 0xF, false));   // row_bcast:15
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x143, 0xC, 0xF, false));   // row_bcast:31
  return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

}  // namespace moe
}  // namespace qmm
