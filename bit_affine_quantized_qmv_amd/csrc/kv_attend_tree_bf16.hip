// Attention of drafted trees over the 4-bit key/value cache, bf16 instantiations.
#include "kv_attend_impl.hpp"

namespace qmm {
namespace kv {

hipError_t launch_attend_tree_bf16(const AttendArgs& a, const AttendPlan& p, hipStream_t stream) {
  return launch_attend<Bf16, true>(a, p, stream);
}

}  // namespace kv
}  // namespace qmm
