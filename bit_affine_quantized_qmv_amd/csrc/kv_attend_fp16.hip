// Attention over the 4-bit key/value cache, fp16 instantiations.
#include "kv_attend_impl.hpp"

namespace qmm {
namespace kv {

hipError_t launch_attend_fp16(const AttendArgs& a, const AttendPlan& p, hipStream_t stream) {
  return launch_attend<Fp16>(a, p, stream);
}

}  // namespace kv
}  // namespace qmm
