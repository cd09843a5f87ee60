// Mixture-of-experts layer, 4-bit expert weights.
#include "moe_impl.hpp"

namespace qmm {
namespace moe {

hipError_t launch_b4(const MoeArgs& a, hipStream_t stream, bool down) { return launch_bits<4>(a, stream, down); }

}  // namespace moe
}  // namespace qmm
