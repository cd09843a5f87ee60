// Mixture-of-experts layer, 8-bit expert weights.
#include "moe_impl.hpp"

namespace qmm {
namespace moe {

hipError_t launch_b8(const MoeArgs& a, hipStream_t stream, bool down) { return launch_bits<8>(a, stream, down); }

}  // namespace moe
}  // namespace qmm
