// Matrix products grouped by expert, 2-, 3-, 5- and 6-bit weights.
#include "grouped_impl.hpp"

namespace qmm {
namespace grouped {

hipError_t launch_bn(const Args& a, Kind kind, int dtype, int tile_rows, hipStream_t stream) {
  switch (a.w[0].bits) {
    case 2: return launch_dtype<2, 0>(a, kind, dtype, tile_rows, stream);
    case 3: return launch_dtype<3, 0>(a, kind, dtype, tile_rows, stream);
    case 5: return launch_dtype<5, 0>(a, kind, dtype, tile_rows, stream);
    case 6: return launch_dtype<6, 0>(a, kind, dtype, tile_rows, stream);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace grouped
}  // namespace qmm
