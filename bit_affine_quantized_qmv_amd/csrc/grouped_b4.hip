// Matrix products grouped by expert, 4-bit weights.
#include "grouped_impl.hpp"

namespace qmm {
namespace grouped {

hipError_t launch_b4(const Args& a, Kind kind, int dtype, int tile_rows, hipStream_t stream) {
  switch (a.w[0].group_size) {
    case 32: return launch_dtype<4, 32>(a, kind, dtype, tile_rows, stream);
    case 64: return launch_dtype<4, 64>(a, kind, dtype, tile_rows, stream);
    case 128: return launch_dtype<4, 128>(a, kind, dtype, tile_rows, stream);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace grouped
}  // namespace qmm
