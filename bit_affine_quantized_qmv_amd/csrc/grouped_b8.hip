// Matrix products grouped by expert, 8-bit weights.
#include "grouped_impl.hpp"

namespace qmm {
namespace grouped {

hipError_t launch_b8(const Args& a, Kind kind, int dtype, int tile_rows, hipStream_t stream) {
  switch (a.w[0].group_size) {
    case 32: return launch_dtype<8, 32>(a, kind, dtype, tile_rows, stream);
    case 64: return launch_dtype<8, 64>(a, kind, dtype, tile_rows, stream);
    case 128: return launch_dtype<8, 128>(a, kind, dtype, tile_rows, stream);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace grouped
}  // namespace qmm
