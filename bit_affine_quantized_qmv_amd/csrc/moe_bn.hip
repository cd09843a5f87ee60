// Mixture-of-experts layer, 2-, 3-, 5- and 6-bit expert weights, and the join of the second
// kernel's splits.
#include "moe_impl.hpp"

namespace qmm {
namespace moe {

hipError_t launch_bn(const MoeArgs& a, hipStream_t stream, bool down) {
  switch (down ? a.down.bits : a.gate.bits) {
    case 2: return launch_bits<2>(a, stream, down);
    case 3: return launch_bits<3>(a, stream, down);
    case 5: return launch_bits<5>(a, stream, down);
    case 6: return launch_bits<6>(a, stream, down);
    default: return hipErrorInvalidValue;
  }
}

namespace {

constexpr int kJoinThreads = 256;

// y = the splits' sums added in split order, rounded to dtype.
template <class T>
__global__ __launch_bounds__(kJoinThreads) void join_kernel(const MoeArgs a) {
  const int64_t i = (int64_t)blockIdx.x * kJoinThreads + threadIdx.x;
  const int64_t n = (int64_t)a.tokens * a.hidden;
  if (i >= n) return;
  float v = 0.f;
  for (int s = 0; s < a.splits; ++s) v += a.part[s * n + i];
  const int64_t t = i / a.hidden;
  a.y[t * a.y_stride + (i - t * a.hidden)] = T::from_f32(v);
}

}  // namespace

hipError_t launch_join(const MoeArgs& a, hipStream_t stream) {
  const dim3 grid((unsigned)(((int64_t)a.tokens * a.hidden + kJoinThreads - 1) / kJoinThreads));
  if (a.dtype == 1)
    hipLaunchKernelGGL(join_kernel<Bf16>, grid, dim3(kJoinThreads), 0, stream, a);
  else
    hipLaunchKernelGGL(join_kernel<Fp16>, grid, dim3(kJoinThreads), 0, stream, a);
  return hipGetLastError();
}

}  // namespace moe
}  // namespace qmm
