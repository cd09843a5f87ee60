// Mixture-of-experts layer, 2-, 3-, 5- and 6-bit expert weights, and the sum over a
// token's choices.
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

constexpr int kSumThreads = 256;

// y_t = sum of t's pairs, each by its share, in the order of its choices, rounded to dtype.
template <class T>
__global__ __launch_bounds__(kSumThreads) void sum_kernel(const MoeArgs a) {
  const int n = (int)(blockIdx.x * kSumThreads + threadIdx.x), t = blockIdx.y;
  if (n >= a.hidden) return;
  const float* o = a.out + (int64_t)t * a.top_k * a.splits * a.hidden + n;
  const float* share = a.pair_share + t * a.top_k;
  float v = 0.f, sum = 0.f;
  constexpr int kAhead = 8;          // choices whose loads are in flight together
  for (int i0 = 0; i0 < a.top_k; i0 += kAhead) {
    float w[kAhead] = {}, f[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) f[i] = i0 + i < a.top_k ? share[i0 + i] : 0.f;
    for (int z = 0; z < a.splits; ++z)
#pragma unroll
      for (int i = 0; i < kAhead; ++i) w[i] += o[(int64_t)(min(i0 + i, a.top_k - 1) * a.splits + z) * a.hidden];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (i0 + i >= a.top_k) break;
      v = __builtin_fmaf(f[i], w[i], v);
      sum += f[i];
    }
  }
  a.y[t * a.y_stride + n] = T::from_f32(a.renormalize ? v / sum : v);
}

}  // namespace

hipError_t launch_sum(const MoeArgs& a, hipStream_t stream) {
  const dim3 grid((unsigned)((a.hidden + kSumThreads - 1) / kSumThreads), (unsigned)a.tokens);
  if (a.dtype == 1)
    hipLaunchKernelGGL(sum_kernel<Bf16>, grid, dim3(kSumThreads), 0, stream, a);
  else
    hipLaunchKernelGGL(sum_kernel<Fp16>, grid, dim3(kSumThreads), 0, stream, a);
  return hipGetLastError();
}

}  // namespace moe
}  // namespace qmm
