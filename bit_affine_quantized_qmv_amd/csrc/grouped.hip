// What comes before the products grouped by expert: sums of activation groups, the rows of every
// expert, and their tiles.
#include "grouped_impl.hpp"
#include "moe_route.hpp"

namespace qmm {
namespace grouped {
namespace {

// Sums of the groups of 2048 elements of a row (thread `at` of 256 has eight of them), in three
// bfloat16 parts; the groups that a row is padded to are zero.  float32, eight in order, then the
// lanes in pairs.  Bound by memory.
template <class T>
__device__ inline void group_sums_of(const PrepareArgs& a, int64_t block, int at) {
  const int per_row = (a.sum_groups * a.group + 8 * kThreads - 1) / (8 * kThreads);
  const int64_t row = block / per_row;
  const int k = (int)(block - row * per_row) * 8 * kThreads + 8 * at;
  float sum = 0.f;
  if (k < a.k) {
    const u32x4 u = *(const u32x4*)(a.x + row * a.x_stride + k);
#pragma unroll
    for (int e = 0; e < 4; ++e) sum += T::to_f32(u[e] & 0xFFFFu) + T::to_f32(u[e] >> 16);
  }
  sum += __shfl_xor(sum, 1);
  sum += __shfl_xor(sum, 2);
  if (a.group >= 64) sum += __shfl_xor(sum, 4);
  if (a.group == 128) sum += __shfl_xor(sum, 8);
  const int g = k / a.group;
  if (k % a.group == 0 && g < a.sum_groups)
    store_sum(a.sums + row * kPlanes * a.sum_groups + g, a.sum_groups, sum);
}

__device__ inline int64_t sum_blocks(const PrepareArgs& a) {
  return a.rows * ((a.sum_groups * a.group + 8 * kThreads - 1) / (8 * kThreads));
}

// Inclusive prefix of one number per thread of the first 512, over the workgroup (kMake threads).
constexpr int kMake = 1024;
__device__ inline int block_prefix(int v, int* lds) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int o = __shfl_up(v, d);
    v += lane >= d ? o : 0;
  }
  __syncthreads();
  if (lane == 63) lds[wave] = v;
  __syncthreads();
  for (int w = 0; w < wave; ++w) v += lds[w];
  return v;
}

// Tiles of at most tile_rows rows; thread e has expert e's rows [begin, begin + count).
__device__ inline void make_tiles(int begin, int count, int tile_rows, Tile* tiles, int max_tiles, int* tile_count,
                                  int* lds) {
  const int n = (count + tile_rows - 1) / tile_rows;
  const int end = block_prefix(n, lds);
  for (int i = 0; i < n; ++i) {
    const int at = end - n + i;
    if (at < max_tiles)
      tiles[at] = Tile{(int)threadIdx.x, begin + i * tile_rows, min(tile_rows, count - i * tile_rows), 0};
  }
  if (threadIdx.x == kMake - 1) *tile_count = min(end, max_tiles);
}

// Tiles of given offsets, by the last workgroup; the sums by the others.  An expert's rows start
// where all before it have ended, whatever the offsets are.
template <class T>
__global__ __launch_bounds__(kMake) void prepare_kernel(const PrepareArgs a) {
  __shared__ int lds[kMake / 64];
  __shared__ int most[kMake / 64];
  if (blockIdx.x + 1 < gridDim.x) {
    const int64_t block = (int64_t)blockIdx.x * (kMake / kThreads) + threadIdx.x / kThreads;
    if (block < sum_blocks(a)) group_sums_of<T>(a, block, threadIdx.x % kThreads);
    return;
  }
  const int e = threadIdx.x;
  const auto at = [&](int i) { return (int)min(max((int64_t)a.offsets[i], (int64_t)0), a.rows); };
  // largest of the offsets up to this one
  int top = e <= a.experts && e < kMake ? at(min(e, a.experts)) : 0;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int o = __shfl_up(top, d);
    top = (threadIdx.x & 63) >= d ? max(top, o) : top;
  }
  if ((e & 63) == 63) most[e >> 6] = top;
  __syncthreads();
  for (int w = 0; w < (e >> 6); ++w) top = max(top, most[w]);
  const int count = e < a.experts ? max(0, at(e + 1) - top) : 0;
  make_tiles(top, count, a.tile_rows, a.tiles, a.max_tiles, a.tile_count, lds);
}

// A token's choices, largest first, and their weights exp(l - max l) (over the sum of all experts
// unless renormalised), by one wave; the sums of the activations' groups by the other workgroups.
template <class T>
__global__ __launch_bounds__(kThreads) void route_kernel(const RouteArgs a, const PrepareArgs p, const int route_blocks) {
  if ((int)blockIdx.x >= route_blocks) {
    group_sums_of<T>(p, (int64_t)blockIdx.x - route_blocks, threadIdx.x);
    return;
  }
  const int lane = threadIdx.x & 63, t = blockIdx.x * (kThreads / 64) + (threadIdx.x >> 6);
  if (t >= a.tokens) return;
  const uint16_t* logits = a.router + t * a.router_stride;
  constexpr int kRegs = moe::kMaxExperts / 64;
  uint32_t word[kRegs];
#pragma unroll
  for (int j = 0; j < kRegs; ++j) {
    const int e = 64 * j + lane;
    word[j] = e < a.experts ? (moe::order_key<T>(logits[e]) << 9) | (uint32_t)(moe::kMaxExperts - 1 - e) : 0u;
  }
  const auto logit = [](uint32_t key) { return T::to_f32((key & 0x8000u) ? (key & 0x7FFFu) : (~key & 0xFFFFu)); };
  uint32_t best = 0xFFFFFFFFu;
  float top = 0.f, sum = 1.f;
  for (int i = 0; i < a.top_k; ++i) {
    uint32_t m = 0u;
#pragma unroll
    for (int j = 0; j < kRegs; ++j) m = word[j] < best ? max(m, word[j]) : m;
    best = moe::wave_max(m);
    const float l = logit(best >> 9);
    if (i == 0) {
      top = l;
      if (!a.renormalize) {
        sum = 0.f;
#pragma unroll
        for (int j = 0; j < kRegs; ++j) sum += 64 * j + lane < a.experts ? expf(logit(word[j] >> 9) - top) : 0.f;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) sum += __shfl_xor(sum, d);
      }
    }
    if (lane == 0) {
      a.pair_expert[t * a.top_k + i] = moe::kMaxExperts - 1 - (int)(best & (moe::kMaxExperts - 1));
      a.pair_share[t * a.top_k + i] = expf(l - top) / sum;
    }
  }
}

// Rows of every expert, by one workgroup: counts, their prefix, and each pair's place.  The order
// of an expert's rows is that of the atomics, and no result depends on it: a row's sums are its own.
__global__ __launch_bounds__(kMake) void list_kernel(const RouteArgs a) {
  __shared__ int count[moe::kMaxExperts];
  __shared__ int lds[kMake / 64];
  const int pairs = a.tokens * a.top_k, e = threadIdx.x;
  if (e < moe::kMaxExperts) count[e] = 0;
  __syncthreads();
  constexpr int kAhead = 8;
  for (int p0 = e; p0 < pairs; p0 += kAhead * kMake) {
    int x[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) x[i] = p0 + i * kMake < pairs ? a.pair_expert[p0 + i * kMake] : -1;
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      if (x[i] >= 0) atomicAdd(&count[x[i]], 1);
  }
  __syncthreads();
  const int mine = e < a.experts ? count[e] : 0;
  const int begin = block_prefix(mine, lds) - mine;
  __syncthreads();
  if (e < a.experts) count[e] = begin;
  make_tiles(begin, mine, a.tile_rows, a.tiles, a.max_tiles, a.tile_count, lds);
  __syncthreads();
  for (int p0 = e; p0 < pairs; p0 += kAhead * kMake) {
    int x[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) x[i] = p0 + i * kMake < pairs ? a.pair_expert[p0 + i * kMake] : -1;
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      if (x[i] >= 0) a.pairs[atomicAdd(&count[x[i]], 1)] = p0 + i * kMake;
  }
}

int64_t host_sum_blocks(const PrepareArgs& a) {
  return a.rows * (((int64_t)a.sum_groups * a.group + 8 * kThreads - 1) / (8 * kThreads));
}

}  // namespace

hipError_t launch_prepare(const PrepareArgs& a, hipStream_t stream) {
  const int64_t per = kMake / kThreads, blocks = (host_sum_blocks(a) + per - 1) / per + 1;
  if (a.dtype == QMM_BF16)
    hipLaunchKernelGGL(prepare_kernel<Bf16>, dim3((unsigned)blocks), dim3(kMake), 0, stream, a);
  else
    hipLaunchKernelGGL(prepare_kernel<Fp16>, dim3((unsigned)blocks), dim3(kMake), 0, stream, a);
  return hipGetLastError();
}

hipError_t launch_route(const RouteArgs& r, const PrepareArgs& p, hipStream_t stream) {
  const int route_blocks = (r.tokens + kThreads / 64 - 1) / (kThreads / 64);
  const dim3 grid((unsigned)(route_blocks + host_sum_blocks(p)));
  if (r.dtype == QMM_BF16)
    hipLaunchKernelGGL(route_kernel<Bf16>, grid, dim3(kThreads), 0, stream, r, p, route_blocks);
  else
    hipLaunchKernelGGL(route_kernel<Fp16>, grid, dim3(kThreads), 0, stream, r, p, route_blocks);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(list_kernel, dim3(1), dim3(kMake), 0, stream, r);
  return hipGetLastError();
}

}  // namespace grouped
}  // namespace qmm
