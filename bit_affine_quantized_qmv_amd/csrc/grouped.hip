// What comes before the products grouped by expert: sums of activation groups, the rows of every
// expert, and their tiles.
#include "grouped_impl.hpp"
#include "moe_route.hpp"

namespace qmm {
namespace grouped {
namespace {

// 2048 elements of a row (thread `at` of 256 has eight of them) as the products take them, and the
// sums of their groups in three bfloat16 parts; what a row is padded to is zero.  Sums in float32,
// eight in order, then the lanes in pairs.  Bound by memory.
template <class T>
__device__ inline void stage_rows(const PrepareArgs& a, int64_t block, int at) {
  const int per_row = (int)blocks_per_row(a);
  const int64_t row = block / per_row;
  const int k = (int)(block - row * per_row) * 8 * kThreads + 8 * at;
  float sum = 0.f;
  u32x4 u = {0u, 0u, 0u, 0u};
  if (k < a.k) {
    u = *(const u32x4*)(a.x + row * a.x_stride + k);
#pragma unroll
    for (int e = 0; e < 4; ++e) sum += T::to_f32(u[e] & 0xFFFFu) + T::to_f32(u[e] >> 16);
  }
  if (k < a.cols) *(u32x4*)(a.staged + row * a.cols + k) = a.bits == 4 ? interleave_even_odd(u) : u;
  sum += __shfl_xor(sum, 1);
  sum += __shfl_xor(sum, 2);
  if (a.group >= 64) sum += __shfl_xor(sum, 4);
  if (a.group == 128) sum += __shfl_xor(sum, 8);
  const int g = k / a.group;
  if (k % a.group == 0 && g < a.sum_groups)
    store_sum(a.sums + row * kPlanes * a.sum_groups + g, a.sum_groups, sum);
}

// Inclusive prefix of one number per thread of the first 512, over the workgroup (kMake threads).
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
      tiles[at] = Tile{(int)threadIdx.x, begin + i * tile_rows, min(tile_rows, count - i * tile_rows), end - n, n, {}};
  }
  if (threadIdx.x == kMake - 1) *tile_count = min(end, max_tiles);
}

// Tiles of given offsets, by the last workgroup; the activations by the others.  An expert's rows start
// where all before it have ended, whatever the offsets are.
template <class T>
__global__ __launch_bounds__(kMake) void prepare_kernel(const PrepareArgs a) {
  __shared__ int lds[kMake / 64];
  __shared__ int most[kMake / 64];
  if (blockIdx.x + 1 < gridDim.x) {
    const int64_t block = (int64_t)blockIdx.x * (kMake / kThreads) + threadIdx.x / kThreads;
    if (block < a.rows * blocks_per_row(a)) stage_rows<T>(a, block, threadIdx.x % kThreads);
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
// unless renormalised), by one wave; the activations by the other workgroups.
template <class T>
__global__ __launch_bounds__(kThreads) void route_kernel(const RouteArgs a, const PrepareArgs p, const int route_blocks) {
  if ((int)blockIdx.x >= route_blocks) {
    stage_rows<T>(p, (int64_t)blockIdx.x - route_blocks, threadIdx.x);
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

// y_t = sum of t's pairs, each by its share, in the order of its choices, rounded to dtype; four
// columns per thread.  Bound by memory.
template <class T>
__global__ __launch_bounds__(kThreads) void sum_kernel(const SumArgs a) {
  const int n = 4 * (int)(blockIdx.x * kThreads + threadIdx.x), t = blockIdx.y;
  if (n >= a.hidden) return;
  const float* o = a.out + (int64_t)t * a.top_k * a.hidden + n;
  const int64_t to_split = (int64_t)a.tokens * a.top_k * a.hidden;
  const float* share = a.share + t * a.top_k;
  f32x4 v = {0.f, 0.f, 0.f, 0.f};
  float sum = 0.f;
  constexpr int kAhead = 8;          // choices whose loads are in flight together
  for (int i0 = 0; i0 < a.top_k; i0 += kAhead) {
    f32x4 w[kAhead];
    float f[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int at = min(i0 + i, a.top_k - 1);
      w[i] = *(const f32x4*)(o + (int64_t)at * a.hidden);
      f[i] = share[at];
    }
    for (int s = 1; s < a.splits; ++s) {
      f32x4 u[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) u[i] = *(const f32x4*)(o + s * to_split + (int64_t)min(i0 + i, a.top_k - 1) * a.hidden);
#pragma unroll
      for (int i = 0; i < kAhead; ++i) w[i] += u[i];
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (i0 + i >= a.top_k) break;
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = __builtin_fmaf(f[i], w[i][e], v[e]);
      sum += f[i];
    }
  }
  if (a.renormalize) {
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] /= sum;
  }
  uint16_t* y = a.y + t * a.y_stride + n;
  const uint2 u = {T::pack2(v[0], v[1]), T::pack2(v[2], v[3])};
  if (((uintptr_t)a.y & 7u) == 0u && (a.y_stride & 3) == 0) {
    *(uint2*)y = u;
  } else {
    y[0] = (uint16_t)u.x;
    y[1] = (uint16_t)(u.x >> 16);
    y[2] = (uint16_t)u.y;
    y[3] = (uint16_t)(u.y >> 16);
  }
}

}  // namespace

hipError_t launch_sum(const SumArgs& a, hipStream_t stream) {
  const dim3 grid((unsigned)((a.hidden + 4 * kThreads - 1) / (4 * kThreads)), (unsigned)a.tokens);
  if (a.dtype == QMM_BF16)
    hipLaunchKernelGGL(sum_kernel<Bf16>, grid, dim3(kThreads), 0, stream, a);
  else
    hipLaunchKernelGGL(sum_kernel<Fp16>, grid, dim3(kThreads), 0, stream, a);
  return hipGetLastError();
}

hipError_t launch_prepare(const PrepareArgs& a, hipStream_t stream) {
  const dim3 grid((unsigned)prepare_blocks(a));
  if (a.dtype == QMM_BF16)
    hipLaunchKernelGGL(prepare_kernel<Bf16>, grid, dim3(kMake), 0, stream, a);
  else
    hipLaunchKernelGGL(prepare_kernel<Fp16>, grid, dim3(kMake), 0, stream, a);
  return hipGetLastError();
}

hipError_t launch_route(const RouteArgs& r, const PrepareArgs& p, hipStream_t stream) {
  const int route_blocks = (r.tokens + kThreads / 64 - 1) / (kThreads / 64);
  const dim3 grid((unsigned)(route_blocks + p.rows * blocks_per_row(p)));
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
