// Pages of the cache: copies of whole pages, and the step that continues block tables from
// others (forks), hands out free pages and takes back those that nobody holds.
#include <algorithm>

#include "device_common.hpp"
#include "kv_pages.hpp"

namespace qmm {
namespace kv {
namespace {

// ---- page copies.  A page of all heads is one run of memory; a workgroup copies 16 KB of one
// page, four quads a thread so that four loads are in flight.  Bound by memory: 96 pages of 256
// tokens, 8 heads of 128, 11.4 us, 5.0 TB/s; up to 32 pages of 64 tokens 3.2 us, the launch.
constexpr int kCopyQuads = 4;                  // 16-byte quads per thread

__global__ __launch_bounds__(256) void copy_pages_kernel(const CopyPagesArgs a) {
  const int64_t first = ((int64_t)blockIdx.x * kCopyQuads) * 256 + threadIdx.x;
  for (int64_t i = blockIdx.y; i < a.count; i += gridDim.y) {
    const int32_t src = a.src[i], dst = a.dst[i];
    if (src < 0 || src >= a.c.pages || dst < 0 || dst >= a.c.pages || src == dst) continue;
    const u32x4* from = (const u32x4*)a.c.data + src * a.page_quads;
    u32x4* to = (u32x4*)a.c.data + dst * a.page_quads;
    u32x4 q[kCopyQuads];
#pragma unroll
    for (int j = 0; j < kCopyQuads; ++j) {
      const int64_t at = first + 256 * j;
      q[j] = from[at < a.page_quads ? at : 0];
    }
#pragma unroll
    for (int j = 0; j < kCopyQuads; ++j) {
      const int64_t at = first + 256 * j;
      if (at < a.page_quads) to[at] = q[j];
    }
  }
}

// ---- forks.  Up to three kernels, each of which needs sums over all workgroups of the one before:
//   fork_count  marks every entry of the new table as a page that stays, none, or fresh, and
//               counts the fresh ones of a row; counts the free pages of each segment of the pool;
//   fork_list   numbers the free pages, lowest first (a pool of one segment's are numbered by
//               fork_count: a launch less, 14.4 us of a call from Python
//               against 17.7);
//   fork_assign gives fresh entry number k (by row, then block) free page number k, and updates
//               the reference counts: integer atomics, whose order changes nothing.
// The counts are not touched before the last kernel, so free means free before the call: a page
// that is taken back by the call is not handed out by it, and may still be the source of a copy.
// Bound by their launches at the sizes of a batch (in three, 32 rows of 32 blocks 10.4 us, 128 rows of
// 18 blocks 11 us).
constexpr int kFresh = -2;                     // a mark in the new table, between the kernels
constexpr int kMaxCut = 16384;                 // a row's blocks past the new table count up to this: sums fit 31 bits

// Sum over the workgroup of one number per thread.
__device__ inline int block_sum(int v, int* lds) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) v += __shfl_xor(v, d);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  return lds[0] + lds[1] + lds[2] + lds[3];
}

// Largest number of the workgroup's.
__device__ inline int block_max(int v, int* lds) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) v = max(v, __shfl_xor(v, d));
  __syncthreads();
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  return max(max(lds[0], lds[1]), max(lds[2], lds[3]));
}

// Number of this thread's set flag among the workgroup's, and their count.
__device__ inline int block_rank(bool flag, int* lds, int* total) {
  const uint64_t m = __ballot(flag);
  const int wave = threadIdx.x >> 6;
  __syncthreads();
  if ((threadIdx.x & 63) == 0) lds[wave] = __popcll(m);
  __syncthreads();
  int before = 0;
#pragma unroll
  for (int w = 0; w < 4; ++w) before += w < wave ? lds[w] : 0;
  *total = lds[0] + lds[1] + lds[2] + lds[3];
  return before + __popcll(m & ((1ull << (threadIdx.x & 63)) - 1));
}

// Numbers the free pages of segment s from `at` on.
__device__ inline void list_segment(const ForkArgs& a, int64_t s, int64_t at, int* lds) {
  const int64_t p0 = s * kSegment, p1 = min(p0 + kSegment, a.pages);
  for (int64_t p = p0; p < p1 && at < a.list_size; p += kForkThreads) {
    const int64_t mine = p + threadIdx.x;
    const bool open = mine < p1 && a.refs[mine] == 0;
    int total;
    const int64_t k = at + block_rank(open, lds, &total);
    if (open && k < a.list_size) a.list[k] = (int32_t)mine;
    at += total;
  }
}

struct ForkRow {
  int64_t parent;            // -1: none
  int64_t full, cover;       // blocks that stay shared, blocks in all
  bool partial;
};
__device__ inline ForkRow fork_row(const ForkArgs& a, int64_t i) {
  ForkRow r;
  const int64_t p = a.parents[i];
  r.parent = p >= 0 && p < a.batch ? p : -1;
  const int64_t length = r.parent >= 0 ? max(0, a.lengths[r.parent]) : 0;
  const int64_t want = a.want ? max(0, a.want[i]) : length;
  const int64_t keep = min(length, want);
  r.full = keep / a.page_size;
  r.partial = keep % a.page_size != 0;
  r.cover = (want + a.page_size - 1) / a.page_size;
  return r;
}

__global__ __launch_bounds__(kForkThreads) void fork_count_kernel(const ForkArgs a) {
  __shared__ int lds[4];
  if (blockIdx.x >= a.rows) {                  // a segment of the pool
    const int64_t s = blockIdx.x - a.rows, p0 = s * kSegment, p1 = min(p0 + kSegment, a.pages);
    int open = 0;
#pragma unroll 4
    for (int64_t p = p0 + threadIdx.x; p < p1; p += kForkThreads) open += a.refs[p] == 0 ? 1 : 0;
    open = block_sum(open, lds);
    if (threadIdx.x == 0) a.open[s] = open;
    if (a.segments == 1) list_segment(a, 0, 0, lds);       // nothing comes before it
    return;
  }
  const int64_t i = blockIdx.x;
  const ForkRow r = fork_row(a, i);
  // The parent's first row keeps its old pages from the first block on that no other row of the parent
  // shares: it writes there, and a row that keeps more tokens reads them.
  int shared = 0;                              // blocks that another row names; all of them for later rows
  if (r.parent >= 0)
    for (int64_t o = threadIdx.x; o < a.rows; o += kForkThreads)
      if (a.parents[o] == r.parent && o != i) shared = max(shared, o < i ? 0x7FFFFFFF : (int)fork_row(a, o).full);
  shared = block_max(shared, lds);
  int need = 0;
  for (int64_t j = threadIdx.x; j < a.new_blocks; j += kForkThreads) {
    const int32_t page = r.parent >= 0 && j < a.blocks ? a.table[r.parent * a.table_stride + j] : -1;
    const bool valid = page >= 0 && page < a.pages;
    int32_t entry = -1;
    if (j < r.full) {
      entry = valid ? page : -1;
    } else if (j < r.cover) {
      const bool keeps = j >= shared && valid && a.refs[page] == 1;
      entry = keeps ? page : kFresh;
      need += keeps ? 0 : 1;
    }
    a.new_table[i * a.new_stride + j] = entry;
    if (j == r.full) a.copy_src[i] = r.partial && entry == kFresh && valid ? page : -1;
  }
  need = block_sum(need, lds);
  if (threadIdx.x == 0) {
    a.need[i] = need;
    a.cut[i] = (int32_t)min((int64_t)kMaxCut, max((int64_t)0, r.cover - a.new_blocks));
    if (r.full >= a.new_blocks) a.copy_src[i] = -1;
  }
}

__global__ __launch_bounds__(kForkThreads) void fork_list_kernel(const ForkArgs a) {
  __shared__ int lds[4];
  const int64_t s = blockIdx.x;
  int before = 0;
  for (int64_t o = threadIdx.x; o < s; o += kForkThreads) before += a.open[o];
  list_segment(a, s, block_sum(before, lds), lds);
}

__global__ __launch_bounds__(kForkThreads) void fork_assign_kernel(const ForkArgs a) {
  __shared__ int lds[4];
  if (blockIdx.x >= a.rows) {                  // a row of the old table lets go of its pages
    const int64_t b = blockIdx.x - a.rows;
    if (a.rows == 0 && b == 0 && threadIdx.x == 0) *a.short_of = 0;
    for (int64_t j = threadIdx.x; b < a.batch && j < a.blocks; j += kForkThreads) {
      const int32_t page = a.table[b * a.table_stride + j];
      if (page >= 0 && page < a.pages) atomicSub(a.refs + page, 1);
    }
    return;
  }
  const int64_t i = blockIdx.x;
  int open = 0, before = 0;
  for (int64_t s = threadIdx.x; s < a.segments; s += kForkThreads) open += a.open[s];
  open = block_sum(open, lds);
  for (int64_t o = threadIdx.x; o < i; o += kForkThreads) before += a.need[o];
  int64_t at = block_sum(before, lds);
  const ForkRow r = fork_row(a, i);
  for (int64_t j0 = 0; j0 < a.new_blocks; j0 += kForkThreads) {
    const int64_t j = j0 + threadIdx.x;
    int32_t entry = j < a.new_blocks ? a.new_table[i * a.new_stride + j] : -1;
    int total;
    const int64_t k = at + block_rank(entry == kFresh, lds, &total);
    at += total;
    if (entry == kFresh) {
      entry = k < open ? a.list[k] : -1;       // (k < list_size: the entries of the new table)
      a.new_table[i * a.new_stride + j] = entry;
      if (j == r.full) {
        const bool copy = entry >= 0 && a.copy_src[i] >= 0;
        a.copy_dst[i] = copy ? entry : -1;
        if (!copy) a.copy_src[i] = -1;
      }
    } else if (j == r.full) {
      a.copy_dst[i] = -1;
    }
    if (entry >= 0) atomicAdd(a.refs + entry, 1);
  }
  if (threadIdx.x == 0 && r.full >= a.new_blocks) a.copy_dst[i] = -1;
  if (i == a.rows - 1) {                       // what the call could not give
    int cut = 0;
    for (int64_t o = threadIdx.x; o < a.rows; o += kForkThreads) cut += a.cut[o];
    cut = block_sum(cut, lds);
    if (threadIdx.x == 0) *a.short_of = (int32_t)(max((int64_t)0, at - open) + cut);
  }
}

}  // namespace

hipError_t launch_copy_pages(const CopyPagesArgs& a, hipStream_t stream) {
  const int64_t per = 256 * kCopyQuads;
  const dim3 g((unsigned)((a.page_quads + per - 1) / per), (unsigned)std::min<int64_t>(a.count, 65535));
  hipLaunchKernelGGL(copy_pages_kernel, g, dim3(256), 0, stream, a);
  return hipGetLastError();
}

hipError_t launch_fork(const ForkArgs& a, hipStream_t stream) {
  const unsigned segments = (unsigned)a.segments;
  hipLaunchKernelGGL(fork_count_kernel, dim3((unsigned)a.rows + segments), dim3(kForkThreads), 0, stream, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (segments > 1) {
    hipLaunchKernelGGL(fork_list_kernel, dim3(segments), dim3(kForkThreads), 0, stream, a);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(fork_assign_kernel, dim3((unsigned)(a.rows + std::max<int64_t>(a.batch, 1))), dim3(kForkThreads), 0, stream, a);
  return hipGetLastError();
}

}  // namespace kv
}  // namespace qmm
