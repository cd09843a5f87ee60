// Trees of drafted tokens: which nodes a node sees, the path that verification accepts, and the
// move of a sequence's rows that follows.
#include <algorithm>

#include "device_common.hpp"
#include "kv_pages.hpp"

namespace qmm {
namespace kv {
namespace {

constexpr int kThreads = 256;

// ---- mask and depth.  A thread walks one node's path to its root for one word of the mask;
// parents come before their children, so a walk is at most `nodes` steps and ends whatever the
// parents hold.  One thread per word, not per bit or node: a path's bits of a word need the same
// walk, and no thread waits for another.  Bound by its launch (16 trees of 32 nodes 4.6 us).
__global__ __launch_bounds__(kThreads) void tree_mask_kernel(const TreeMaskArgs a) {
  __shared__ int32_t up[kMaxNodes];
  const int64_t b = blockIdx.y;
  for (int i = threadIdx.x; i < a.nodes; i += kThreads) up[i] = a.parents[b * a.stride + i];
  __syncthreads();
  const int t = blockIdx.x * kThreads + threadIdx.x;
  if (t >= a.nodes * a.words) return;
  const int node = t / a.words, word = t - node * a.words;
  uint32_t bits = 0u;
  int at = node, steps = 0;
  while (at >= 0) {
    if ((at >> 5) == word && (a.window == 0 || steps < a.window)) bits |= 1u << (at & 31);
    const int p = up[at];
    at = p >= -1 && p < at ? p : -2;
    ++steps;
  }
  const bool whole = at == -1;                 // else: a node of the path is none
  a.mask[(b * a.nodes + node) * a.words + word] = whole ? bits : 0u;
  if (word == 0 && a.depth) a.depth[b * a.nodes + node] = whole ? steps - 1 : 0;
}

// ---- the accepted path, one wave per sequence: from node 0 on, the lowest child whose drafted
// token is the one sampled after its parent.  A step is one pass over the later nodes in LDS, 64 at a
// time and no further than the child: a tree fits one wave, which then needs no barrier.  Bound by
// its launch (64 trees of 63 nodes 4.1 us, one of 13 nodes 2.2 us).
__global__ __launch_bounds__(64) void tree_accept_kernel(const TreeAcceptArgs a) {
  __shared__ int32_t up[kMaxNodes], token[kMaxNodes], sampled[kMaxNodes];
  const int64_t b = blockIdx.x;
  const int lane = threadIdx.x;
  for (int i = lane; i < a.nodes; i += 64) {
    up[i] = a.parents[b * a.parents_stride + i];
    token[i] = a.tokens[b * a.tokens_stride + i];
    sampled[i] = a.sampled[b * a.sampled_stride + i];
    a.path[b * a.nodes + i] = -1;
  }
  __syncthreads();
  int at = up[0] == -1 ? 0 : -1, count = 0, last = -1;
  while (at >= 0) {
    if (lane == (count & 63)) a.path[b * a.nodes + count] = at;   // (the lane that wrote -1 there)
    ++count;
    last = sampled[at];
    int next = -1;
    for (int i0 = at & ~63; i0 < a.nodes; i0 += 64) {
      const int i = i0 + lane;
      const bool fits = i > at && i < a.nodes && up[i] == at && token[i] == last;
      const uint64_t m = __ballot(fits);
      if (m) {
        next = i0 + __builtin_ctzll(m);
        break;
      }
    }
    at = next;
  }
  if (lane == 0) {
    a.count[b] = count;
    a.last[b] = last;
  }
}

// ---- rows of a sequence to other positions, as they are (codes, scales and biases).
//
// A workgroup takes one head of one sequence and 64 consecutive positions at a time, in whole
// groups of four: a word of V's codes holds four consecutive tokens (kv_cache.hpp), so a word is
// put together from its four source rows.  In the same pages every source of a step is in
// registers before anything is written, and the steps go up: with ascending sources that are
// not below their destinations, a step writes nothing that a later one reads.  Into other pages
// the steps are independent workgroups.
// Bound by latency for a path (table, rows, barrier, stores: 64 paths of 63 nodes, 8 heads of 128, 6 us),
// by memory for long moves (10240 rows of 8 heads of 128 to other pages 11.4 us, 26 MB in all,
// 2.3 TB/s; in whole sectors, of which a kept row's V bytes, scales and biases are a part each, about
// 48 MB).
template <int D>
__global__ __launch_bounds__(kThreads) void move_kernel(const MoveArgs a) {
  constexpr int kStep = 64;
  constexpr int KQ = D / 32;                    // 16-byte quads of a K row
  constexpr int VQ = D / 8;                     // 16-byte quads of four V rows
  constexpr int KN = (kStep * KQ + kThreads - 1) / kThreads, VN = (kStep / 4 * VQ + kThreads - 1) / kThreads;
  constexpr int SN = kStep * 2 * (D / 32) / kThreads;   // scale words at most: groups of 32
  struct Row {
    int64_t from, to;                           // words of the pages of this head, -1: no row
    int32_t from_token, to_token;
  };
  __shared__ Row rows[kStep];
  const int64_t n = blockIdx.x / a.c.heads;
  const int head = (int)(blockIdx.x - n * a.c.heads);
  const int64_t page_words = 2 * a.c.side;
  const int64_t start = a.start[n], origin = a.origin ? a.origin[n] : 0;
  const int64_t code_at = code_words(a.c.page_size, D);
  const int groups = D / a.c.group_size;
  const int64_t p0 = start & ~(int64_t)3, p1 = start + a.count;
  const int64_t step = a.in_place ? kStep : (int64_t)kStep * gridDim.y;

  for (int64_t p = p0 + (a.in_place ? 0 : (int64_t)kStep * blockIdx.y); p < p1; p += step) {
    __syncthreads();                            // the last step's rows have been used
    if (threadIdx.x < kStep) {
      const int64_t pos = p + threadIdx.x, i = pos - start;
      Row r{-1, -1, 0, 0};
      if (i >= 0 && i < a.count && pos >= 0) {
        const int64_t x = a.index[n * a.index_stride + i];
        const int64_t src = x < 0 ? -1 : origin + x;
        if (src >= 0) {
          const int64_t sb = src / a.c.page_size, db = pos / a.c.page_size;
          if (sb < a.blocks && db < a.to_blocks) {
            const int32_t sp = a.table[n * a.table_stride + sb], dp = a.to[n * a.to_stride + db];
            if (sp >= 0 && sp < a.c.pages && dp >= 0 && dp < a.c.pages && (sp != dp || src != pos || !a.in_place)) {
              r.from = ((int64_t)sp * a.c.heads + head) * page_words;
              r.to = ((int64_t)dp * a.c.heads + head) * page_words;
              r.from_token = (int32_t)(src - sb * a.c.page_size);
              r.to_token = (int32_t)(pos - db * a.c.page_size);
            }
          }
        }
      }
      rows[threadIdx.x] = r;
    }
    __syncthreads();
    u32x4 k[KN], v[VN];
    uint32_t sb[SN], valid[VN];
#pragma unroll
    for (int u = 0; u < KN; ++u) {
      const int t = threadIdx.x + u * kThreads, row = t / KQ, quad = t - row * KQ;
      if (row < kStep && rows[row].from >= 0)
        k[u] = *(const u32x4*)(a.c.data + rows[row].from + rows[row].from_token * (D / 8) + 4 * quad);
    }
#pragma unroll
    for (int u = 0; u < SN; ++u) {
      const int t = threadIdx.x + u * kThreads, row = t & (kStep - 1), g = t / kStep;   // side * groups + group
      if (g < 2 * groups && rows[row].from >= 0)
        sb[u] = a.c.data[rows[row].from + (g >= groups ? a.c.side : 0) + code_at +
                         (int64_t)(g >= groups ? g - groups : g) * a.c.page_size + rows[row].from_token];
    }
#pragma unroll
    for (int u = 0; u < VN; ++u) {
      const int t = threadIdx.x + u * kThreads, four = t / VQ, quad = t - four * VQ;
      valid[u] = 0u;
      v[u] = u32x4{0u, 0u, 0u, 0u};
      if (four < kStep / 4) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const Row r = rows[4 * four + e];
          if (r.from >= 0) {
            const u32x4 w = *(const u32x4*)(a.c.data + r.from + a.c.side + (r.from_token / 4) * (D / 2) + 4 * quad);
            const int shift = 8 * (r.from_token & 3);
            valid[u] |= 1u << e;
#pragma unroll
            for (int c = 0; c < 4; ++c) v[u][c] |= ((w[c] >> shift) & 0xFFu) << (8 * e);
          }
        }
      }
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // every source of the step has arrived,
    __syncthreads();                                   // in every wave
#pragma unroll
    for (int u = 0; u < KN; ++u) {
      const int t = threadIdx.x + u * kThreads, row = t / KQ, quad = t - row * KQ;
      if (row < kStep && rows[row].from >= 0)
        *(u32x4*)(a.c.data + rows[row].to + rows[row].to_token * (D / 8) + 4 * quad) = k[u];
    }
#pragma unroll
    for (int u = 0; u < SN; ++u) {
      const int t = threadIdx.x + u * kThreads, row = t & (kStep - 1), g = t / kStep;
      if (g < 2 * groups && rows[row].from >= 0)
        a.c.data[rows[row].to + (g >= groups ? a.c.side : 0) + code_at +
                 (int64_t)(g >= groups ? g - groups : g) * a.c.page_size + rows[row].to_token] = sb[u];
    }
#pragma unroll
    for (int u = 0; u < VN; ++u) {
      const int t = threadIdx.x + u * kThreads, four = t / VQ, quad = t - four * VQ;
      if (valid[u] == 0xFu) {                   // four positions from a multiple of four: one page
        const Row r = rows[4 * four];
        *(u32x4*)(a.c.data + r.to + a.c.side + (r.to_token / 4) * (D / 2) + 4 * quad) = v[u];
      } else if (valid[u]) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (!((valid[u] >> e) & 1u)) continue;
          const Row r = rows[4 * four + e];
          uint8_t* to = (uint8_t*)(a.c.data + r.to + a.c.side + (r.to_token / 4) * (D / 2) + 4 * quad) + e;
#pragma unroll
          for (int c = 0; c < 4; ++c) to[4 * c] = (uint8_t)(v[u][c] >> (8 * e));
        }
      }
    }
  }
}

}  // namespace

hipError_t launch_tree_mask(const TreeMaskArgs& a, hipStream_t stream) {
  const unsigned blocks = (unsigned)((a.nodes * a.words + kThreads - 1) / kThreads);
  hipLaunchKernelGGL(tree_mask_kernel, dim3(blocks, (unsigned)a.batch), dim3(kThreads), 0, stream, a);
  return hipGetLastError();
}

hipError_t launch_tree_accept(const TreeAcceptArgs& a, hipStream_t stream) {
  hipLaunchKernelGGL(tree_accept_kernel, dim3((unsigned)a.batch), dim3(64), 0, stream, a);
  return hipGetLastError();
}

hipError_t launch_move(const MoveArgs& a, hipStream_t stream) {
  const int64_t steps = (a.count + 3 + 63) / 64;          // a start that is no multiple of four adds up to three
  const dim3 g((unsigned)(a.batch * a.c.heads), (unsigned)(a.in_place ? 1 : std::min<int64_t>(steps, 65535))), t(kThreads);
  switch (a.c.head_dim) {
    case 64: hipLaunchKernelGGL(move_kernel<64>, g, t, 0, stream, a); break;
    case 128: hipLaunchKernelGGL(move_kernel<128>, g, t, 0, stream, a); break;
    case 256: hipLaunchKernelGGL(move_kernel<256>, g, t, 0, stream, a); break;
    default: return hipErrorInvalidValue;
  }
  return hipGetLastError();
}

}  // namespace kv
}  // namespace qmm
