// Rows into and out of the 4-bit key/value cache (kv_cache.hpp has the layout).
//
// Append quantizes each (token, head) row of K and of V per group of gs elements in the steps
// of the weight quantizer, every operation in float32 with contraction disabled:
//     s = (max - min) / 15,  b = min,  q = clamp(rint((x - b) / s), 0, 15), q = 0 when s == 0,
// then s and b are rounded to nearest even in the storage dtype; a read gives
// round(fma(s, q, b)).  D/8 lanes hold one row, 8 consecutive elements each (one 16-byte
// load), so a group's extremes are a butterfly over gs/8 lanes.
// A workgroup takes consecutive tokens of one head's K or V, so that the byte stores of four
// tokens that share V's words leave from one wave.  An append moves 2*D + D/2 + 4*D/gs bytes
// per row, but is bound by its vector instructions, about 30 per element with the exact
// quotient (a plain division each: 22 us against 19).  Measured, 8191 tokens x 8 heads x 128
// elements in groups of 32: append 19 us (2.2 TB/s), read 15 us; 32 tokens 3 us each, their
// launch.
#include "device_common.hpp"
#include "kv_cache.hpp"

#pragma clang fp contract(off)

namespace qmm {
namespace kv {
namespace {

constexpr int kThreads = kCopyThreads;

// Address of (slot, head)'s page words, and the token inside the page.
__device__ inline uint32_t* page_of(const CacheArgs& c, int32_t slot, int head, int* token) {
  const int page = slot / c.page_size;
  *token = slot - page * c.page_size;
  return c.data + ((int64_t)page * c.heads + head) * (2 * c.side);
}

// A workgroup takes one (side, head) of consecutive tokens, as many as it has rows.
struct Place {
  int64_t token;
  int rest;             // side * heads + head
};
__device__ inline Place place(int heads, int rows, int row) {
  const uint32_t group = blockIdx.x / (uint32_t)(2 * heads);
  return Place{(int64_t)group * rows + row, (int)(blockIdx.x - group * (uint32_t)(2 * heads))};
}

template <class T, int D>
__global__ __launch_bounds__(kThreads) void append_kernel(const AppendArgs a) {
  constexpr int kLanes = D / 8;                    // lanes per row
  const int lane = threadIdx.x % kLanes;
  const int heads = a.c.heads;
  const Place at = place(heads, kThreads / kLanes, threadIdx.x / kLanes);
  const int64_t token = at.token;
  if (token >= a.tokens) return;                   // whole rows leave: the butterflies stay inside a row
  const int rest = at.rest;
  const int side = rest >= heads ? 1 : 0;
  const int head = rest - side * heads;
  const int32_t slot = a.slots[token];
  if (slot < 0 || slot >= a.c.pages * a.c.page_size) return;
  const uint16_t* x = (const uint16_t*)a.x[side] + token * a.token_stride[side] + head * a.head_stride[side] + 8 * lane;
  const u32x4 u = *(const u32x4*)x;
  float v[8];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    v[2 * e] = T::to_f32(u[e] & 0xFFFFu);
    v[2 * e + 1] = T::to_f32(u[e] >> 16);
  }
  float lo = v[0], hi = v[0];
#pragma unroll
  for (int e = 1; e < 8; ++e) {
    lo = fminf(lo, v[e]);
    hi = fmaxf(hi, v[e]);
  }
  const int lanes = a.c.group_size >> 3;
  for (int d = 1; d < lanes; d <<= 1) {
    lo = fminf(lo, __shfl_xor(lo, d));
    hi = fmaxf(hi, __shfl_xor(hi, d));
  }
  const float range = hi - lo;
  const float s = range / 15.0f;
  // (x - b) / s, rounded: from the rounded reciprocal and two corrections by the remainder
  // (Markstein 1990), in five operations where nothing can underflow; else by division
  uint32_t word = 0;
  if (s >= 0x1p-100f && s <= 0x1p100f) {
    const float inv = 1.0f / s;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float d = v[e] - lo;
      float t = d * inv;
      t = __builtin_fmaf(__builtin_fmaf(-t, s, d), inv, t);
      t = __builtin_fmaf(__builtin_fmaf(-t, s, d), inv, t);
      word |= (uint32_t)fminf(fmaxf(__builtin_rintf(t), 0.0f), 15.0f) << (4 * e);
    }
  } else if (s != 0.0f) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float t = (v[e] - lo) / s;
      word |= (uint32_t)fminf(fmaxf(__builtin_rintf(t), 0.0f), 15.0f) << (4 * e);
    }
  }
  int t;
  uint32_t* page = page_of(a.c, slot, head, &t) + side * a.c.side;
  if ((lane & (lanes - 1)) == 0) {
    uint32_t* sb = page + code_words(a.c.page_size, D) + (lane / lanes) * a.c.page_size + t;
    *sb = (uint32_t)T::from_f32(s) | ((uint32_t)T::from_f32(lo) << 16);
  }
  if (side == 0) {
    page[k_word(t, lane, D)] = word;
  } else {
    // lanes l and l ^ 2 hold the same o range of the element tiles i = 2j and 2j + 1: the
    // even tile's lane stores the bytes of o = 0..3 of the range, the odd one's o = 4..7
    const uint32_t other = __shfl_xor(word, 2);
    const int i = lane >> 1, odd = i & 1;
    const uint32_t low = (odd ? other : word) >> (16 * odd), high = (odd ? word : other) >> (16 * odd);
    uint8_t* bytes = (uint8_t*)page;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t b = ((low >> (4 * e)) & 15u) | (((high >> (4 * e)) & 15u) << 4);
      bytes[v_byte(t, 8 * (lane & 1) + 4 * odd + e, i >> 1, D)] = (uint8_t)b;
    }
  }
}

template <class T, int D>
__global__ __launch_bounds__(kThreads) void read_kernel(const ReadArgs a) {
  constexpr int kLanes = D / 8;
  const int lane = threadIdx.x % kLanes;
  const int heads = a.c.heads;
  const Place at = place(heads, kThreads / kLanes, threadIdx.x / kLanes);
  const int64_t n = at.token;
  if (n >= a.count) return;
  const int rest = at.rest;
  const int side = rest >= heads ? 1 : 0;
  const int head = rest - side * heads;
  const int32_t slot = a.slots[n];
  const bool bad = slot < 0 || slot >= a.c.pages * a.c.page_size;
  int t;
  const uint32_t* page = page_of(a.c, bad ? 0 : slot, head, &t) + side * a.c.side;
  const uint32_t sb = page[code_words(a.c.page_size, D) + (8 * lane / a.c.group_size) * a.c.page_size + t];
  const float s = T::to_f32(sb & 0xFFFFu), b = T::to_f32(sb >> 16);
  uint32_t word = 0;
  if (side == 0) {
    word = page[k_word(t, lane, D)];
  } else {
    const uint8_t* bytes = (const uint8_t*)page;
    const int i = lane >> 1;
#pragma unroll
    for (int e = 0; e < 8; ++e)
      word |= (((uint32_t)bytes[v_byte(t, 8 * (lane & 1) + e, i >> 1, D)] >> (4 * (i & 1))) & 15u) << (4 * e);
  }
  u32x4 r;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float lo = __builtin_fmaf(s, (float)((word >> (8 * e)) & 15u), b);
    const float hi = __builtin_fmaf(s, (float)((word >> (8 * e + 4)) & 15u), b);
    r[e] = bad ? 0x7FFF7FFFu : T::pack2(lo, hi);   // NaN in both types
  }
  *(u32x4*)((uint16_t*)a.out[side] + (n * heads + head) * D + 8 * lane) = r;
}

template <template <class, int> class K, class A>
hipError_t dispatch(const A& a, int64_t tokens, hipStream_t stream) {
  const dim3 g((unsigned)copy_blocks(a.c, tokens)), t(kThreads);
  const bool bf = a.c.dtype == QMM_BF16;
  switch (a.c.head_dim) {
    case 64: bf ? K<Bf16, 64>::go(a, g, t, stream) : K<Fp16, 64>::go(a, g, t, stream); break;
    case 128: bf ? K<Bf16, 128>::go(a, g, t, stream) : K<Fp16, 128>::go(a, g, t, stream); break;
    case 256: bf ? K<Bf16, 256>::go(a, g, t, stream) : K<Fp16, 256>::go(a, g, t, stream); break;
    default: return hipErrorInvalidValue;
  }
  return hipGetLastError();
}

template <class T, int D>
struct Append {
  static void go(const AppendArgs& a, dim3 g, dim3 t, hipStream_t s) {
    hipLaunchKernelGGL((append_kernel<T, D>), g, t, 0, s, a);
  }
};
template <class T, int D>
struct Read {
  static void go(const ReadArgs& a, dim3 g, dim3 t, hipStream_t s) {
    hipLaunchKernelGGL((read_kernel<T, D>), g, t, 0, s, a);
  }
};

}  // namespace

hipError_t launch_append(const AppendArgs& a, hipStream_t stream) {
  return dispatch<Append>(a, a.tokens, stream);
}
hipError_t launch_read(const ReadArgs& a, hipStream_t stream) {
  return dispatch<Read>(a, a.count, stream);
}

}  // namespace kv
}  // namespace qmm
