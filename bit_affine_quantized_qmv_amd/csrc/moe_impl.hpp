// Mixture-of-experts layer for up to 32 tokens over quantized expert stacks:
//     S_t  = the top_k largest router logits of token t (equal ones: lower expert),
//     w_te = softmax over S_t (renormalize) or over all experts, taken at e,
//     y_t  = sum_{e in S_t}  ( w_te silu(Wg_e x_t) * (Wu_e x_t) ) Wd_e^T.
//
// The layer reads each chosen expert's weights once and little else, so it is bound by that
// stream (and, for one token, by latency).  Two kernels: the products with Wg and Wu together,
// since both take x and the activation needs both, then the product with Wd.
//
// Both kernels give every wave one 16-row tile of weights (16 rows of Wg and the same of Wu,
// or 16 rows of Wd) and one stretch of K, and load the activations' operands straight from
// global memory: x and h are small and stay in L2, only the rows of tokens that use the
// expert are loaded, and no wave waits for another before its weights are in flight.  The
// matrix-core operand's 16 (or 32) activation rows are the call's tokens, rows of tokens
// that do not use the expert being zero: sums over several experts then stay in the same
// accumulators.  Arithmetic per output as in the decode kernels, s * sum xq + b * sum x per
// group with exact integer codes and float32 sums; here sum x comes from a second product
// with an all-ones operand, which costs nothing beside the weight stream.
// h = w silu(g) u is rounded once to dtype, as the second product's operand.
#pragma once

#include "decode_impl.hpp"
#include "moe.hpp"

namespace qmm {
namespace moe {

using decode::generic_lane_offsets;
using decode::load_slot;
using decode::Slot;
using decode::slot_codes;
using decode::SlotData;
using decode::slot_reorder;

constexpr int kWaves = 8;
constexpr int kThreads = 64 * kWaves;
constexpr int kExpertRegs = kMaxExperts / 64;   // router logits of one token per lane

// Order key of a 16-bit float: larger values have larger keys, NaN the largest.
template <class T>
__device__ inline uint32_t order_key(uint32_t b) {
  constexpr uint32_t kInf = T::kDtype == 2 ? 0x7C00u : 0x7F80u;
  if ((b & 0x7FFFu) > kInf) return 0xFFFFu;
  if (b == 0x8000u) b = 0u;                     // -0 and +0 are equal
  return (b & 0x8000u) ? (~b & 0xFFFFu) : (b | 0x8000u);
}

__device__ inline uint32_t wave_max(uint32_t v) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const uint32_t o = __shfl_xor(v, d);
    v = o > v ? o : v;
  }
  return v;
}
__device__ inline float wave_sum(float v) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) v += __shfl_xor(v, d);
  return v;
}

// The call's routing, in LDS.
struct Routing {
  uint32_t chosen[kMaxTokens][kMaxExperts / 32];   // bit e: token uses expert e
  float top[kMaxTokens];                           // largest router logit
  float inv[kMaxTokens];                           // 1 / the softmax sum
  uint32_t any[kMaxExperts / 32];                  // experts that some token uses
};

// Fill r (every workgroup does: a token's choice costs one wave top_k rounds of a maximum).
template <class T>
__device__ inline void route(const MoeArgs& a, Routing& r) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (int t = wave; t < a.tokens; t += kWaves) {
    const uint16_t* logits = a.router + t * a.router_stride;
    // (key, lowest expert first) words; experts are below 2^9
    uint32_t word[kExpertRegs];
    float v[kExpertRegs];
#pragma unroll
    for (int j = 0; j < kExpertRegs; ++j) {
      const int e = 64 * j + lane;
      word[j] = 0u;
      v[j] = 0.f;
      if (64 * j < a.experts && e < a.experts) {
        const uint32_t b = logits[e];
        word[j] = (order_key<T>(b) << 9) | (uint32_t)(kMaxExperts - 1 - e);
        v[j] = T::to_f32(b);
      }
    }
    uint32_t mine = 0u;            // lane i < 16 collects bits 32 i .. 32 i + 31
    float top = 0.f, sum = 0.f;
    for (int i = 0; i < a.top_k; ++i) {
      uint32_t best = 0u;
#pragma unroll
      for (int j = 0; j < kExpertRegs; ++j) best = word[j] > best ? word[j] : best;
      best = wave_max(best);
      const int e = kMaxExperts - 1 - (int)(best & (kMaxExperts - 1));
      const float l = T::to_f32(logits[e]);
      if (i == 0) top = l;
      sum += expf(l - top);
      if (lane == (e >> 5)) mine |= 1u << (e & 31);
#pragma unroll
      for (int j = 0; j < kExpertRegs; ++j) word[j] = word[j] == best ? 0u : word[j];
    }
    if (!a.renormalize) {
      sum = 0.f;
#pragma unroll
      for (int j = 0; j < kExpertRegs; ++j)
        if (64 * j + lane < a.experts) sum += expf(v[j] - top);
      sum = wave_sum(sum);
    }
    if (lane < kMaxExperts / 32) r.chosen[t][lane] = mine;
    if (lane == 0) {
      r.top[t] = top;
      r.inv[t] = 1.0f / sum;
    }
  }
  __syncthreads();
  if (threadIdx.x < kMaxExperts / 32) {
    uint32_t m = 0u;
    for (int t = 0; t < a.tokens; ++t) m |= r.chosen[t][threadIdx.x];
    r.any[threadIdx.x] = m;
  }
  __syncthreads();
}

// Bits of m[0 .. e) that are set.
__device__ inline int rank_of(const uint32_t* m, int e) {
  int n = 0;
  for (int i = 0; i < e >> 5; ++i) n += __popc(m[i]);
  return n + __popc(m[e >> 5] & ((1u << (e & 31)) - 1u));
}

// One wave's products of TN weight tiles with MT * 16 activation rows over slots [s0, s1).
template <class T, int BITS, int GS, int TN, int MT>
struct Stream {
  using S = Slot<BITS, GS>;
  static constexpr int kSteps = S::kSteps;
  static constexpr int kDepth = MT == 1 ? 4 : 2;      // slots in flight
  static constexpr int kSub8 = BITS == 8;

  const uint32_t* w[TN];      // the lane's weight row of each tile
  const uint16_t* s[TN];
  const uint16_t* b[TN];
  const uint16_t* x[MT];      // the lane's activation row, null: zeros
  int K, row_words, lg, gword;
  uint32_t gshift;
  bool narrow;

  struct Data {
    SlotData<BITS, GS> d[TN];
    u32x4 x[MT][kSteps];
  };

  __device__ inline void setup(const MoeArgs& a, int k) {
    K = k;
    lg = (threadIdx.x & 63) >> 4;
    row_words = (K * BITS) >> 5;
    gword = 0;
    gshift = 0u;
    if constexpr (BITS != 4 && BITS != 8) generic_lane_offsets<BITS>(lg, gword, gshift);
  }
  // tile t: rows [16 * tile, ..) of expert e of a stack with n rows
  __device__ inline void tile(int t, const Stack& k, int e, int64_t row, int64_t n) {
    const int64_t rr = row < n ? row : n - 1;
    w[t] = k.w + e * k.w_expert_stride + rr * k.w_row_stride;
    s[t] = k.s + e * k.sb_expert_stride + rr * k.sb_row_stride;
    b[t] = k.b + e * k.sb_expert_stride + rr * k.sb_row_stride;
  }
  __device__ inline void load(Data& r, int slot) const {
#pragma unroll
    for (int t = 0; t < TN; ++t)
      load_slot<BITS, GS>(r.d[t], w[t] + (int64_t)slot * S::kRowWordsPerSlot, s[t] + slot * S::kGroups,
                          b[t] + slot * S::kGroups, lg, gword, row_words - slot * S::kRowWordsPerSlot,
                          K - slot * S::kSpan, narrow);
    const int sub = kSub8 && (lg == 1 || lg == 2) ? 3 - lg : lg;   // 8-bit words arrive with groups 1 and 2 swapped
#pragma unroll
    for (int c = 0; c < kSteps; ++c) {
      const int k = slot * S::kSpan + 32 * c + 8 * sub;
#pragma unroll
      for (int m = 0; m < MT; ++m) r.x[m][c] = x[m] != nullptr && k < K ? *(const u32x4*)(x[m] + k) : u32x4{0u, 0u, 0u, 0u};
    }
  }
  __device__ inline void consume(const Data& r, int slot, f32x4 (&acc)[TN][MT]) const {
    constexpr int SPG = GS / 32;
    const uint32_t one2 = T::pack2(1.0f, 1.0f);
    const u32x4 ones = {one2, one2, one2, one2};
    const f32x4 zero4 = {0.f, 0.f, 0.f, 0.f};
    decode::SlotCodes<BITS, GS> rc[TN];
#pragma unroll
    for (int t = 0; t < TN; ++t) rc[t] = slot_reorder<BITS, GS>(r.d[t]);
    f32x4 part[TN][MT], sum[MT];
#pragma unroll
    for (int c = 0; c < kSteps; ++c) {
      typename T::v8 q[TN];
#pragma unroll
      for (int t = 0; t < TN; ++t) q[t] = as_v8<T>(slot_codes<T, BITS, GS>(r.d[t], rc[t], c, gshift));
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const typename T::v8 av = as_v8<T>(BITS == 4 ? interleave_even_odd(r.x[m][c]) : r.x[m][c]);
        sum[m] = T::mfma(av, as_v8<T>(ones), c % SPG == 0 ? zero4 : sum[m]);
#pragma unroll
        for (int t = 0; t < TN; ++t) part[t][m] = T::mfma(av, q[t], c % SPG == 0 ? zero4 : part[t][m]);
      }
      if ((c + 1) % SPG == 0) {
        const int g = c / SPG;
        // groups past K (the last slot of a K that is no multiple of the span) scale by zero
        const bool ok = slot * S::kSpan + g * GS < K;
#pragma unroll
        for (int t = 0; t < TN; ++t) {
          const float sv = ok ? T::to_f32(r.d[t].s.get(g)) : 0.f, bv = ok ? T::to_f32(r.d[t].b.get(g)) : 0.f;
#pragma unroll
          for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              acc[t][m][i] = __builtin_fmaf(sv, part[t][m][i], __builtin_fmaf(bv, sum[m][i], acc[t][m][i]));
        }
      }
    }
  }
  __device__ inline void run(int s0, int s1, f32x4 (&acc)[TN][MT]) const {
    Data ring[kDepth];
#pragma unroll
    for (int i = 0; i < kDepth; ++i)
      if (s0 + i < s1) load(ring[i], s0 + i);
    for (int base = s0; base < s1; base += kDepth) {
#pragma unroll
      for (int i = 0; i < kDepth; ++i) {
        if (base + i >= s1) break;
        consume(ring[i], base + i, acc);
        if (base + i + kDepth < s1) load(ring[i], base + i + kDepth);
      }
    }
  }
};

// Whether a slot's scales (and biases) can be read as one load: every row, expert and array
// start aligned to the slot's groups.
template <int KG>
__device__ inline bool sb_aligned(const Stack& k) {
  if constexpr (KG == 1) {
    return true;
  } else {
    return (((uintptr_t)k.s | (uintptr_t)k.b) % (2 * KG)) == 0 && (uint64_t)(k.sb_row_stride * 2) % (2 * KG) == 0 &&
           (uint64_t)(k.sb_expert_stride * 2) % (2 * KG) == 0;
  }
}

// h[row of (t, e)][n] = w_te silu(g) u.  Workgroup (x, y): the y-th expert in use, tiles
// [x * kWaves / parts, ..) of inter; `parts` waves share a tile, each a stretch of hidden, and
// meet in LDS.
template <class T, int BITS, int GS, int MT>
__global__ __launch_bounds__(kThreads) void gate_up_kernel(const MoeArgs a) {
  using S = Slot<BITS, GS>;
  __shared__ Routing r;
  __shared__ f32x4 hand[kWaves][2 * MT][64];
  route<T>(a, r);
  const int words = (a.experts + 31) >> 5;
  int in_use = 0;
  for (int i = 0; i < words; ++i) in_use += __popc(r.any[i]);
  if (blockIdx.x == 0 && blockIdx.y == 0) {
    // the plan that the second kernel reads
    if (threadIdx.x == 0) a.active[0] = in_use;
    for (int e = threadIdx.x; e < a.experts; e += kThreads) {
      if (!((r.any[e >> 5] >> (e & 31)) & 1u)) continue;
      const int n = rank_of(r.any, e);
      a.active[1 + n] = e;
      for (int t = 0; t < kMaxTokens; ++t) {
        const bool use = t < a.tokens && ((r.chosen[t][e >> 5] >> (e & 31)) & 1u);
        a.row_of[n * kMaxTokens + t] = use ? (int16_t)(t * a.top_k + rank_of(r.chosen[t], e)) : (int16_t)-1;
      }
    }
  }
  const int n_th = blockIdx.y;
  if (n_th >= in_use) return;                 // the same in the whole workgroup
  int e = 0;                                  // the n_th expert in use
  for (int i = 0, left = n_th; i < words; ++i) {
    const int have = __popc(r.any[i]);
    if (left < have) {
      uint32_t m = r.any[i];
      for (; left > 0; --left) m &= m - 1u;
      e = 32 * i + __ffs(m) - 1;
      break;
    }
    left -= have;
  }
  const int lane = threadIdx.x & 63, lg = lane >> 4, col = lane & 15;
  const int wave = threadIdx.x >> 6;
  const int part = wave % a.parts, group = wave / a.parts;
  const int64_t n0 = ((int64_t)blockIdx.x * (kWaves / a.parts) + group) * 16;
  const bool live = n0 < a.inter;
  f32x4 acc[2][MT];
#pragma unroll
  for (int t = 0; t < 2; ++t)
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[t][m] = f32x4{0.f, 0.f, 0.f, 0.f};
  if (live) {
    Stream<T, BITS, GS, 2, MT> st;
    st.setup(a, a.hidden);
    st.narrow = !sb_aligned<S::kGroups>(a.gate) || !sb_aligned<S::kGroups>(a.up);
    st.tile(0, a.gate, e, n0 + col, a.inter);
    st.tile(1, a.up, e, n0 + col, a.inter);
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const int t = 16 * m + col;
      const bool use = t < a.tokens && ((r.chosen[t][e >> 5] >> (e & 31)) & 1u);
      st.x[m] = use ? a.x + t * a.x_stride : nullptr;
    }
    const int slots = (a.hidden + S::kSpan - 1) / S::kSpan, per = (slots + a.parts - 1) / a.parts;
    st.run(part * per, min(slots, (part + 1) * per), acc);
  }
  if (a.parts > 1) {
    if (part != 0) {
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int m = 0; m < MT; ++m) hand[wave][t * MT + m][lane] = acc[t][m];
    }
    __syncthreads();
    if (part != 0) return;
    for (int p = 1; p < a.parts; ++p)
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int m = 0; m < MT; ++m) acc[t][m] += hand[wave + p][t * MT + m][lane];
  }
  const int64_t n = n0 + col;
  if (n >= a.inter) return;
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int t = 16 * m + 4 * lg + i;
      if (t >= a.tokens || !((r.chosen[t][e >> 5] >> (e & 31)) & 1u)) continue;
      const float w = expf(T::to_f32(a.router[t * a.router_stride + e]) - r.top[t]) * r.inv[t];
      const float g = acc[0][m][i];
      const float v = w * (g / (1.0f + expf(-g))) * acc[1][m][i];
      a.h[(int64_t)(t * a.top_k + rank_of(r.chosen[t], e)) * a.inter + n] = T::from_f32(v);
    }
}

// y_t += h Wd^T over the experts.  Workgroup (x, y): tile x of hidden, split y; its waves and
// the splits share the pieces (expert in use, one of `cuts` stretches of inter) evenly.  The
// waves' sums meet in LDS, in wave order; the splits' in `part`, in split order.
template <class T, int BITS, int GS, int MT>
__global__ __launch_bounds__(kThreads) void down_kernel(const MoeArgs a) {
  using S = Slot<BITS, GS>;
  __shared__ f32x4 hand[kWaves][MT][64];
  const int lane = threadIdx.x & 63, lg = lane >> 4, col = lane & 15;
  const int wave = threadIdx.x >> 6;
  const int64_t n0 = (int64_t)blockIdx.x * 16;
  f32x4 acc[1][MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) acc[0][m] = f32x4{0.f, 0.f, 0.f, 0.f};
  const int slots = (a.inter + S::kSpan - 1) / S::kSpan, per = (slots + a.cuts - 1) / a.cuts;
  const int pieces = a.active[0] * a.cuts, workers = kWaves * a.splits;
  Stream<T, BITS, GS, 1, MT> st;
  st.setup(a, a.inter);
  st.narrow = !sb_aligned<S::kGroups>(a.down);
  for (int p = blockIdx.y * kWaves + wave; p < pieces; p += workers) {
    const int n_th = p / a.cuts, cut = p - n_th * a.cuts;
    const int e = a.active[1 + n_th];
    st.tile(0, a.down, e, n0 + col, a.hidden);
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const int row = a.row_of[n_th * kMaxTokens + 16 * m + col];
      st.x[m] = row >= 0 ? a.h + (int64_t)row * a.inter : nullptr;
    }
    st.run(cut * per, min(slots, (cut + 1) * per), acc);
  }
  if (wave != 0) {
#pragma unroll
    for (int m = 0; m < MT; ++m) hand[wave][m][lane] = acc[0][m];
  }
  __syncthreads();
  if (wave != 0) return;
  for (int w = 1; w < kWaves; ++w)
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[0][m] += hand[w][m][lane];
  const int64_t n = n0 + col;
  if (n >= a.hidden) return;
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int t = 16 * m + 4 * lg + i;
      if (t >= a.tokens) continue;
      if (a.splits > 1)
        a.part[((int64_t)blockIdx.y * a.tokens + t) * a.hidden + n] = acc[0][m][i];
      else
        a.y[t * a.y_stride + n] = T::from_f32(acc[0][m][i]);
    }
}

template <class T, int BITS, int GS>
hipError_t launch_group(const MoeArgs& a, hipStream_t stream, bool down) {
  if (down) {
    const dim3 grid((unsigned)((a.hidden + 15) / 16), (unsigned)a.splits);
    if (a.tokens <= 16)
      hipLaunchKernelGGL((down_kernel<T, BITS, GS, 1>), grid, dim3(kThreads), 0, stream, a);
    else
      hipLaunchKernelGGL((down_kernel<T, BITS, GS, 2>), grid, dim3(kThreads), 0, stream, a);
  } else {
    const int tiles = (a.inter + 15) / 16, per = kWaves / a.parts;
    const int experts = a.tokens * a.top_k < a.experts ? a.tokens * a.top_k : a.experts;
    const dim3 grid((unsigned)((tiles + per - 1) / per), (unsigned)experts);
    if (a.tokens <= 16)
      hipLaunchKernelGGL((gate_up_kernel<T, BITS, GS, 1>), grid, dim3(kThreads), 0, stream, a);
    else
      hipLaunchKernelGGL((gate_up_kernel<T, BITS, GS, 2>), grid, dim3(kThreads), 0, stream, a);
  }
  return hipGetLastError();
}

template <int BITS>
hipError_t launch_bits(const MoeArgs& a, hipStream_t stream, bool down) {
  const int gs = down ? a.down.group_size : a.gate.group_size;
  if (a.dtype == 1)
    return gs == 32   ? launch_group<Bf16, BITS, 32>(a, stream, down)
           : gs == 64 ? launch_group<Bf16, BITS, 64>(a, stream, down)
                      : launch_group<Bf16, BITS, 128>(a, stream, down);
  return gs == 32   ? launch_group<Fp16, BITS, 32>(a, stream, down)
         : gs == 64 ? launch_group<Fp16, BITS, 64>(a, stream, down)
                    : launch_group<Fp16, BITS, 128>(a, stream, down);
}

}  // namespace moe
}  // namespace qmm
