// Mixture-of-experts layer for up to 32 tokens over quantized expert stacks:
//     S_t  = the top_k largest router logits of token t (equal ones: lower expert),
//     w_te = softmax over S_t (renormalize) or over all experts, taken at e,
//     y_t  = sum_{e in S_t}  w_te ( silu(Wg_e x_t) * (Wu_e x_t) ) Wd_e^T.
//
// The layer reads each chosen expert's weights once and little else, so it is bound by that
// stream (and, for one token, by latency).  Three kernels: the products with Wg and Wu
// together, since both take x and the activation needs both; the product with Wd, for every
// (token, choice) pair; and the sum over a token's choices.
//
// Routing is not a kernel of its own.  A workgroup of the first kernel works for one expert e
// and only has to know which tokens chose it: token t did if fewer than top_k of its logits
// beat logit e, one pass over the logits.  The weights stay unnormalised, exp(l_te - max l_t),
// until the last kernel has every chosen expert of a token and divides by their sum.
//
// Streams: a wave takes two 16-row tiles of weights (the same rows of Wg and Wu, or 32 rows of
// Wd) and a stretch of K, with kDepth slots of loads in flight.  The activations of the
// expert's tokens (up to 16 per pass over the weights; an expert seldom has more) are staged
// in LDS in operand order: fetched from global memory they would share the memory counter
// with the weights, which retires loads in order, and take the registers of three more slots.
// No load is conditional: addresses are clamped into the row, and what a clamp repeats is
// multiplied by zero.
// Arithmetic per output as in the decode kernels, s * sum xq + b * sum x per group with exact
// integer codes and float32 sums; sum x comes from a product with an all-ones operand.
// h = silu(g) u reaches the second product as two bfloat16 operands, its leading bits and the
// rest (2^-17 of it is lost): the one rounding that a single operand would add is as large as
// the output's own.  In fp16 calls too, where the codes are exact in either type: h there may
// pass 65504, or lie where fp16 has few bits, and y still be an ordinary fp16 number.
//
// What bounds it: the stream, at 3.6 TB/s of the 5.2 of a copy -- each workgroup's first
// loads wait for its users and its activations, and the last ones leave CUs idle.  Measured:
// 32 tokens, 128 experts of [704, 1408] in 8 bits, top 8: 104 us, 374 MB (67 + 36 + 5); 7 tokens,
// 8 experts of [14336, 4096] in 4 bits, top 2: 179 us, 649 MB (106 + 71 + 5); one token, 8 of 64 experts of
// [1024, 2048] in 4 bits: 20 us for 28 MB, of which three launches take 7 and the chain of
// logits, expert, weights and sums most of the rest.
#pragma once

#include "decode_impl.hpp"
#include "moe.hpp"

namespace qmm {
namespace moe {

using decode::generic_lane_offsets;
using decode::SbRegs;
using decode::Slot;
using decode::slot_codes;
using decode::SlotData;
using decode::slot_reorder;

constexpr int kThreads = 64 * kWaves;
constexpr int kWorkgroups = 3;       // per compute unit: 168 registers per thread

// Order key of a 16-bit float: larger values have larger keys, NaN the largest.
template <class T>
__device__ inline uint32_t order_key(uint32_t b) {
  constexpr uint32_t kInf = T::kDtype == 2 ? 0x7C00u : 0x7F80u;
  if ((b & 0x7FFFu) > kInf) return 0xFFFFu;
  if (b == 0x8000u) b = 0u;                     // -0 and +0 are equal
  return (b & 0x8000u) ? (~b & 0xFFFFu) : (b | 0x8000u);
}

// Largest v of the wave, in every lane: row-local steps, then the row broadcasts.
__device__ inline uint32_t wave_max(uint32_t v) {
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, false));    // quad_perm [1,0,3,2]
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, false));    // quad_perm [2,3,0,1]
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x141, 0xF, 0xF, false));   // row_half_mirror
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x140, 0xF, 0xF, false));   // row_mirror
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x142, 0xA, 0xF, false));   // row_bcast:15
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x143, 0xC, 0xF, false));   // row_bcast:31
  return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

// The expert with rank n (0: the largest logit) of a token's logits, by one wave: n + 1 rounds
// of the largest (key, lower expert first) word below the last one.
template <class T>
__device__ inline int expert_of_rank(const uint16_t* logits, int experts, int n, int lane) {
  constexpr int kRegs = kMaxExperts / 64;
  uint32_t word[kRegs];
#pragma unroll
  for (int j = 0; j < kRegs; ++j) {
    const int e = 64 * j + lane;
    word[j] = e < experts ? (order_key<T>(logits[e]) << 9) | (uint32_t)(kMaxExperts - 1 - e) : 0u;
  }
  uint32_t best = 0xFFFFFFFFu;
  for (int i = 0; i <= n; ++i) {
    uint32_t m = 0u;
#pragma unroll
    for (int j = 0; j < kRegs; ++j) m = word[j] < best ? max(m, word[j]) : m;
    best = wave_max(m);
  }
  return kMaxExperts - 1 - (int)(best & (kMaxExperts - 1));
}

// The tokens that chose an expert, in LDS, ascending.
struct Users {
  int16_t token[kMaxTokens];
  int16_t pair[kMaxTokens];     // t * top_k + which of t's choices it is
  float share[kMaxTokens];      // exp(l_te - max l_t), over the sum of all experts unless renormalised
  int16_t pair_of[kMaxTokens];  // by token, -1: not chosen
  float share_of[kMaxTokens];
  int count;
};

// Compact pair_of (and share_of) into the ascending lists, by the first wave; with the barriers.
__device__ inline void list_users(const MoeArgs& a, Users& u) {
  __syncthreads();
  if (threadIdx.x < 64) {
    const bool use = (int)threadIdx.x < a.tokens && u.pair_of[threadIdx.x] >= 0;
    const uint64_t m = __ballot(use);
    if (use) {
      const int i = __popcll(m & ((1ull << threadIdx.x) - 1));
      u.token[i] = (int16_t)threadIdx.x;
      u.pair[i] = u.pair_of[threadIdx.x];
      u.share[i] = u.share_of[threadIdx.x];
    }
    if (threadIdx.x == 0) u.count = __popcll(m);
  }
  __syncthreads();
}

// Fill u from the router logits; 8 to 64 lanes per token.
template <class T>
__device__ inline void find_users(const MoeArgs& a, int e, Users& u) {
  const int per = a.tokens > 16 ? 8 : (a.tokens > 8 ? 16 : (a.tokens > 4 ? 32 : 64));   // tokens * per <= kThreads
  const int t = threadIdx.x / per, i = threadIdx.x & (per - 1);
  if (t < a.tokens) {
    const uint16_t* logits = a.router + t * a.router_stride;
    const uint32_t mine = (order_key<T>(logits[e]) << 9) | (uint32_t)(kMaxExperts - 1 - e);
    uint32_t top = 0u;
    int beats = 0;
#pragma unroll 4
    for (int j = i; j < a.experts; j += per) {
      const uint32_t key = order_key<T>(logits[j]);
      beats += ((key << 9) | (uint32_t)(kMaxExperts - 1 - j)) > mine ? 1 : 0;
      top = max(top, key);
    }
    for (int d = 1; d < per; d <<= 1) {
      beats += __shfl_xor(beats, d);
      top = max(top, (uint32_t)__shfl_xor(top, d));
    }
    const float top_l = T::to_f32((top & 0x8000u) ? (top & 0x7FFFu) : (~top & 0xFFFFu));
    float sum = 1.0f;
    if (!a.renormalize) {
      sum = 0.f;
#pragma unroll 4
      for (int j = i; j < a.experts; j += per) sum += expf(T::to_f32(logits[j]) - top_l);
      for (int d = 1; d < per; d <<= 1) sum += __shfl_xor(sum, d);
    }
    if (i == 0) {
      u.pair_of[t] = beats < a.top_k ? (int16_t)(t * a.top_k + beats) : (int16_t)-1;
      u.share_of[t] = expf(T::to_f32(logits[e]) - top_l) / sum;
    }
  }
  list_users(a, u);
}

// Fill u from the first kernel's pairs.
__device__ inline void read_users(const MoeArgs& a, int e, Users& u) {
  if (threadIdx.x < kMaxTokens) u.pair_of[threadIdx.x] = -1;
  __syncthreads();
  for (int i = threadIdx.x; i < a.tokens * a.top_k; i += kThreads)
    if (a.pair_expert[i] == e) u.pair_of[i / a.top_k] = (int16_t)i;
  list_users(a, u);
}

// The only token's pair, which nobody else has (by_pair with one token): nothing to look up.
__device__ inline void only_user(int pair, Users& u) {
  if (threadIdx.x == 0) {
    u.token[0] = 0;
    u.pair[0] = (int16_t)pair;
    u.count = 1;
  }
  __syncthreads();
}

// [x0 .. x7] -> [x0, x2, x4, x6, x1, x3, x5, x7], the order in which 4-bit codes are expanded.
__device__ inline u32x4 even_odd(u32x4 u) {
  return u32x4{__builtin_amdgcn_perm(u.y, u.x, 0x05040100u), __builtin_amdgcn_perm(u.w, u.z, 0x05040100u),
               __builtin_amdgcn_perm(u.y, u.x, 0x07060302u), __builtin_amdgcn_perm(u.w, u.z, 0x07060302u)};
}

// One wave's weight stream of two 16-row tiles, through buffer descriptors over one expert: a
// slot's offset is a scalar, the lane's row a register, rows past the last read as zeros, and
// what a slot reads past its row's end is multiplied by zero.  Scales and biases are of type T,
// the operands of the product of type X.  The scales and biases of a
// round of kDepth slots are one load per tile, a round ahead: one load per slot asked for
// twice as many cache lines as the codes (16 rows of two bytes each).  NARROW: they are read
// one halfword at a time (rows, experts or arrays that are not whole words).
template <class T, class X, int BITS, int GS, bool NARROW>
struct Stream {
  using S = Slot<BITS, GS>;
  static constexpr int TN = 2;
  static constexpr int kBits = BITS;
  static constexpr int kSteps = S::kSteps;
  static constexpr int KG = S::kGroups;
  static constexpr int kDepth = S::kWords <= 4 && KG < 4 ? 4 : 2;   // slots in flight
  static constexpr int NH = kDepth * KG;                            // groups of a round
  static constexpr int kSlotX = kSteps * 4;                         // 16-byte operand entries of a slot per row

  __amdgpu_buffer_rsrc_t w_rs[TN], s_rs[TN], b_rs[TN];
  int w_voff[TN], sb_voff[TN];    // the lane's row of each tile, bytes
  int w_row_bytes, sb_row_bytes;
  int K, lg, col;
  uint32_t gshift;
  SlotData<BITS, GS> ring[kDepth][TN];
  struct Sb {
    SbRegs<NH> s[TN], b[TN];
  };

  // Tile t's weights: expert e of a stack with n rows.
  __device__ inline void setup(int t, const Stack& k, int e, int64_t n, int cols) {
    K = cols;
    lg = (threadIdx.x & 63) >> 4;
    col = threadIdx.x & 15;
    w_row_bytes = (int)(k.w_row_stride * 4);
    sb_row_bytes = (int)(k.sb_row_stride * 2);
    gshift = 0u;
    int gword = 0;
    if constexpr (BITS != 4 && BITS != 8) generic_lane_offsets<BITS>(lg, gword, gshift);
    const uint32_t w_bytes = (uint32_t)(n - 1) * (uint32_t)w_row_bytes + (uint32_t)(K / 32 * BITS * 4);
    const uint32_t sb_bytes = (uint32_t)(n - 1) * (uint32_t)sb_row_bytes + (uint32_t)(K / GS * 2);
    w_rs[t] = decode::make_rsrc(k.w + e * k.w_expert_stride, w_bytes);
    s_rs[t] = decode::make_rsrc(k.s + e * k.sb_expert_stride, sb_bytes);
    b_rs[t] = decode::make_rsrc(k.b + e * k.sb_expert_stride, sb_bytes);
    lane_word = BITS == 4 || BITS == 8 ? 16 * lg : 4 * gword;
  }
  int lane_word;                  // byte of the lane's words in a slot
  // Tile t starts at row `row`.
  __device__ inline void tile(int t, int row) {
    w_voff[t] = (row + col) * w_row_bytes + lane_word;
    sb_voff[t] = (row + col) * sb_row_bytes;
  }
  __device__ inline void load(SlotData<BITS, GS> (&d)[TN], int slot) const {
    const int soff = slot * S::kRowWordsPerSlot * 4;
#pragma unroll
    for (int t = 0; t < TN; ++t) {
      if constexpr (BITS == 4 || BITS == 8) {
        decode::load_slot_buf<BITS, GS, false>(d[t], w_rs[t], s_rs[t], b_rs[t], w_voff[t], soff, 0, 0);
      } else {
#pragma unroll
        for (int c = 0; c < kSteps; ++c) {
          d[t].w[2 * c] = __builtin_amdgcn_raw_buffer_load_b32(w_rs[t], w_voff[t] + 4 * c * BITS, soff, 0);
          d[t].w[2 * c + 1] = __builtin_amdgcn_raw_buffer_load_b32(w_rs[t], w_voff[t] + 4 * c * BITS + 4, soff, 0);
        }
      }
    }
  }
  __device__ inline void load_sb(Sb& r, int slot) const {
    const int soff = slot * KG * 2;
#pragma unroll
    for (int t = 0; t < TN; ++t) {
      if constexpr (NARROW) {
        decode::load_sb_buf_narrow<NH>(r.s[t], s_rs[t], sb_voff[t], soff);
        decode::load_sb_buf_narrow<NH>(r.b[t], b_rs[t], sb_voff[t], soff);
      } else {
        decode::load_sb_buf<NH>(r.s[t], s_rs[t], sb_voff[t], soff);
        decode::load_sb_buf<NH>(r.b[t], b_rs[t], sb_voff[t], soff);
      }
    }
  }
  // x: the chunk's staged operands, entry (((slot - x0) * kSteps + step) * 4 + lane group) << xrl,
  // plus `plane` entries for the rest; 2^xrl rows.  The slot is the nth of its round.
  template <int PLANES>
  __device__ inline void consume(const SlotData<BITS, GS> (&d)[TN], const Sb& sb, int nth, int slot, const u32x4* x,
                                 int plane, int xrl, f32x4 (&acc)[TN]) const {
    constexpr int SPG = GS / 32;
    const uint32_t one2 = X::pack2(1.0f, 1.0f);
    const u32x4 ones = {one2, one2, one2, one2};
    const f32x4 zero4 = {0.f, 0.f, 0.f, 0.f};
    const bool whole = (slot + 1) * S::kSpan <= K;
    decode::SlotCodes<BITS, GS> rc[TN];
#pragma unroll
    for (int t = 0; t < TN; ++t) rc[t] = slot_reorder<BITS, GS>(d[t]);
    const int row = col & ((1 << xrl) - 1);
    f32x4 part[TN], sum;
#pragma unroll
    for (int c = 0; c < kSteps; ++c) {
      typename X::v8 q[TN];
#pragma unroll
      for (int t = 0; t < TN; ++t) q[t] = as_v8<X>(slot_codes<X, BITS, GS>(d[t], rc[t], c, gshift));
#pragma unroll
      for (int p = 0; p < PLANES; ++p) {
        const typename X::v8 av = as_v8<X>(x[p * plane + ((c * 4 + lg) << xrl) + row]);
        const bool fresh = c % SPG == 0 && p == 0;
        sum = X::mfma(av, as_v8<X>(ones), fresh ? zero4 : sum);
#pragma unroll
        for (int t = 0; t < TN; ++t) part[t] = X::mfma(av, q[t], fresh ? zero4 : part[t]);
      }
      if ((c + 1) % SPG == 0) {
        const int g = c / SPG;
        const bool ok = whole || slot * S::kSpan + g * GS < K;   // groups past K scale by zero
#pragma unroll
        for (int t = 0; t < TN; ++t) {
          const float sv = ok ? T::to_f32(sb.s[t].get(nth * KG + g)) : 0.f;
          const float bv = ok ? T::to_f32(sb.b[t].get(nth * KG + g)) : 0.f;
#pragma unroll
          for (int i = 0; i < 4; ++i)
            acc[t][i] = __builtin_fmaf(sv, part[t][i], __builtin_fmaf(bv, sum[i], acc[t][i]));
        }
      }
    }
  }
};

// Whether a stack's scales and biases can be read in whole words: every row, expert and array
// starts on one, and a row ends on one.
template <int GS>
inline bool sb_wide(const Stack& k, int64_t K) {
  return K / GS % 2 == 0 && (((uintptr_t)k.s | (uintptr_t)k.b) % 4) == 0 && k.sb_row_stride % 2 == 0 &&
         k.sb_expert_stride % 2 == 0;
}

// How a workgroup walks its tiles: tile units first, first + step, .. below units; a unit is
// kWaves / parts tile pairs, one per group of `parts` waves, each of which takes an equal
// stretch of every chunk of the slots [k0, k1); a chunk is what LDS holds of the activations.
struct Walk {
  int first, step, units;
  int parts, part;
  int k0, k1, chunk;
};

// The products of the walk's tiles with up to 16 rows of activations, PLANES operand planes
// each.  row(m): address of row m < rows (plane p at + p * plane_stride).  set_tiles(st, unit)
// points the stream's loads at a unit; finish(unit, acc) gets its sums, in the waves of part 0.
// The ring of loads runs on over chunks and tiles.
template <int PLANES, class St, class Row, class Tiles, class Finish>
struct Products {
  static constexpr int kDepth = St::kDepth, kSlotX = St::kSlotX;
  St& st;
  const Walk& w;
  // the next slot to load
  int unit, c0, at;

  // slots of a wave's stretch of a chunk; the loop goes over whole rounds of the ring, whose last
  // slots may be the next wave's (loaded, and not used)
  __device__ inline int stretch(int c) const { return stretch_of(min(w.chunk, w.k1 - c), w.parts); }
  __device__ static inline int whole_rounds(int n) { return (n + kDepth - 1) / kDepth * kDepth; }
  __device__ inline int next_slot() const { return c0 + w.part * stretch(c0) + at; }
  __device__ inline void load_next(int i, Tiles& set_tiles) {
    st.load(st.ring[i], next_slot() + i);
    if (i + 1 < kDepth) return;
    at += kDepth;
    if (at >= stretch(c0)) {
      at = 0;
      c0 += w.chunk;
      if (c0 >= w.k1) {
        c0 = w.k0;
        unit += w.step;                  // rows past the last unit read as zeros
        set_tiles(st, unit);
      }
    }
  }
  __device__ inline void stage(int rows, Row& row, int64_t plane_stride, u32x4* xs, int k, int n, int xrl) {
    const int plane = (n * kSlotX) << xrl, entries = plane * PLANES;
    constexpr int kBatch = 4;
    for (int e0 = threadIdx.x; e0 < entries; e0 += kBatch * kThreads) {
      u32x4 v[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int en = min(e0 + i * kThreads, entries - 1);
        const int p = en >= plane ? 1 : 0, x = en - p * plane;
        const int m = min(x & ((1 << xrl) - 1), rows - 1), kk = k * St::S::kSpan + 8 * (x >> xrl);
        v[i] = *(const u32x4*)(row(m) + p * plane_stride + min(kk, st.K - 8));
        if (kk >= st.K) v[i] = u32x4{0u, 0u, 0u, 0u};
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int en = e0 + i * kThreads;
        if (en >= entries) break;
        const int p = en >= plane ? 1 : 0, x = en - p * plane;
        const int m = x & ((1 << xrl) - 1), k8 = x >> xrl;   // 8 consecutive k
        xs[p * plane + (((k8 & ~3) + decode::lane_group_of_sub<St::kBits>(k8 & 3)) << xrl) + m] =
            St::kBits == 4 ? even_odd(v[i]) : v[i];
      }
    }
  }
  __device__ inline void run(int rows, Row row, int64_t plane_stride, Tiles set_tiles, Finish finish, int xrl,
                             u32x4* xs, f32x4* hand) {
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    unit = w.first;
    c0 = w.k0;
    at = 0;
    set_tiles(st, unit);
    typename St::Sb sb, sb_next;
    st.load_sb(sb, next_slot());
#pragma unroll
    for (int i = 0; i < kDepth; ++i) load_next(i, set_tiles);
    const bool resident = w.k1 - w.k0 <= w.chunk;     // one chunk: staged once for all tiles
    if (resident) {
      stage(rows, row, plane_stride, xs, w.k0, w.k1 - w.k0, xrl);
      lds_barrier();
    }
    for (int u = w.first; u < w.units; u += w.step) {
      f32x4 acc[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
      for (int c = w.k0; c < w.k1; c += w.chunk) {
        const int c1 = min(w.k1, c + w.chunk), per = stretch(c);
        const int s0 = c + w.part * per, s1 = min(c1, s0 + per);
        const int plane = ((c1 - c) * kSlotX) << xrl;
        if (!resident) {
          lds_barrier();
          stage(rows, row, plane_stride, xs, c, c1 - c, xrl);
          lds_barrier();
        }
        for (int base = s0; base < s0 + whole_rounds(per); base += kDepth) {
          st.load_sb(sb_next, next_slot());
#pragma unroll
          for (int i = 0; i < kDepth; ++i) {
            if (base + i < s1)
              st.template consume<PLANES>(st.ring[i], sb, i, base + i, xs + (((base + i - c) * kSlotX) << xrl), plane,
                                          xrl, acc);
            load_next(i, set_tiles);
          }
          sb = sb_next;
        }
      }
      if (w.parts > 1) {
        if (w.part != 0) {
          hand[(wave * 2 + 0) * 64 + lane] = acc[0];
          hand[(wave * 2 + 1) * 64 + lane] = acc[1];
        }
        lds_barrier();
        if (w.part == 0)
          for (int p = 1; p < w.parts; ++p) {
            acc[0] += hand[((wave + p) * 2 + 0) * 64 + lane];
            acc[1] += hand[((wave + p) * 2 + 1) * 64 + lane];
          }
        lds_barrier();
      }
      if (w.part == 0) finish(u, acc);
    }
    lds_barrier();                                    // the next pass stages over xs
  }
};

// log2 of the staged rows, and the slots of a chunk of `rows` rows (PLANES planes).
template <int PLANES, class St>
__device__ inline int fit_chunk(int rows, int parts, int* xrl) {
  int l = 0;
  while ((1 << l) < rows) ++l;
  *xrl = l;
  static_assert(St::kDepth % 2 == 0 && chunk_of(St::kSlotX * PLANES, 4, kWaves * St::kDepth) >= 2, "even, not empty");
  return chunk_of(St::kSlotX * PLANES, l, parts * St::kDepth);
}

// Workgroup (x, y) of both product kernels: y is an expert or, when the call has fewer (token,
// choice) pairs than there are experts (`by_pair`), the pair whose expert it is, unless an
// earlier token has the same; x the workgroup's first tile unit.

// h rows of expert e's tokens.
template <class T, int BITS, int GS, bool NARROW>
__global__ __launch_bounds__(kThreads, kWorkgroups) void gate_up_kernel(const MoeArgs a, const int by_pair) {
  using St = Stream<T, T, BITS, GS, NARROW>;
  __shared__ Users u;
  __shared__ u32x4 xs[kXBytes / 16];
  __shared__ f32x4 hand[kWaves * 2 * 64];
  const int lane = threadIdx.x & 63, lg = lane >> 4, col = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int group = wave / a.parts, per = kWaves / a.parts;
  int e = blockIdx.y, pair_token = 0;
  if (by_pair) {
    pair_token = blockIdx.y / a.top_k;
    e = expert_of_rank<T>(a.router + pair_token * a.router_stride, a.experts, blockIdx.y - pair_token * a.top_k, lane);
  }
  const bool only = by_pair && a.tokens == 1;
  if (only)
    only_user(blockIdx.y, u);
  else
    find_users<T>(a, e, u);
  // the same in the whole workgroup: nobody uses the expert, or an earlier pair's workgroup does it
  if (u.count == 0 || (by_pair && u.token[0] != pair_token)) return;
  St st;
  st.setup(0, a.gate, e, a.inter, a.hidden);
  st.setup(1, a.up, e, a.inter, a.hidden);
  const auto first_row = [&](int unit) { return (unit * per + group) * 16; };
  const auto set_tiles = [&](St& t, int unit) {
    t.tile(0, first_row(unit));
    t.tile(1, first_row(unit));
  };
  const auto publish = [&]() {
    if (blockIdx.x == 0 && (int)threadIdx.x < u.count) {
      a.pair_expert[u.pair[threadIdx.x]] = e;
      a.pair_share[u.pair[threadIdx.x]] = u.share[threadIdx.x];
    }
  };
  if (!only) publish();
  for (int r0 = 0; r0 < u.count; r0 += 16) {   // a second pass only for more than 16 tokens
    const int rows = min(16, u.count - r0);
    int xrl;
    const int chunk = fit_chunk<1, St>(rows, a.parts, &xrl);
    const Walk w{(int)blockIdx.x, (int)gridDim.x, (int)((a.inter + 16 * per - 1) / (16 * per)), a.parts,
                 wave - group * a.parts, 0, (a.hidden + St::S::kSpan - 1) / St::S::kSpan, chunk};
    const auto row = [&](int m) { return a.x + (int64_t)u.token[r0 + m] * a.x_stride; };
    const auto finish = [&](int unit, const f32x4 (&acc)[2]) {
      const int n = first_row(unit) + col;
      if (n >= a.inter) return;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = r0 + 4 * lg + i;
        if (r >= u.count) continue;
        const float g = acc[0][i];
        const float v = g / (1.0f + expf(-g)) * acc[1][i];
        uint16_t* h = a.h + (int64_t)u.pair[r] * 2 * a.inter + n;
        const uint16_t hi = Bf16::from_f32(v);
        h[0] = hi;
        h[a.inter] = Bf16::from_f32(v - Bf16::to_f32(hi));
      }
    };
    Products<1, St, decltype(row), decltype(set_tiles), decltype(finish)> p{st, w};
    p.run(rows, row, 0, set_tiles, finish, xrl, xs, hand);
  }
  if (only && blockIdx.x == 0) {               // the share is not needed before the last kernel
    find_users<T>(a, e, u);
    publish();
  }
}

// out[pair][z] = h Wd_e^T over the z-th stretch of inter, of expert e's pairs, in float32.
template <class T, int BITS, int GS, bool NARROW>
__global__ __launch_bounds__(kThreads, kWorkgroups) void down_kernel(const MoeArgs a, const int by_pair) {
  using St = Stream<T, Bf16, BITS, GS, NARROW>;
  __shared__ Users u;
  __shared__ u32x4 xs[kXBytes / 16];
  __shared__ f32x4 hand[kWaves * 2 * 64];
  const int lane = threadIdx.x & 63, lg = lane >> 4, col = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int group = wave / a.down_parts, per = kWaves / a.down_parts;
  const int e = by_pair ? __builtin_amdgcn_readfirstlane(a.pair_expert[blockIdx.y]) : (int)blockIdx.y;
  if (by_pair && a.tokens == 1)
    only_user(blockIdx.y, u);
  else
    read_users(a, e, u);
  if (u.count == 0 || (by_pair && u.pair[0] != (int)blockIdx.y)) return;
  St st;
  st.setup(0, a.down, e, a.hidden, a.inter);
  st.setup(1, a.down, e, a.hidden, a.inter);
  const auto first_row = [&](int unit) { return (unit * per + group) * 32; };
  const auto set_tiles = [&](St& t, int unit) {
    t.tile(0, first_row(unit));
    t.tile(1, first_row(unit) + 16);
  };
  const int slots = (a.inter + St::S::kSpan - 1) / St::S::kSpan, share = stretch_of(slots, a.splits);
  const int z = blockIdx.z;
  for (int r0 = 0; r0 < u.count; r0 += 16) {
    const int rows = min(16, u.count - r0);
    int xrl;
    const int chunk = fit_chunk<2, St>(rows, a.down_parts, &xrl);
    const Walk w{(int)blockIdx.x, (int)gridDim.x, (int)((a.hidden + 32 * per - 1) / (32 * per)), a.down_parts,
                 wave - group * a.down_parts, min(slots, z * share), min(slots, (z + 1) * share), chunk};
    const auto row = [&](int m) { return a.h + (int64_t)u.pair[r0 + m] * 2 * a.inter; };
    const auto finish = [&](int unit, const f32x4 (&acc)[2]) {
      const int n = first_row(unit) + col;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = r0 + 4 * lg + i;
        if (r >= u.count) continue;
        float* o = a.out + ((int64_t)u.pair[r] * a.splits + z) * a.hidden + n;
        if (n < a.hidden) o[0] = acc[0][i];
        if (n + 16 < a.hidden) o[16] = acc[1][i];
      }
    };
    Products<2, St, decltype(row), decltype(set_tiles), decltype(finish)> p{st, w};
    p.run(rows, row, a.inter, set_tiles, finish, xrl, xs, hand);
  }
}

template <class T, int BITS, int GS>
hipError_t launch_group(const MoeArgs& a, hipStream_t stream, bool down) {
  const int pairs = a.tokens * a.top_k, by_pair = pairs < a.experts;
  const dim3 grid((unsigned)(down ? a.down_blocks : a.blocks), (unsigned)(by_pair ? pairs : a.experts),
                  (unsigned)(down ? a.splits : 1));
  if (down) {
    if (sb_wide<GS>(a.down, a.inter))
      hipLaunchKernelGGL((down_kernel<T, BITS, GS, false>), grid, dim3(kThreads), 0, stream, a, by_pair);
    else
      hipLaunchKernelGGL((down_kernel<T, BITS, GS, true>), grid, dim3(kThreads), 0, stream, a, by_pair);
  } else {
    if (sb_wide<GS>(a.gate, a.hidden) && sb_wide<GS>(a.up, a.hidden))
      hipLaunchKernelGGL((gate_up_kernel<T, BITS, GS, false>), grid, dim3(kThreads), 0, stream, a, by_pair);
    else
      hipLaunchKernelGGL((gate_up_kernel<T, BITS, GS, true>), grid, dim3(kThreads), 0, stream, a, by_pair);
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
