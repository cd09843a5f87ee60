// Attention over the 4-bit key/value cache, for one element type (included by kv_attend_bf16.hip
// and kv_attend_fp16.hip, and by kv_attend_tree_bf16.hip and kv_attend_tree_fp16.hip for trees of
// drafted tokens).
//
// With k_j = s_jg c_jd + b_jg (codes c, groups g of the head dimension) the score of query q is
//     q . k_j = sum_g ( s_jg * sum_{d in g} q_d c_jd  +  b_jg * sum_{d in g} q_d ),
// and the output, with p_j = exp2(score_j - m) for a running maximum m and V's own s, b, c,
//     o_d = ( sum_j (p_j s_jg) c_jd  +  sum_j p_j b_jg ) / sum_j p_j        (g the group of d).
// Both sums over codes run on the matrix cores with the codes as exact integers; scales and
// biases enter in float32.  Nothing is dequantized to memory, and each code is unpacked once
// for all the query rows of a wave.
//
// The score product takes tokens as its rows (K codes are the first operand) and query rows
// as its columns, so a lane's accumulator holds four consecutive tokens of one query row --
// the layout that the second product needs for its right operand, whose contraction index is
// the token: probabilities never move between lanes.  A step is 32 tokens (two 16-token
// tiles): contraction slot (h, e) of the second product is token 4h + e of the first tile for
// e < 4, 4h + e - 4 of the second one otherwise.
//
// Softmax: m, the sum of p, the bias sums and both accumulators are float32.  m is raised only
// when a score exceeds it by more than kSlack (in powers of two), so most steps rescale
// nothing; p is then at most 2^kSlack.  p_j s_jg goes to the matrix cores as two bfloat16
// operands, its leading bits and the rest (split2), so that the product carries 16 bits of it:
// with one operand, a row that attends to one token would return that token's codes with an
// error of up to 2^-8 of their span.  They are bfloat16 in fp16 calls too (the codes are exact in
// either type): fp16 has nothing below 2^-24, where the small p of a row with most of its weight
// on one token lie, and their codes would vanish while their biases and their share of the sum
// stay.
#pragma once

#include <cfloat>
#include <type_traits>

#include "device_common.hpp"
#include "kv_cache.hpp"

namespace qmm {
namespace kv {

constexpr int kWaves = 4;
constexpr int kThreads = 64 * kWaves;
constexpr int kStep = 32;              // tokens per wave and step
constexpr float kNone = -FLT_MAX;      // running maximum before any token

constexpr float kSlack = 8.0f;         // largest exponent of an unnormalised probability

// Two float32 values as bfloat16 pairs hi + lo: hi their leading bits (truncated), lo the rest
// rounded to nearest: 2^-16 of the value at most is lost.
__device__ inline void split2(float x, float y, uint32_t* hi, uint32_t* lo) {
  const uint32_t a = __float_as_uint(x), b = __float_as_uint(y);
  *hi = __builtin_amdgcn_perm(b, a, 0x07060302u);
  *lo = Bf16::pack2(x - __uint_as_float(a & 0xFFFF0000u), y - __uint_as_float(b & 0xFFFF0000u));
}

template <int N>
__device__ inline void load_words(uint32_t (&r)[N], const uint32_t* p) {
  if constexpr (N == 2) {
    const uint2 u = *(const uint2*)p;
    r[0] = u.x;
    r[1] = u.y;
  } else {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const u32x4 u = *(const u32x4*)(p + 4 * i);
      r[4 * i] = u.x;
      r[4 * i + 1] = u.y;
      r[4 * i + 2] = u.z;
      r[4 * i + 3] = u.w;
    }
  }
}

// What a tree's query sees (TREE): of the tokens before the tree those from row_lo on, of the
// nodes, which are the sequence's last q_len tokens, those of its mask row.
struct TreeRow {
  const uint32_t* mask;
  int words;
  bool there;               // the row has a bit: else the query sees nothing

  __device__ inline void setup(const AttendArgs& a, int64_t b, int query) {
    words = a.mask_words;
    mask = a.mask + (b * a.q_len + query) * words;
    uint32_t any = 0u;
    for (int w = 0; w < words; ++w) any |= mask[w];
    there = any != 0u;
  }
  // Bits of the nodes node .. node + 31; those before the first node and past the words are zero.
  __device__ inline uint32_t bits(int node) const {
    const int w = node >> 5;
    const uint32_t lo = w >= 0 && w < words ? mask[w] : 0u, hi = w + 1 >= 0 && w + 1 < words ? mask[w + 1] : 0u;
    return (uint32_t)(((((uint64_t)hi) << 32) | lo) >> (node & 31));
  }
};
// The first token that a tree's query sees with a window, of the tokens before the tree, which ends at
// `off`.  Depths may be the caller's own: any from 0 on (below 2^30, as positions are), less counts as 0.
__device__ inline int tree_row_begin(const AttendArgs& a, int64_t b, int query, int off) {
  return off + min(max(a.depth[b * a.q_len + query], 0), 1 << 30) - a.window + 1;
}
// Largest v of the wave, the same in every lane; lanes 16 apart hold the same row.
__device__ inline int max_of_rows(int v) {
#pragma unroll
  for (int d = 1; d < 16; d <<= 1) v = max(v, __shfl_xor(v, d));
  return __builtin_amdgcn_readfirstlane(v);
}
// A sequence's length is in order: its tree fits in it, or it is empty.
template <bool TREE>
__device__ inline bool length_bad(const AttendArgs& a, int len) {
  return len < 0 || len > a.max_length || (TREE && len > 0 && len < a.q_len);
}

// The sequence of a tree call's workgroups with blockIdx.y = at: the at-th longest, so that what
// starts last is short (16 sequences of 512 to 8192 tokens, 128 query rows: 112 to 124 us; in the
// order of the batch, their lengths rising, 151).  At most 64 sequences, one per lane, are
// ordered: of more, each fills the chip for a smaller part of the call.
__device__ inline int by_length(const AttendArgs& a, int at) {
  if (a.batch > 64) return at;
  const int i = threadIdx.x & 63, n = (int)a.batch;
  const int mine = i < n ? a.lengths[i] : -1;
  int rank = 0;
  for (int j = 0; j < n; ++j) {
    const int other = __builtin_amdgcn_readlane(mine, j);
    rank += other > mine || (other == mine && j < i);
  }
  return __builtin_ctzll(__builtin_amdgcn_ballot_w64(i < n && rank == at));
}

// One side (K or V) of a 32-token step in registers: codes and (s, b) words of the lane's
// tokens, for the two 16-token tiles.
template <int D, int GS>
struct Side {
  uint32_t code[2][D / 32];
  uint32_t sb[2][D / GS][4];
};

// Four elements of one query row: its sums of this split, or the finished output.
template <class T, int D>
__device__ inline void store4(const AttendArgs& a, int64_t b, int head, int split, int64_t row0, int r, int d, f32x4 o,
                              float sum) {
  if (a.splits > 1) {
    *(f32x4*)(a.part + ((row0 + r) * a.splits + split) * D + d) = o;
  } else {
    const float inv = sum == 0.f ? 0.f : 1.0f / sum;    // a row that sees nothing is zero
    const int i = r / a.rep, g = r - i * a.rep;
    uint2 u;
    u.x = T::pack2(o[0] * inv, o[1] * inv);
    u.y = T::pack2(o[2] * inv, o[3] * inv);
    *(uint2*)((uint16_t*)a.out + ((b * a.q_len + i) * (int64_t)a.q_heads + head * a.rep + g) * D + d) = u;
  }
}

// ---- few query rows per cached head: single tokens, drafted tokens, short chunks.
//
// A workgroup takes 16 query rows of one cached head and one split of the tokens; its four waves
// take the split's 32-token steps in turn, each with its own softmax, and meet in LDS once at
// the end.  K and V of the next step are in flight while a step is computed, the pages of the
// step after it are looked up already.  Two tiles of 16 rows per wave would unpack each code
// once for 32 rows, but their registers leave one or two waves per SIMD: slower at every size
// measured (20 rows: 63 us against 42; 128 rows: 66 against 43; 8192 tokens, 8 heads of 128).
// Trees of many query rows take them all the same (R = 2), where the other choice is a workgroup
// of 256 rows: 64 nodes of 64 heads over 8 after 131071 tokens, 128 elements in one group, 524 us,
// 0.52 PFLOP/s of the definition's products (the other form 600 us, one tile 640); the vector units
// are busy 72% of the time there, the matrix cores 31%.
// Trees of fewer rows: 16 of 32 nodes after 480 to 8160 tokens, 32 heads over 8, 110 us, 413 vector
// instructions a step (two groups), also bound by these.
// What bounds it: a step is 384 vector instructions, about 1600 cycles, for 4.6 KB of codes and
// scales, so at 5 TB/s the vector units are as busy as the memory; with lengths that differ,
// what is left is the longest sequences' share.  Measured: 131071 tokens, 8 cached heads of
// 128 elements 35 us (4.1 TB/s); 32 sequences of 0 to 8192 tokens 53 us (2.9 TB/s).

// Workgroups per compute unit that the registers allow: the loads' latency decides, so as many
// as possible without spills.
template <int D, int GS>
constexpr int workgroups() { return D > 128 ? 1 : (D / GS == 1 ? 4 : (D / GS == 2 ? 3 : 2)); }

template <class T, int D, int GS, bool TREE, int R>
__global__ __launch_bounds__(kThreads, (R > 1 ? 2 : workgroups<D, GS>())) void attend_kernel(const AttendArgs a) {
  constexpr int KC = D / 32;          // 32-element steps of a score; code words per lane and tile
  constexpr int NT = D / 16;          // 16-element output tiles
  constexpr int NG = D / GS;
  constexpr int CPG = GS / 32;
  constexpr int kRows = 16 * R;       // query rows per workgroup
  constexpr int kPitch = D + 4;       // LDS row of the merge, padded against bank conflicts
  using P = Bf16;                     // operands of the second product

  const int lane = threadIdx.x & 63, col = lane & 15, h = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int split = blockIdx.z;
  const int head = blockIdx.x % a.c.heads, row_tile = blockIdx.x / a.c.heads;
  const int64_t b = TREE ? by_length(a, blockIdx.y) : blockIdx.y;
  const int base = row_tile * kRows;

  int len = a.lengths[b];
  const bool bad = length_bad<TREE>(a, len);
  if (bad) len = 0;
  // token ranges: [lo_min, hi_max) is seen by some row of the wave, [lo_max, hi_min) by all
  const int off = len - a.q_len;
  const int i_first = base / a.rep, i_last = (min(a.rows, base + kRows) - 1) / a.rep;
  // (a tree's rows have depths from 0 on, whatever their order; lo_max comes from them)
  const int hi_max = TREE ? len : (a.causal ? max(0, off + i_last + 1) : len);
  const int hi_min = TREE ? max(0, off) : (a.causal ? max(0, off + i_first + 1) : len);
  const int lo_min = a.window ? max(0, off + (TREE ? 0 : i_first) - a.window + 1) : 0;
  int lo_max = a.window && !TREE ? max(0, off + i_last - a.window + 1) : 0;
  const int c0 = (lo_min & ~(kStep - 1)) + split * a.chunk;
  const int c1 = min(c0 + a.chunk, hi_max);
  const int stride = kStep * kWaves;
  // scores stay unscaled until their exponential, so that one multiply-add scales and subtracts
  // m: the scale's sign goes to q, and zero becomes the least number (masked scores are -inf)
  const uint32_t flip = a.scale_log2 < 0.f ? 0x80008000u : 0u;
  const float magnitude = __builtin_fabsf(a.scale_log2), scale = magnitude < FLT_MIN ? FLT_MIN : magnitude;

  float m[R], l[R], bsum[R][NG] = {};
  f32x4 acc[R][NT];
#pragma unroll
  for (int k = 0; k < R; ++k) {
    m[k] = kNone;
    l[k] = 0.f;
#pragma unroll
    for (int i = 0; i < NT; ++i) acc[k][i] = f32x4{0.f, 0.f, 0.f, 0.f};
  }

  // The page of a 16-token tile that starts at token t0, and the token's place in it.  Tiles
  // that no row sees read page 0 (their tokens are masked), and so do needed ones that have no
  // page of the pool: rows that see those get NaN scores.
  const int32_t* table = a.table + b * a.table_stride;
  const int64_t page_words = 2 * a.c.side;
  struct Place {
    int page, token;
  };
  const auto place = [&](int t0) {
    Place p{0, 0};
    if (t0 < hi_max && t0 + 16 > lo_min) {
      const int blk = block_of_tile((uint32_t)t0 >> 4, a.page_recip);
      p.token = t0 - blk * a.c.page_size;
      p.page = __builtin_amdgcn_readfirstlane(table[blk]);
    }
    return p;
  };
  const auto outside = [&](const Place& p) { return p.page < 0 || p.page >= a.c.pages; };
  const auto base_of = [&](const Place& p) -> const uint32_t* {
    return a.c.data + ((int64_t)(outside(p) ? 0 : p.page) * a.c.heads + head) * page_words;
  };
  const uint32_t lane_k = (uint32_t)(col * (D / 8) + h * KC), lane_v = (uint32_t)((h * 16 + col) * KC), lane_sb = 4u * h;
  Side<D, GS> ks, vs;
  auto load_side = [&](Side<D, GS>& s, int tile, const uint32_t* p, int token, bool value) {
    if (value)
      load_words<KC>(s.code[tile], p + (int64_t)(token / 4) * (16 * KC) + lane_v);
    else
      load_words<KC>(s.code[tile], p + (int64_t)token * (D / 8) + lane_k);
    const uint32_t* sb = p + (int64_t)a.c.page_size * (D / 8) + token;
#pragma unroll
    for (int g = 0; g < NG; ++g) load_words<4>(s.sb[tile][g], sb + (int64_t)g * a.c.page_size + lane_sb);
  };
  // the next step's tiles, and the pages of the step after it
  const uint32_t* base_next[2] = {nullptr, nullptr};
  int token_next[2] = {0, 0};
  bool bad_next[2] = {false, false};
  Place place_next[2];
  auto find = [&](int t0) {
#pragma unroll
    for (int i = 0; i < 2; ++i) place_next[i] = place(t0 + 16 * i);
  };
  auto take = [&]() {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      base_next[i] = base_of(place_next[i]);
      bad_next[i] = outside(place_next[i]);
      token_next[i] = place_next[i].token;
    }
  };
  auto load_k = [&]() {
#pragma unroll
    for (int i = 0; i < 2; ++i) load_side(ks, i, base_next[i], token_next[i], false);
  };
  auto load_v = [&]() {
#pragma unroll
    for (int i = 0; i < 2; ++i) load_side(vs, i, base_next[i] + a.c.side, token_next[i], true);
  };

  const int first = c0 + kStep * wave;
  if (first < c1) {
    find(first);
    take();
    load_k();
    load_v();
    find(first + stride);
  }

  // query operands: column col is query row base + col (rows past the last repeat it and are not stored)
  typename T::v8 q[R][KC];
  float qsum[R][NG];
  const uint32_t one2 = T::pack2(1.0f, 1.0f);
  const u32x4 ones = {one2, one2, one2, one2};
  int row_lo[R], row_hi[R];
  TreeRow tree[R];
#pragma unroll
  for (int k = 0; k < R; ++k) {
    const int row = min(base + 16 * k + col, a.rows - 1);
    const int query = row / a.rep;
    const uint16_t* qp = (const uint16_t*)a.q + b * a.q_batch_stride + (int64_t)query * a.q_token_stride +
                         (int64_t)(head * a.rep + row - query * a.rep) * a.q_head_stride + 8 * h;
#pragma unroll
    for (int c = 0; c < KC; ++c) q[k][c] = as_v8<T>(interleave_even_odd(*(const u32x4*)(qp + 32 * c) ^ flip));
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      f32x4 d = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int c = 0; c < CPG; ++c) d = T::mfma(as_v8<T>(ones), q[k][g * CPG + c], d);
      qsum[k][g] = d[0];
    }
    row_hi[k] = TREE ? off : (a.causal ? off + query + 1 : len);
    row_lo[k] = a.window ? off + query - a.window + 1 : 0;
    if constexpr (TREE) {
      tree[k].setup(a, b, query);
      if (a.window) {
        row_lo[k] = tree_row_begin(a, b, query, off);
        lo_max = max(lo_max, max_of_rows(row_lo[k]));
      }
    }
  }

  for (int t0 = first; t0 < c1; t0 += stride) {
    const bool bad_now[2] = {bad_next[0], bad_next[1]};
    // ---- scores: sc[k][i][r] of token t0 + 16 i + 4 h + r
    float sc[R][2][4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        f32x4 d[R];
#pragma unroll
        for (int k = 0; k < R; ++k) d[k] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = g * CPG; c < (g + 1) * CPG; ++c) {
          const typename T::v8 codes = as_v8<T>(codes4_to_v8<T>(ks.code[i][c]));
#pragma unroll
          for (int k = 0; k < R; ++k) d[k] = T::mfma(codes, q[k][c], d[k]);
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float s = T::to_f32(ks.sb[i][g][r] & 0xFFFFu), kb = T::to_f32(ks.sb[i][g][r] >> 16);
#pragma unroll
          for (int k = 0; k < R; ++k)
            sc[k][i][r] = __builtin_fmaf(s, d[k][r], g == 0 ? kb * qsum[k][0] : __builtin_fmaf(kb, qsum[k][g], sc[k][i][r]));
        }
      }
    }
    take();                          // past the last step: words of page 0, not used
    load_k();
    find(t0 + 2 * stride);
    // ---- rows that do not see every token of the step, and tiles without a page of the pool
    const bool edge = t0 < lo_max || t0 + kStep > hi_min || bad_now[0] || bad_now[1];
    if (edge) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int k = 0; k < R; ++k) {
          const uint32_t nodes = TREE && t0 + kStep > off ? tree[k].bits(t0 + 16 * i + 4 * h - off) : 0u;
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int token = t0 + 16 * i + 4 * h + r;
            const bool seen =
                TREE && token >= off ? ((nodes >> r) & 1u) && token < len : token >= row_lo[k] && token < row_hi[k];
            sc[k][i][r] = seen ? (bad_now[i] ? __builtin_nanf("") : sc[k][i][r]) : -__builtin_inff();
            if constexpr (R == 1) {
#pragma unroll
              for (int g = 0; g < NG; ++g) vs.sb[i][g][r] = seen ? vs.sb[i][g][r] : 0u;   // whatever it holds, it adds nothing
            }
          }
        }
      }
    }
    // ---- probabilities
#pragma unroll
    for (int k = 0; k < R; ++k) {
      float(&x)[2][4] = sc[k];
      float top = fmaxf(fmaxf(x[0][0], x[0][1]), fmaxf(x[0][2], x[0][3]));
      top = fmaxf(top, fmaxf(fmaxf(x[1][0], x[1][1]), fmaxf(x[1][2], x[1][3]))) * scale;
      if (__builtin_amdgcn_ballot_w64(top > m[k] + kSlack) != 0ull) {
        top = fmaxf(top, __shfl_xor(top, 16));
        top = fmaxf(top, __shfl_xor(top, 32));
        const float raised = fmaxf(m[k], top);
        const float f = __builtin_amdgcn_exp2f(m[k] - raised);
        m[k] = raised;
        l[k] *= f;
#pragma unroll
        for (int g = 0; g < NG; ++g) bsum[k][g] *= f;
#pragma unroll
        for (int i = 0; i < NT; ++i) acc[k][i] *= f;
      }
#pragma unroll
      for (int n = 0; n < 8; ++n) {
        float& p = x[n >> 2][n & 3];
        p = __builtin_amdgcn_exp2f(__builtin_fmaf(p, scale, -m[k]));
        l[k] += p;
      }
    }
    // ---- second product, group by group
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      u32x4 hi[R], lo[R];
#pragma unroll
      for (int k = 0; k < R; ++k) {
        float x[8];
        const auto weighted = [&](auto guarded) {
#pragma unroll
          for (int n = 0; n < 8; ++n) {
            // (a token that only the wave's other rows see adds nothing, whatever it holds)
            const float p = sc[k][n >> 2][n & 3];
            const uint32_t sb = decltype(guarded)::value && p == 0.f ? 0u : vs.sb[n >> 2][g][n & 3];
            x[n] = p * T::to_f32(sb & 0xFFFFu);
            bsum[k][g] = __builtin_fmaf(p, T::to_f32(sb >> 16), bsum[k][g]);
          }
        };
        if (R > 1 && edge)
          weighted(std::true_type{});
        else
          weighted(std::false_type{});
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          uint32_t uh, ul;
          split2(x[2 * n], x[2 * n + 1], &uh, &ul);
          hi[k][n] = uh;
          lo[k][n] = ul;
        }
      }
#pragma unroll
      for (int j = g * CPG; j < (g + 1) * CPG; ++j) {
        const uint32_t w0 = vs.code[0][j], w1 = vs.code[1][j];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          const uint32_t e0 = (n ? w0 >> 4 : w0) & 0x0F0F0F0Fu, e1 = (n ? w1 >> 4 : w1) & 0x0F0F0F0Fu;
          const u32x4 vc = {P::fp8x2_lo(e0), P::fp8x2_hi(e0), P::fp8x2_lo(e1), P::fp8x2_hi(e1)};
#pragma unroll
          for (int k = 0; k < R; ++k) {
            acc[k][2 * j + n] = P::mfma(as_v8<P>(vc), as_v8<P>(lo[k]), acc[k][2 * j + n]);
            acc[k][2 * j + n] = P::mfma(as_v8<P>(vc), as_v8<P>(hi[k]), acc[k][2 * j + n]);
          }
        }
      }
    }
    load_v();
  }

  // ---- the lanes' shares of the sums, and the bias term: element d = 16 i + 4 h + r of row col
#pragma unroll
  for (int k = 0; k < R; ++k) {
    l[k] += __shfl_xor(l[k], 16);
    l[k] += __shfl_xor(l[k], 32);
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      bsum[k][g] += __shfl_xor(bsum[k][g], 16);
      bsum[k][g] += __shfl_xor(bsum[k][g], 32);
    }
#pragma unroll
    for (int i = 0; i < NT; ++i) acc[k][i] += bsum[k][i * 16 / GS];
    if (TREE && !tree[k].there) {    // its scores were of tokens that it does not see
      l[k] = 0.f;
      m[k] = kNone;
#pragma unroll
      for (int i = 0; i < NT; ++i) acc[k][i] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
    if (bad) {
      l[k] = __builtin_nanf("");
      m[k] = 0.f;
    }
  }

  // ---- the four waves' sums meet in LDS
  __shared__ float o_s[kWaves][kRows][kPitch];
  __shared__ float2 ml_s[kWaves][kRows];
#pragma unroll
  for (int k = 0; k < R; ++k) {
#pragma unroll
    for (int i = 0; i < NT; ++i) *(f32x4*)&o_s[wave][16 * k + col][16 * i + 4 * h] = acc[k][i];
    if (h == 0) ml_s[wave][16 * k + col] = float2{m[k], l[k]};
  }
  __syncthreads();
  const int64_t row0 = (b * a.c.heads + head) * a.rows;
  float* part_ml = a.part + a.batch * a.c.heads * a.rows * a.splits * D;
  for (int e = threadIdx.x; e < kRows * (D / 4); e += kThreads) {
    const int rr = e / (D / 4), d = (e - rr * (D / 4)) * 4;
    const int r = base + rr;
    if (r >= a.rows) break;
    float top = kNone;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) top = fmaxf(top, ml_s[w][rr].x);
    float sum = 0.f;
    f32x4 o = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      const float f = __builtin_amdgcn_exp2f(ml_s[w][rr].x - top);
      sum = __builtin_fmaf(f, ml_s[w][rr].y, sum);
      o += f * *(const f32x4*)&o_s[w][rr][d];
    }
    store4<T, D>(a, b, head, split, row0, r, d, o, sum);
    if (a.splits > 1 && d == 0) {
      float* ml = part_ml + ((row0 + r) * a.splits + split) * 2;
      ml[0] = top;
      ml[1] = sum;
    }
  }
}

// ---- prompts: many query rows per cached head.
//
// Here the work per score decides, not the memory: the workgroup's waves take 16 query rows
// each and share what a step's 32 tokens cost to unpack, in LDS, in operand order
// (double-buffered, one barrier per step; the next step's words are in registers meanwhile):
//   K  its codes as exact integers, and its scales and biases as float32: a score costs one
//      matrix-core pass and two multiply-adds per group;
//   V  the values s c + b themselves, as two bfloat16 operands (leading bits, rest), so that the
//      probabilities need no scale per token and group: they are split once, and
//      p v = p_hi v_lo + p_lo v_hi + p_hi v_hi, to 2^-14 of each |p v| (2^-15 in fp16 calls,
//      where V is rounded instead of cut off).
// (Codes and scales for V, as in the single-token form, cost 11 vector operations per score
// more, two of them per group, against a third matrix-core pass here: 1223 us against 800 in
// the case below.)
// What bounds it: LDS.  A wave reads 32 16-byte operands a lane for 32 products, and the
// sixteen waves' reads take 4100 of a step's 5400 cycles, the matrix cores 2050 and the vector
// units about 3000, with four waves per SIMD to overlap them.  Two 16-row tiles per wave halve
// the reads, but then two waves per SIMD wait for each other (650 us; 680 with the products of
// half of the waves a step late); two workgroups of eight waves unpack everything twice (656).
// Measured: 2048 queries after 6144 tokens, 32 query heads over 8 of 128 elements, 550 us, 0.44
// PFLOP/s of the two products of the definition (0.87 with the passes for V's two operands).
// Tokens outside every row's range are zero in LDS, and so are values that are not finite,
// which a token that only some rows see may hold: the unpacking notes the token, and a row
// that gives it weight becomes NaN.
// Scores leave the multiply-adds relative to the running maximum: -m is where they start.

// split2 with hi rounded to nearest, for values below half the type's largest: 2^-17 is lost.
__device__ inline void split2_near(float x, float y, uint32_t* hi, uint32_t* lo) {
  *hi = Bf16::pack2(x, y);
  *lo = Bf16::pack2(x - Bf16::to_f32(*hi & 0xFFFFu), y - Bf16::to_f32(*hi >> 16));
}

// Waves per workgroup: 16 where 128 registers hold a wave, of which the first eight unpack.
constexpr int row_waves(int head_dim) { return head_dim == 256 ? 8 : 16; }
constexpr int kUnpackers = 8;

template <class T, int D, int GS, bool TREE>
__global__ __launch_bounds__(64 * row_waves(D), 1) void attend_rows_kernel(const AttendArgs a) {
  constexpr int W = row_waves(D);
  constexpr int KC = D / 32, NT = D / 16, NG = D / GS, CPG = GS / 32;
  constexpr int kRows = 16;
  using P = Bf16;                 // operands of the second product
  constexpr int kKUnits = (2 * KC + kUnpackers - 1) / kUnpackers, kVUnits = (NT + kUnpackers - 1) / kUnpackers;
  static_assert(NG * kStep <= 64 * kUnpackers, "one thread per scale word of a step");
  struct Buffer {
    u32x4 k[2 * KC][64];          // [tile, 32-element step][lane]
    u32x4 v[2][NT][64];           // [leading bits, rest][16-element tile][lane]
    float s[NG][kStep], b[NG][kStep];   // times the score's scale
  };
  __shared__ Buffer bufs[2];
  __shared__ uint32_t odd_tokens[4];    // by step % 4: tokens of the step with values that are not finite

  const int lane = threadIdx.x & 63, col = lane & 15, h = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int split = blockIdx.z;
  const int head = blockIdx.x % a.c.heads, row_tile = blockIdx.x / a.c.heads;
  const int64_t b = blockIdx.y;
  const int wg_base = row_tile * W * kRows, base = wg_base + wave * kRows;

  int len = a.lengths[b];
  const bool bad = length_bad<TREE>(a, len);
  if (bad) len = 0;
  const int off = len - a.q_len;
  // (a tree's rows have depths from 0 on, whatever their order; lo_max comes from them)
  const auto row_end = [&](int r) { return TREE || !a.causal ? len : max(0, off + r / a.rep + 1); };
  const auto row_begin = [&](int r) { return a.window ? max(0, off + (TREE ? 0 : r / a.rep) - a.window + 1) : 0; };
  // ranges of the workgroup, and of this wave (empty for a wave without rows)
  const int wg_last = min(a.rows, wg_base + W * kRows) - 1;
  const int wg_lo = row_begin(wg_base), wg_hi = row_end(wg_last);
  const bool live = base < a.rows;
  const int last = min(a.rows, base + kRows) - 1;
  const int lo_min = live ? row_begin(base) : 0, hi_max = live ? row_end(last) : 0;
  int lo_max = live && !TREE ? row_begin(last) : 0;
  const int hi_min = !live ? 0 : (!TREE ? row_end(base) : max(0, off));
  const int c0 = (wg_lo & ~(kStep - 1)) + split * a.chunk;
  const int c1 = min(c0 + a.chunk, wg_hi);

  // ---- a step's words, from global memory
  const int32_t* table = a.table + b * a.table_stride;
  const int64_t page_words = 2 * a.c.side;
  const uint32_t* tile_at[2];      // K words of the tile's page; its token
  int tile_token[2];
  bool tile_bad[2], loaded_bad[2] = {false, false};
  int page_next[2] = {0, 0}, token_next[2] = {0, 0};
  const auto find = [&](int t0) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int t = t0 + 16 * i;
      page_next[i] = 0;
      token_next[i] = 0;
      if (t < wg_hi && t + 16 > wg_lo) {
        const int blk = block_of_tile((uint32_t)t >> 4, a.page_recip);
        token_next[i] = t - blk * a.c.page_size;
        page_next[i] = __builtin_amdgcn_readfirstlane(table[blk]);
      }
    }
  };
  uint32_t kw[kKUnits], vw[kVUnits][2], ksb = 0;
  u32x4 vsb[kVUnits][2];
  const int sb_token = threadIdx.x & (kStep - 1), sb_group = threadIdx.x / kStep;
  const auto load = [&]() {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      tile_bad[i] = page_next[i] < 0 || page_next[i] >= a.c.pages;
      tile_at[i] = a.c.data + ((int64_t)(tile_bad[i] ? 0 : page_next[i]) * a.c.heads + head) * page_words;
      tile_token[i] = token_next[i];
      loaded_bad[i] = tile_bad[i];
    }
#pragma unroll
    for (int n = 0; n < kKUnits; ++n) {
      const int u = wave + n * kUnpackers, i = u / KC, c = u - i * KC;
      if (u < 2 * KC) kw[n] = tile_at[i][(tile_token[i] + col) * (D / 8) + h * KC + c];
    }
    if (sb_group < NG) {
      const int i = sb_token >> 4;
      ksb = (i ? tile_at[1] : tile_at[0])[(int64_t)a.c.page_size * (D / 8) + sb_group * a.c.page_size +
                                         (i ? tile_token[1] : tile_token[0]) + (sb_token & 15)];
    }
#pragma unroll
    for (int n = 0; n < kVUnits; ++n) {
      const int u = wave + n * kUnpackers;
      if (u < NT) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t* p = tile_at[i] + a.c.side;
          vw[n][i] = p[((tile_token[i] / 4 + h) * 16 + col) * KC + u / 2];
          vsb[n][i] = *(const u32x4*)(p + (int64_t)a.c.page_size * (D / 8) + (u * 16 / GS) * a.c.page_size +
                                      tile_token[i] + 4 * h);
        }
      }
    }
  };
  // ---- unpack them into a buffer, for the step at t0
  const auto unpack = [&](Buffer& buf, int t0) {
#pragma unroll
    for (int n = 0; n < kKUnits; ++n) {
      const int u = wave + n * kUnpackers;
      if (u < 2 * KC) buf.k[u][lane] = codes4_to_v8<T>(kw[n]);
    }
    if (sb_group < NG) {
      // a needed tile without a page of the pool makes the scores of those who see it NaN
      const bool nan = (sb_token >> 4) ? loaded_bad[1] : loaded_bad[0];
      buf.s[sb_group][sb_token] = nan ? __builtin_nanf("") : T::to_f32(ksb & 0xFFFFu) * a.scale_log2;
      buf.b[sb_group][sb_token] = T::to_f32(ksb >> 16) * a.scale_log2;
    }
    const bool edge = t0 < wg_lo || t0 + kStep > wg_hi || loaded_bad[0] || loaded_bad[1];
#pragma unroll
    for (int n = 0; n < kVUnits; ++n) {
      const int u = wave + n * kUnpackers;
      if (u >= NT) continue;
      u32x4 hi, lo;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t e = (u & 1 ? vw[n][i] >> 4 : vw[n][i]) & 0x0F0F0F0Fu;
        float v[4], zero = 0.f;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          v[r] = __builtin_fmaf(T::to_f32(vsb[n][i][r] & 0xFFFFu), (float)((e >> (8 * r)) & 0xFFu),
                                T::to_f32(vsb[n][i][r] >> 16));
          if (edge) {
            const int token = t0 + 16 * i + 4 * h + r;
            if (token < wg_lo || token >= wg_hi || loaded_bad[i]) v[r] = 0.f;
          }
          zero = __builtin_fmaf(v[r], 0.f, zero);      // NaN for an infinity or a NaN
        }
        if (__builtin_amdgcn_ballot_w64(zero != 0.f) != 0ull) {
#pragma unroll
          for (int r = 0; r < 4; ++r)
            if (!(__builtin_fabsf(v[r]) <= FLT_MAX)) {
              v[r] = 0.f;
              atomicOr(&odd_tokens[(t0 / kStep) & 3], 1u << (16 * i + 4 * h + r));
            }
        }
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          uint32_t uh, ul;
          if constexpr (T::kDtype == QMM_BF16)
            split2(v[2 * r], v[2 * r + 1], &uh, &ul);        // any bfloat16: none rounds up to infinity
          else
            split2_near(v[2 * r], v[2 * r + 1], &uh, &ul);
          hi[2 * i + r] = uh;
          lo[2 * i + r] = ul;
        }
      }
      buf.v[0][u][lane] = hi;
      buf.v[1][u][lane] = lo;
    }
  };
  if (threadIdx.x < 4) odd_tokens[threadIdx.x] = 0u;
  if (wave < kUnpackers && c0 < c1) {
    find(c0);
    load();
    if (c0 + kStep < c1) find(c0 + kStep);
  }

  typename T::v8 q[KC];
  float qsum[NG], m = 0.f, l = 0.f;
  float over = -__builtin_inff();    // scores above m + over raise m: any score at first, then kSlack
  f32x4 acc[NT];
  const uint32_t one2 = T::pack2(1.0f, 1.0f);
  const u32x4 ones = {one2, one2, one2, one2};
  const int r = min(base + col, a.rows - 1), query = r / a.rep;
  const uint16_t* qp = (const uint16_t*)a.q + b * a.q_batch_stride + (int64_t)query * a.q_token_stride +
                       (int64_t)(head * a.rep + r - query * a.rep) * a.q_head_stride + 8 * h;
#pragma unroll
  for (int c = 0; c < KC; ++c) q[c] = as_v8<T>(interleave_even_odd(*(const u32x4*)(qp + 32 * c)));
#pragma unroll
  for (int g = 0; g < NG; ++g) {
    f32x4 d = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int c = 0; c < CPG; ++c) d = T::mfma(as_v8<T>(ones), q[g * CPG + c], d);
    qsum[g] = d[0];
  }
  const int row_hi = TREE ? off : (a.causal ? off + query + 1 : len);
  int row_lo = a.window ? off + query - a.window + 1 : 0;
  TreeRow tree;
  if constexpr (TREE) {
    tree.setup(a, b, query);
    if (a.window) {
      row_lo = tree_row_begin(a, b, query, off);
      lo_max = max_of_rows(row_lo);
    }
  }
#pragma unroll
  for (int j = 0; j < NT; ++j) acc[j] = f32x4{0.f, 0.f, 0.f, 0.f};
  __syncthreads();                   // the flags are clear
  if (wave < kUnpackers && c0 < c1) {
    unpack(bufs[0], c0);
    if (c0 + kStep < c1) {
      load();
      if (c0 + 2 * kStep < c1) find(c0 + 2 * kStep);
    }
  }
  lds_barrier();

  const auto prepare = [&](int t0, Buffer& to) {
    if (t0 + kStep >= c1) return;
    unpack(to, t0 + kStep);
    if (t0 + 2 * kStep < c1) {
      load();
      if (t0 + 3 * kStep < c1) find(t0 + 3 * kStep);
    }
  };
  // ---- scores and probabilities of a step, as operands
  u32x4 ph, pl;
  const auto weigh = [&](const Buffer& buf, int t0) {
    float sc[2][4];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        const f32x4 s = *(const f32x4*)&buf.s[g][16 * i + 4 * h], bb = *(const f32x4*)&buf.b[g][16 * i + 4 * h];
        f32x4 d = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = g * CPG; c < (g + 1) * CPG; ++c) d = T::mfma(as_v8<T>(buf.k[i * KC + c][lane]), q[c], d);
#pragma unroll
        for (int n = 0; n < 4; ++n)
          sc[i][n] = __builtin_fmaf(s[n], d[n], __builtin_fmaf(bb[n], qsum[g], g == 0 ? -m : sc[i][n]));
      }
    if (t0 < lo_max || t0 + kStep > hi_min) {     // rows that do not see every token of the step
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t nodes = TREE && t0 + kStep > off ? tree.bits(t0 + 16 * i + 4 * h - off) : 0u;
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          const int token = t0 + 16 * i + 4 * h + n;
          const bool seen = TREE && token >= off ? ((nodes >> n) & 1u) && token < len : token >= row_lo && token < row_hi;
          sc[i][n] = seen ? sc[i][n] : -__builtin_inff();
        }
      }
    }
    float top = fmaxf(fmaxf(sc[0][0], sc[0][1]), fmaxf(sc[0][2], sc[0][3]));
    top = fmaxf(top, fmaxf(fmaxf(sc[1][0], sc[1][1]), fmaxf(sc[1][2], sc[1][3])));
    if (__builtin_amdgcn_ballot_w64(top > over) != 0ull) {
      top = fmaxf(top, __shfl_xor(top, 16));
      top = fmaxf(top, __shfl_xor(top, 32));
      const bool some = top > -__builtin_inff();             // false: nothing seen yet, m stays
      const bool empty = over < 0.f;                         // no score yet: m may go down too
      const float up = empty ? (some ? top : 0.f) : fmaxf(top, 0.f);
      over = empty && !some ? over : kSlack;
      const float f = empty ? 1.0f : __builtin_amdgcn_exp2f(-up);   // (of zero sums: 2^-up can be infinite)
      m += up;
      l *= f;
#pragma unroll
      for (int i = 0; i < NT; ++i) acc[i] *= f;
#pragma unroll
      for (int n = 0; n < 8; ++n) sc[n >> 2][n & 3] -= up;
    }
#pragma unroll
    for (int n = 0; n < 8; ++n) {
      sc[n >> 2][n & 3] = __builtin_amdgcn_exp2f(sc[n >> 2][n & 3]);
      l += sc[n >> 2][n & 3];
    }
    const uint32_t odd = __builtin_amdgcn_readfirstlane(odd_tokens[(t0 / kStep) & 3]);
    if (odd) {
#pragma unroll
      for (int n = 0; n < 8; ++n)
        if (((odd >> (16 * (n >> 2) + 4 * h + (n & 3))) & 1u) && sc[n >> 2][n & 3] != 0.f) l = __builtin_nanf("");
    }
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      uint32_t uh, ul;
      split2_near(sc[n >> 1][2 * (n & 1)], sc[n >> 1][2 * (n & 1) + 1], &uh, &ul);
      ph[n] = uh;
      pl[n] = ul;
    }
  };
  const auto add = [&](const Buffer& buf) {
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const typename P::v8 vh = as_v8<P>(buf.v[0][i][lane]), vl = as_v8<P>(buf.v[1][i][lane]);
      acc[i] = P::mfma(vl, as_v8<P>(ph), acc[i]);
      acc[i] = P::mfma(vh, as_v8<P>(pl), acc[i]);
      acc[i] = P::mfma(vh, as_v8<P>(ph), acc[i]);
    }
  };
  // ---- the steps
  int at = 0;
  for (int t0 = c0; t0 < c1; t0 += kStep, at ^= 1) {
    if (threadIdx.x == 0) odd_tokens[(t0 / kStep + 2) & 3] = 0u;   // last read two steps ago, next set in the next one
    // of eight waves, half unpack after their products: the two of a SIMD need the matrix core in turn
    const bool first = W > kUnpackers || wave < W / 2;
    if (wave < kUnpackers && first) prepare(t0, bufs[at ^ 1]);
    if (t0 < hi_max && t0 + kStep > lo_min) {
      weigh(bufs[at], t0);
      add(bufs[at]);
    }
    if (!first) prepare(t0, bufs[at ^ 1]);
    lds_barrier();
  }

  if (!live) return;
  const int64_t row0 = (b * a.c.heads + head) * a.rows;
  float* part_ml = a.part + a.batch * a.c.heads * a.rows * a.splits * D;
  l += __shfl_xor(l, 16);
  l += __shfl_xor(l, 32);
  if (TREE && !tree.there) {         // its scores were of tokens that it does not see
    l = 0.f;
    m = kNone;
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[j] = f32x4{0.f, 0.f, 0.f, 0.f};
  }
  if (bad) {
    l = __builtin_nanf("");
    m = 0.f;
  }
  if (base + col >= a.rows) return;
#pragma unroll
  for (int i = 0; i < NT; ++i) store4<T, D>(a, b, head, split, row0, r, 16 * i + 4 * h, acc[i], l);
  if (a.splits > 1 && h == 0) {
    float* ml = part_ml + ((row0 + r) * a.splits + split) * 2;
    ml[0] = over < 0.f && !bad ? kNone : m;             // kNone: no token of the split was seen
    ml[1] = l;
  }
}

// Joins the splits of one query row: o = sum_s 2^(m_s - M) o_s / sum_s 2^(m_s - M) l_s.
// D/4 lanes hold the row's elements, the other lanes of the workgroup further splits.
template <class T, int D, bool TREE>
__global__ __launch_bounds__(kThreads) void attend_join_kernel(const AttendArgs a) {
  constexpr int kLanes = D / 4, kGroups = kThreads / kLanes;
  __shared__ float top_s[kWaves];
  __shared__ float sum_s[kGroups];
  __shared__ f32x4 o_s[kGroups][kLanes];
  const int64_t row = blockIdx.x;                        // ((batch, head), query row)
  const int lane = threadIdx.x % kLanes, grp = threadIdx.x / kLanes;
  const float* o_part = a.part + row * a.splits * D;
  const float* ml = a.part + a.batch * a.c.heads * a.rows * a.splits * D + row * a.splits * 2;
  float top = kNone;
  for (int s = threadIdx.x; s < a.splits; s += kThreads) top = fmaxf(top, ml[2 * s]);
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) top = fmaxf(top, __shfl_xor(top, d));
  if ((threadIdx.x & 63) == 0) top_s[threadIdx.x >> 6] = top;
  __syncthreads();
  top = fmaxf(fmaxf(top_s[0], top_s[1]), fmaxf(top_s[2], top_s[3]));
  float sum = 0.f;
  f32x4 o = {0.f, 0.f, 0.f, 0.f};
  constexpr int kAhead = 8;                              // splits loaded before the first is used
  for (int s0 = grp; s0 < a.splits; s0 += kAhead * kGroups) {
    float m[kAhead], l[kAhead];
    f32x4 v[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int s = min(s0 + i * kGroups, a.splits - 1);
      m[i] = ml[2 * s];
      l[i] = ml[2 * s + 1];
      v[i] = *(const f32x4*)(o_part + (int64_t)s * D + 4 * lane);
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (s0 + i * kGroups >= a.splits || l[i] == 0.f) continue;   // no token of the split was seen
      const float f = __builtin_amdgcn_exp2f(m[i] - top);
      sum = __builtin_fmaf(f, l[i], sum);
      o += f * v[i];
    }
  }
  o_s[grp][lane] = o;
  if (lane == 0) sum_s[grp] = sum;
  __syncthreads();
  if (grp != 0) return;
  for (int g = 1; g < kGroups; ++g) {
    o += o_s[g][lane];
    sum += sum_s[g];
  }
  const float inv = sum == 0.f ? 0.f : 1.0f / sum;
  const int64_t bh = row / a.rows;
  const int r = (int)(row - bh * a.rows);
  const int64_t b = bh / a.c.heads;
  const int head = (int)(bh - b * a.c.heads), i = r / a.rep, g = r - i * a.rep;
  uint2 u;
  u.x = T::pack2(o[0] * inv, o[1] * inv);
  u.y = T::pack2(o[2] * inv, o[3] * inv);
  *(uint2*)((uint16_t*)a.out + ((b * a.q_len + i) * (int64_t)a.q_heads + head * a.rep + g) * D + 4 * lane) = u;
}

template <class T, int D, int GS, bool TREE>
hipError_t launch_shape(const AttendArgs& a, const AttendPlan& p, hipStream_t stream) {
  // Workgroups go to the eight XCDs in turn, x fastest.  Of sequences of unequal length only the
  // longest have work in the last splits, so splits are the slowest index: with splits fastest
  // (4 of them), two XCDs had every first split.
  const dim3 grid((unsigned)(a.c.heads * p.row_tiles), (unsigned)a.batch, (unsigned)p.splits);
  if (p.form == kRowsForm)
    hipLaunchKernelGGL((attend_rows_kernel<T, D, GS, TREE>), grid, dim3(64 * row_waves(D)), 0, stream, a);
  else if (p.form == kPairsForm) {
    if constexpr (TREE && has_pairs(D, GS))
      hipLaunchKernelGGL((attend_kernel<T, D, GS, TREE, 2>), grid, dim3(kThreads), 0, stream, a);
  } else
    hipLaunchKernelGGL((attend_kernel<T, D, GS, TREE, 1>), grid, dim3(kThreads), 0, stream, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.splits == 1) return e;
  hipLaunchKernelGGL((attend_join_kernel<T, D, TREE>), dim3((unsigned)(a.batch * a.c.heads * a.rows)), dim3(kThreads), 0,
                     stream, a);
  return hipGetLastError();
}

template <class T, bool TREE>
hipError_t launch_attend(const AttendArgs& a, const AttendPlan& p, hipStream_t stream) {
  const int gs = a.c.group_size;
  switch (a.c.head_dim) {
    case 64: return gs == 32 ? launch_shape<T, 64, 32, TREE>(a, p, stream) : launch_shape<T, 64, 64, TREE>(a, p, stream);
    case 128:
      return gs == 32   ? launch_shape<T, 128, 32, TREE>(a, p, stream)
             : gs == 64 ? launch_shape<T, 128, 64, TREE>(a, p, stream)
                        : launch_shape<T, 128, 128, TREE>(a, p, stream);
    case 256:
      return gs == 32   ? launch_shape<T, 256, 32, TREE>(a, p, stream)
             : gs == 64 ? launch_shape<T, 256, 64, TREE>(a, p, stream)
                        : launch_shape<T, 256, 128, TREE>(a, p, stream);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace kv
}  // namespace qmm
