// Matrix products grouped by expert, y[r] = x[r] W_e^T for the rows r of expert e, with weights
// w = s q + b per group (included by grouped_b4.hip, grouped_b8.hip and grouped_bn.hip).
//
// Arithmetic as in the decode kernels: the codes are exact operands of the matrix cores, and
//     y[r][n] = sum_g ( s_ng * sum_{k in g} x_rk q_nk  +  b_ng * X_rg ),   X_rg = sum_{k in g} x_rk,
// so a weight is never rounded.  A group's code product is scaled with one multiply-add per output.
// The second term is a product over groups: X comes from a kernel before this one, as three
// bfloat16 parts (24 bits), and b (two parts of an fp16) is its other operand; it costs 3 (5) matrix
// instructions for 32 groups where multiply-adds would cost as many vector instructions as the
// scales do.
//
// A workgroup takes 16 FM rows of one expert (a Tile) and 256 weight rows, each of its four waves
// 64 of them, so a code is unpacked once per tile.  Weights go from memory to the registers of the
// wave that needs them, a step of 128 columns ahead.  Activations are shared: direct loads put
// them into LDS in operand order (a load moves the 16 rows x 32 columns that one matrix
// instruction takes), double-buffered, a step ahead too, with one barrier per step.  A wave reads
// each operand once per step for the products with its four tiles: half of the LDS' rate when the
// matrix cores are busy all the time.
#pragma once

#include <type_traits>

#include "decode_impl.hpp"
#include "grouped.hpp"

namespace qmm {
namespace grouped {

constexpr int TN = 4;                          // weight tiles per wave
constexpr int kMfmaSteps = kStepK / 32;
constexpr uint32_t kPast = 0x7FFFFF00u;        // an offset past every descriptor: reads zero

typedef __attribute__((address_space(3))) void lds_void_t;

// 16 bytes per lane, at byte offset `off`, to the wave's 1 KB of LDS at `to`.
__device__ inline void load_to_lds(__amdgpu_buffer_rsrc_t rs, u32x4* to, uint32_t off) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_void_t*)to, 16, off, 0, 0, 0);
}

// Eight 4-bit codes in natural order.
template <class X>
__device__ inline u32x4 codes4_natural(uint32_t w) {
  const uint32_t even = w & 0x0F0F0F0Fu, odd = (w >> 4) & 0x0F0F0F0Fu;
  const uint32_t lo = __builtin_amdgcn_perm(odd, even, 0x05010400u), hi = __builtin_amdgcn_perm(odd, even, 0x07030602u);
  return u32x4{X::fp8x2_lo(lo), X::fp8x2_hi(lo), X::fp8x2_lo(hi), X::fp8x2_hi(hi)};
}

// x as leading bits and rest, both bfloat16.
__device__ inline void split_pair(float x, float y, uint32_t* hi, uint32_t* lo) {
  const uint32_t a = __float_as_uint(x), b = __float_as_uint(y);
  *hi = __builtin_amdgcn_perm(b, a, 0x07060302u);
  *lo = Bf16::pack2(x - __uint_as_float(a & 0xFFFF0000u), y - __uint_as_float(b & 0xFFFF0000u));
}

// A float32 sum as three bfloat16 parts, `plane` elements apart.
__device__ inline void store_sum(uint16_t* to, int64_t plane, float sum) {
  const uint32_t a = __float_as_uint(sum) & 0xFFFF0000u;
  const float rest = sum - __uint_as_float(a);
  const uint32_t b = __float_as_uint(rest) & 0xFFFF0000u;
  to[0] = (uint16_t)(a >> 16);
  to[plane] = (uint16_t)(b >> 16);
  to[2 * plane] = Bf16::from_f32(rest - __uint_as_float(b));
}

// The weights of a wave's four tiles over one step.  GS = 0: a width other than 4 and 8, whose
// group size is an argument.
template <class T, class X, int BITS, int GS>
struct Weights {
  static constexpr bool kWide = BITS == 4 || BITS == 8;   // 16-byte loads
  static constexpr int kVec = BITS == 4 ? 1 : 2;
  static constexpr int kLoads = TN * (kWide ? kVec : 2 * kMfmaSteps);   // loads of codes per step
  // halfwords of scales per load: two steps of them
  static constexpr int kPeriod = GS == 0 ? 1 : 2;
  static constexpr int NH = GS == 0 ? 4 : kPeriod * kStepK / (GS == 0 ? 1 : GS);
  static constexpr int kScaleRegs = GS == 0 ? 4 : NH / 2;

  __amdgpu_buffer_rsrc_t w_rs[2], s_rs[2];
  int w_voff[TN], s_voff[TN];
  u32x4 v[TN][kWide ? kVec : 1];
  uint32_t w[TN][kWide ? 1 : 2 * kMfmaSteps];
  uint32_t s[TN][kScaleRegs], s_next[TN][kScaleRegs];
  uint32_t gshift;
  int groups, group_shift;
  bool narrow;

  // row(j): first weight row of tile j; two: tiles from TN / 2 on are of the second matrix
  template <class Row>
  __device__ inline void setup(const Args& a, int e, int lane, Row row, bool two) {
    const int lg = lane >> 4, col = lane & 15;
    int gword = 0;
    gshift = 0u;
    if constexpr (!kWide) decode::generic_lane_offsets<BITS>(lg, gword, gshift);
    const int gs = a.w[0].group_size;
    group_shift = __builtin_ctz((unsigned)gs);
    groups = a.k >> group_shift;
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      const Stack& k = a.w[m];
      const uint32_t w_bytes = (uint32_t)(a.n - 1) * (uint32_t)(k.w_row_stride * 4) + (uint32_t)(a.k / 32 * BITS * 4);
      const uint32_t s_bytes = (uint32_t)(a.n - 1) * (uint32_t)(k.sb_row_stride * 2) + (uint32_t)(groups * 2);
      w_rs[m] = decode::make_rsrc(k.w + e * k.w_expert_stride, w_bytes);
      s_rs[m] = decode::make_rsrc(k.s + e * k.sb_expert_stride, s_bytes);
    }
    // scales as words: rows, experts and arrays start on one, and a row ends on one
    narrow = (groups & 1) != 0 || (((uintptr_t)a.w[0].s | (uintptr_t)a.w[1].s | (uintptr_t)a.w[0].b | (uintptr_t)a.w[1].b) % 4) != 0 ||
             ((a.w[0].sb_row_stride | a.w[1].sb_row_stride | a.w[0].sb_expert_stride | a.w[1].sb_expert_stride) & 1) != 0;
#pragma unroll
    for (int j = 0; j < TN; ++j) {
      const Stack& k = a.w[two && j >= TN / 2 ? 1 : 0];
      const int r = row(j) + col;
      w_voff[j] = r * (int)(k.w_row_stride * 4) + (kWide ? 16 * lg : 4 * gword);
      s_voff[j] = r * (int)(k.sb_row_stride * 2);
    }
  }
  __device__ inline void load_half(int j, int half, int t) {
    const auto u = __builtin_amdgcn_raw_buffer_load_b128(w_rs[j >= TN / 2], w_voff[j] + 64 * half, t * (kStepK * BITS / 8), 0);
    v[j][half] = u32x4{u[0], u[1], u[2], u[3]};
  }
  __device__ inline void load_generic(int j, int c, int t) {
    const int soff = t * (kStepK * BITS / 8);
#pragma unroll
    for (int i = 0; i < 2; ++i)
      w[j][2 * c + i] = __builtin_amdgcn_raw_buffer_load_b32(w_rs[j >= TN / 2], w_voff[j] + 4 * c * BITS + 4 * i, soff, 0);
  }
  __device__ inline void load_codes(int t) {
#pragma unroll
    for (int j = 0; j < TN; ++j) {
      if constexpr (kWide) {
#pragma unroll
        for (int h = 0; h < kVec; ++h) load_half(j, h, t);
      } else {
#pragma unroll
        for (int c = 0; c < kMfmaSteps; ++c) load_generic(j, c, t);
      }
    }
  }
  // Scales from step t on, into s_next.
  __device__ inline void load_scales(int t) {
#pragma unroll
    for (int j = 0; j < TN; ++j) {
      const __amdgpu_buffer_rsrc_t rs = s_rs[j >= TN / 2];
      if constexpr (GS == 0) {
#pragma unroll
        for (int c = 0; c < kMfmaSteps; ++c)
          s_next[j][c] = __builtin_amdgcn_raw_buffer_load_b16(rs, s_voff[j], ((t * kStepK + 32 * c) >> group_shift) * 2, 0);
      } else {
        const int soff = t * (kStepK / GS) * 2;
        decode::SbRegs<NH> r;
        if (narrow)
          decode::load_sb_buf_narrow<NH>(r, rs, s_voff[j], soff);
        else
          decode::load_sb_buf<NH>(r, rs, s_voff[j], soff);
#pragma unroll
        for (int i = 0; i < NH / 2; ++i) s_next[j][i] = r.v[i];
      }
    }
  }
  __device__ inline void next_scales() {
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int i = 0; i < kScaleRegs; ++i) s[j][i] = s_next[j][i];
  }
  // Scale of tile j in matrix step c of step t, the nth since the scales were loaded.
  __device__ inline float scale(int j, int nth, int c) const {
    if constexpr (GS == 0) return T::to_f32(s[j][c]);
    const int i = nth * (kStepK / (GS == 0 ? 1 : GS)) + c * 32 / (GS == 0 ? 1 : GS);
    return T::to_f32((s[j][i >> 1] >> (16 * (i & 1))) & 0xFFFFu);
  }
};

// LDS of the activations of one step: [plane][32-column step][row tile] of 64 operands.
template <int FM, int PLANES>
struct Shared {
  static constexpr int kEntries = PLANES * kMfmaSteps * FM * 64;
};

template <class T, class X, int BITS, int GS, int FM, int KIND>
__global__ __launch_bounds__(kThreads, FM == 2 ? 3 : 2) void grouped_kernel(const Args a) {
  constexpr int PLANES = KIND == kDown ? 2 : 1;
  constexpr int kDma = PLANES * kMfmaSteps * FM / 4;      // direct loads per wave and step
  using W = Weights<T, X, BITS, GS>;
  __shared__ u32x4 as0[Shared<FM, PLANES>::kEntries];
  __shared__ u32x4 as1[Shared<FM, PLANES>::kEntries];
  __shared__ float tile_s[KIND == kDown ? 1 : 16 * 132];

  // Workgroups go to the eight XCDs in turn.  Each XCD takes a run of consecutive tiles of a run
  // of consecutive weight blocks, tiles fastest: the tiles of an expert share its weights there.
  const int total = a.max_tiles * a.n_blocks, run = (total + 7) / 8;
  const int id = (int)(blockIdx.x & 7) * run + (int)(blockIdx.x >> 3);
  if (id >= total) return;
  const int nb = id / a.max_tiles, mt = id - nb * a.max_tiles;
  if (mt >= *a.tile_count) return;
  Tile tile = a.tiles[mt];                     // the same in every lane, which the descriptors need to know
  tile.expert = __builtin_amdgcn_readfirstlane(tile.expert);
  tile.first = __builtin_amdgcn_readfirstlane(tile.first);
  tile.rows = __builtin_amdgcn_readfirstlane(tile.rows);

  const int lane = threadIdx.x & 63, lg = lane >> 4, col = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  constexpr bool kTwo = KIND == kGated;
  // first weight row of the wave's tile j
  const auto weight_row = [&](int j) {
    return kTwo ? nb * (kBlockN / 2) + wave * 32 + 16 * (j & 1) : nb * kBlockN + wave * 64 + 16 * j;
  };
  W w;
  w.setup(a, tile.expert, lane, weight_row, kTwo);

  // ---- activations: load d of the wave is row tile di, matrix step dc, plane dp
  const auto x_row = [&](int m) -> int64_t {               // row of x of the tile's row m < rows
    if constexpr (KIND == kGated) return a.pairs[tile.first + m] / a.top_k;
    return (int64_t)tile.first + m;
  };
  // descriptor over all of x where rows are looked up, else over the tile's rows
  const uint16_t* x_base = KIND == kGated ? a.x : a.x + (int64_t)tile.first * a.x_stride;
  const uint32_t x_bytes = KIND == kGated ? a.x_bytes : (uint32_t)((int64_t)(tile.rows - 1) * a.x_stride * 2 +
                                                                   a.x_plane * (PLANES - 1) * 2 + (int64_t)a.k * 2);
  const __amdgpu_buffer_rsrc_t x_rs = decode::make_rsrc(x_base, x_bytes);
  // FM = 4: wave w loads row tile w, all its steps and planes; FM = 2: row tile w / 2, half of them
  static_assert(FM == 4 || FM == 2, "loads divide evenly");
  const int di = FM == 4 ? wave : wave >> 1, d0 = FM == 4 ? 0 : (wave & 1) * kDma;
  uint32_t x_off = kPast;                                  // of the lane's row
  if (16 * di + col < tile.rows)
    x_off = (uint32_t)((KIND == kGated ? x_row(16 * di + col) : 16 * di + col) * a.x_stride * 2);
  const int sub = decode::lane_group_of_sub<BITS>(lg);     // (its own inverse)
  uint32_t off[kDma];
  const auto load_x = [&](int t, u32x4* buf) {
#pragma unroll
    for (int d = 0; d < kDma; ++d) {
      const int dd = d0 + d, dp = dd / kMfmaSteps, dc = dd - dp * kMfmaSteps;
      const int k = t * kStepK + 32 * dc + 8 * sub;
      off[d] = k < a.k && x_off != kPast ? x_off + (uint32_t)(2 * (k + dp * (int)a.x_plane)) : kPast;
      load_to_lds(x_rs, buf + ((dp * kMfmaSteps + dc) * FM + di) * 64, off[d]);
    }
  };

  f32x4 acc[TN][FM];
  const f32x4 zero4 = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int j = 0; j < TN; ++j)
#pragma unroll
    for (int i = 0; i < FM; ++i) acc[j][i] = zero4;

  const int steps = (a.k + kStepK - 1) / kStepK;
  w.load_scales(0);
  load_x(0, as0);
  w.load_codes(0);
  w.next_scales();
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  lds_barrier();

  // Step t: reads `cur`, loads step t + 1 into `nxt` and the registers that it has emptied.  The
  // two memory fences keep the loads of codes between them, so that the count at the end says
  // that the direct loads, which came before, have landed.
  // The last step loads itself once more, which nobody uses.
  const auto step = [&](int t_in, const u32x4* cur, u32x4* nxt, auto nth_c) __attribute__((always_inline)) {
    constexpr int nth = decltype(nth_c)::value;
    const int t = __builtin_amdgcn_readfirstlane(t_in);    // (else it may be kept per lane, offset and all)
    const int next = min(t + 1, steps - 1);
    if (nth == W::kPeriod - 1) w.load_scales(next);
    asm volatile("" ::: "memory");
    load_x(next, nxt);
    asm volatile("" ::: "memory");
    const bool whole = (t + 1) * kStepK <= a.k;
    f32x4 part[TN][FM];
    u32x4 rc[TN];
#pragma unroll
    for (int c = 0; c < kMfmaSteps; ++c) {
      __builtin_amdgcn_sched_barrier(0);       // (else operands of several steps are unpacked first, and spilled)
      if constexpr (BITS == 4) {
        if (c == 0) {
#pragma unroll
          for (int j = 0; j < TN; ++j) rc[j] = decode::transpose_lane_groups(w.v[j][0]);
#pragma unroll
          for (int j = 0; j < TN; ++j) w.load_half(j, 0, next);
        }
      } else if constexpr (BITS == 8) {
        if (c % 2 == 0) {
#pragma unroll
          for (int j = 0; j < TN; ++j) rc[j] = decode::swap_halves(w.v[j][c / 2]);
#pragma unroll
          for (int j = 0; j < TN; ++j) w.load_half(j, c / 2, next);
        }
      }
      typename X::v8 av[PLANES][FM];
#pragma unroll
      for (int p = 0; p < PLANES; ++p)
#pragma unroll
        for (int i = 0; i < FM; ++i) av[p][i] = as_v8<X>(cur[((p * kMfmaSteps + c) * FM + i) * 64 + lane]);
      constexpr int kGroupSteps = GS == 0 ? 1 : GS / 32;
      const bool fresh = c % kGroupSteps == 0, last = (c + 1) % kGroupSteps == 0;
#pragma unroll
      for (int j = 0; j < TN; ++j) {
        u32x4 q;
        if constexpr (BITS == 4) {
          q = codes4_natural<X>(rc[j][c]);
        } else if constexpr (BITS == 8) {
          q = c % 2 ? codes8_to_v8<X>(rc[j].z, rc[j].w) : codes8_to_v8<X>(rc[j].x, rc[j].y);
        } else {
          q = codesN_to_v8<X, BITS>(w.w[j][2 * c], w.w[j][2 * c + 1], w.gshift);
          w.load_generic(j, c, next);
        }
        const typename X::v8 bq = as_v8<X>(q);
#pragma unroll
        for (int p = PLANES - 1; p >= 0; --p)
#pragma unroll
          for (int i = 0; i < FM; ++i) part[j][i] = X::mfma(av[p][i], bq, fresh && p == PLANES - 1 ? zero4 : part[j][i]);
        if (last) {
          // groups past K: their scales are not theirs
          const bool ok = whole || t * kStepK + 32 * c < a.k;
          const float s = ok ? w.scale(j, nth, c) : 0.f;
#pragma unroll
          for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r) acc[j][i][r] = __builtin_fmaf(s, part[j][i][r], acc[j][i][r]);
        }
      }
    }
    if (nth == W::kPeriod - 1) w.next_scales();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0x0F70 | (W::kLoads & 15) | ((W::kLoads >> 4) << 14));   // vmcnt(kLoads)
    asm volatile("" ::: "memory");
#pragma unroll
    for (int d = 0; d < kDma; ++d) asm volatile("" ::"v"(off[d]));
    lds_barrier();
  };
  using First = std::integral_constant<int, 0>;
  using Second = std::integral_constant<int, W::kPeriod - 1>;
  for (int t = 0; t < steps; t += 2) {
    step(t, as0, as1, First{});
    if (t + 1 >= steps) break;
    step(t + 1, as1, as0, Second{});
  }

  // ---- biases: 32 groups at a time
  {
    const uint16_t* sum_rows[FM];
#pragma unroll
    for (int i = 0; i < FM; ++i)
      sum_rows[i] = a.sums + x_row(min(16 * i + col, tile.rows - 1)) * (kPlanes * (int64_t)a.sum_groups) + 8 * lg;
    for (int g0 = 0; g0 < w.groups; g0 += 32) {
      bf16x8 sv[kPlanes][FM];
#pragma unroll
      for (int p = 0; p < kPlanes; ++p)
#pragma unroll
        for (int i = 0; i < FM; ++i) sv[p][i] = as_v8<Bf16>(*(const u32x4*)(sum_rows[i] + p * a.sum_groups + g0));
#pragma unroll
      for (int j = 0; j < TN; ++j) {
        const Stack& k = a.w[kTwo && j >= TN / 2 ? 1 : 0];
        const int row = weight_row(j) + col;
        uint32_t b[4] = {0u, 0u, 0u, 0u};
        const uint16_t* p = k.b + tile.expert * k.sb_expert_stride + (int64_t)min(row, a.n - 1) * k.sb_row_stride + g0 + 8 * lg;
        const int left = w.groups - g0 - 8 * lg;
        if (!w.narrow && left >= 8) {
#pragma unroll
          for (int e = 0; e < 4; ++e) b[e] = ((const uint32_t*)p)[e];
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (e < left) b[e >> 1] |= (uint32_t)p[e] << (16 * (e & 1));
        }
        u32x4 hi = {b[0], b[1], b[2], b[3]}, lo = {0u, 0u, 0u, 0u};
        if constexpr (T::kDtype == QMM_FP16) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            uint32_t h, l;
            split_pair(T::to_f32(b[e] & 0xFFFFu), T::to_f32(b[e] >> 16), &h, &l);
            hi[e] = h;
            lo[e] = l;
          }
        }
#pragma unroll
        for (int i = 0; i < FM; ++i) {
          if constexpr (T::kDtype == QMM_FP16) {
            acc[j][i] = Bf16::mfma(sv[1][i], as_v8<Bf16>(lo), acc[j][i]);
            acc[j][i] = Bf16::mfma(sv[0][i], as_v8<Bf16>(lo), acc[j][i]);
          }
#pragma unroll
          for (int q = kPlanes - 1; q >= 0; --q) acc[j][i] = Bf16::mfma(sv[q][i], as_v8<Bf16>(hi), acc[j][i]);
        }
      }
    }
  }

  // ---- results: element (row 16 i + 4 lg + r, weight row weight_row(j) + col) is acc[j][i][r]
  if constexpr (KIND == kDown) {
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int m = 16 * i + 4 * lg + r;
        if (m >= tile.rows) continue;
        float* o = a.out + (int64_t)a.pairs[tile.first + m] * a.n;
#pragma unroll
        for (int j = 0; j < TN; ++j) {
          const int n = weight_row(j) + col;
          if (n < a.n) o[n] = acc[j][i][r];
        }
      }
  } else if constexpr (KIND == kGated) {
    // 16 rows at a time through LDS, so that a thread has eight consecutive columns of a row
    const int row = threadIdx.x >> 4, c8 = (threadIdx.x & 15) * 8;
    const int n0 = nb * (kBlockN / 2);
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      if (16 * i >= tile.rows) break;
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float g = acc[j][i][r];
          tile_s[(4 * lg + r) * 132 + wave * 32 + 16 * j + col] = g / (1.0f + expf(-g)) * acc[j + 2][i][r];
        }
      lds_barrier();
      const int m = 16 * i + row;
      float v[8], sum = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        v[e] = n0 + c8 + e < a.n ? tile_s[row * 132 + c8 + e] : 0.f;
        sum += v[e];
      }
      sum += __shfl_xor(sum, 1);
      sum += __shfl_xor(sum, 2);
      if (a.h_group >= 64) sum += __shfl_xor(sum, 4);
      if (a.h_group == 128) sum += __shfl_xor(sum, 8);
      if (m < tile.rows) {
        const int64_t pos = (int64_t)tile.first + m;
        u32x4 hi, lo;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          uint32_t h, l;
          split_pair(v[2 * e], v[2 * e + 1], &h, &l);
          hi[e] = h;
          lo[e] = l;
        }
        uint16_t* to = a.h + pos * 2 * a.h_cols + n0 + c8;
        *(u32x4*)to = hi;
        *(u32x4*)(to + a.h_cols) = lo;
        if (c8 % a.h_group == 0) store_sum(a.h_sums + pos * kPlanes * a.h_sum_groups + (n0 + c8) / a.h_group, a.h_sum_groups, sum);
      }
      lds_barrier();
    }
    // groups that the sums are padded to: zero
    if (nb == a.n_blocks - 1) {
      const int g0 = a.h_cols / a.h_group, pad = a.h_sum_groups - g0;
      for (int e = threadIdx.x; e < tile.rows * pad; e += kThreads) {
        const int m = e / pad;
        store_sum(a.h_sums + ((int64_t)tile.first + m) * kPlanes * a.h_sum_groups + g0 + (e - m * pad), a.h_sum_groups, 0.f);
      }
    }
  } else {
    uint16_t* ys = (uint16_t*)tile_s;                      // [16][264]
    const int row = threadIdx.x >> 4, c16 = (threadIdx.x & 15) * 16;
    const int n0 = nb * kBlockN;
    const bool vec = a.y_stride % 8 == 0 && ((uintptr_t)a.y & 15u) == 0u;
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      if (16 * i >= tile.rows) break;
#pragma unroll
      for (int j = 0; j < TN; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r) ys[(4 * lg + r) * 264 + wave * 64 + 16 * j + col] = T::from_f32(acc[j][i][r]);
      lds_barrier();
      const int m = 16 * i + row;
      if (m < tile.rows) {
        uint16_t* to = a.y + ((int64_t)tile.first + m) * a.y_stride + n0 + c16;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const u32x4 u = *(const u32x4*)(ys + row * 264 + c16 + 8 * h);
          if (vec && n0 + c16 + 8 * h + 8 <= a.n) {
            *(u32x4*)(to + 8 * h) = u;
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
              if (n0 + c16 + 8 * h + e < a.n) to[8 * h + e] = (uint16_t)(u[e >> 1] >> (16 * (e & 1)));
          }
        }
      }
      lds_barrier();
    }
  }
}

template <class T, class X, int BITS, int GS, int KIND>
hipError_t launch_kind(const Args& a, int tile_rows, hipStream_t stream) {
  const unsigned blocks = (unsigned)((a.max_tiles * a.n_blocks + 7) / 8 * 8);
  if (tile_rows == 64)
    hipLaunchKernelGGL((grouped_kernel<T, X, BITS, GS, 4, KIND>), dim3(blocks), dim3(kThreads), 0, stream, a);
  else
    hipLaunchKernelGGL((grouped_kernel<T, X, BITS, GS, 2, KIND>), dim3(blocks), dim3(kThreads), 0, stream, a);
  return hipGetLastError();
}

template <class T, int BITS, int GS>
hipError_t launch_group(const Args& a, Kind kind, int tile_rows, hipStream_t stream) {
  switch (kind) {
    case kPlain: return launch_kind<T, T, BITS, GS, kPlain>(a, tile_rows, stream);
    case kGated: return launch_kind<T, T, BITS, GS, kGated>(a, tile_rows, stream);
    case kDown: return launch_kind<T, Bf16, BITS, GS, kDown>(a, tile_rows, stream);
  }
  return hipErrorInvalidValue;
}

template <int BITS, int GS>
hipError_t launch_dtype(const Args& a, Kind kind, int dtype, int tile_rows, hipStream_t stream) {
  return dtype == QMM_BF16 ? launch_group<Bf16, BITS, GS>(a, kind, tile_rows, stream)
                           : launch_group<Fp16, BITS, GS>(a, kind, tile_rows, stream);
}

}  // namespace grouped
}  // namespace qmm
