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
// 64 of them, so a code is unpacked once per tile.  Codes and activations go from memory to LDS
// by direct loads, a step of STEP columns ahead, and from there to registers as operands; a wave's
// codes are its own, the activations are shared and double-buffered, with one barrier per step.
//
// What decides is how the lanes of a load are laid out.  Four consecutive lanes that stay within
// 64 bytes move 54 to 59 bytes per cycle and CU from L2, also straight to LDS; in the layout that the
// matrix instruction takes, lane = row, they are in four rows, and the same load moves 15.5.  With
// codes loaded that way into registers (and activations 16 rows x 64 bytes at a time) the products of
// 4094 rows, 4096 x 14336, took 1240 us (gate, up) and 1040 (down).
//
// Measured: 4094 rows, 8 experts of [14336, 4096] in 4 bits, groups of 128: gate and up 1010 us, 0.95
// PFLOP/s, the matrix cores busy half of the time; down (two passes for the two parts of h) 805 us, busy
// 64%.  The unpacking and the scaling are 2.9 vector instructions for each matrix instruction (1.5 in down,
// whose two passes share them; 4.0 in groups of 64), and with two waves per SIMD their cycles add up: gate and
// up issue 2.34e8 of 4 cycles and 6.58e7 of 16, 0.97 ms at the about 2 GHz that the clock falls to under both.
// 509 rows, 128 experts of [704, 1408] in 8 bits: 32 us, 4.4 TB/s.  Codes two steps ahead instead of one, waiting for the older half of
// the loads only: no faster (gate and up of 32 rows 139 us against 142, of 384 rows in 128 experts 39
// against 34).
#pragma once

#include <type_traits>

#include "decode_impl.hpp"
#include "grouped.hpp"

namespace qmm {
namespace grouped {

constexpr int TN = 4;                          // weight tiles per wave
constexpr uint32_t kPast = 0x7FFFFF00u;        // an offset past every descriptor: reads zero

typedef __attribute__((address_space(3))) void lds_void_t;

// 16 bytes per lane, at byte offset `off` + `soff`, to the wave's 1 KB of LDS at `to`.
__device__ inline void load_to_lds(__amdgpu_buffer_rsrc_t rs, u32x4* to, uint32_t off, int soff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_void_t*)to, 16, off, soff, 0, 0);
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

// LDS of the activations of one step: [plane][64-column half][row][8 chunks of 8 columns]; chunk q of row
// r is at place q ^ Codes::x_place(r).  A direct load moves 8 rows of 128 bytes.
template <int FM, int PLANES, int STEP>
struct Shared {
  static constexpr int kHalf = 16 * FM * 8;              // entries of one half
  static constexpr int kEntries = PLANES * (STEP / 64) * kHalf;
};

// How the codes of a wave's 64 rows lie in LDS and reach the operands.  A row has 64 bytes there (128
// 4-bit or 64 8-bit codes), 16-byte piece p of row r at place p ^ row_place(r).  A chunk is eight consecutive codes, what a lane gives to one matrix step.  Any chunks of a group
// can meet in a matrix step, as long as the activations' are the same: a lane group takes kRun
// consecutive chunks, as many as the group allows, for one wide read.
template <int BITS, int GS, int STEP>
struct Codes {
  static constexpr int kSteps = STEP / 32;                // matrix steps
  static constexpr int kRun = GS == 32 ? 1 : (STEP == 128 && GS == 128 ? 4 : 2);
  static constexpr int kReads = kSteps / kRun;            // reads per tile and step
  static constexpr int kBytes = kRun * BITS;              // of one
  static constexpr int kBlockSteps = BITS == 4 ? 128 / STEP : 1;   // steps that a direct load covers
  // The LDS serves a 16-byte read of lane = row in groups of 16 lanes: of two neighbouring lane groups
  // rows 0-3 and 12-15 of the first with 4-11 of the second, then the others.  The places put such
  // a group's 16 pieces into different banks, where the two lane groups read different chunks.
  __device__ static constexpr int row_place(int r) {
    const int t = (r >> 2) & 3;
    return (((t << 1) ^ t) & 2) | (t >> 1);
  }
  __device__ static constexpr int x_place(int r) {
    const int p = (r >> 1) & 7;
    return kRun == 1 ? p : ((p << 1) & 6) | (((p >> 2) ^ (p >> 1)) & 1);
  }
  // place and offset of the lane group's first chunk; what read r of a step is xored with
  __device__ static constexpr int piece(int lg) { return kBytes == 16 ? lg : (kBytes == 8 ? lg >> 1 : 0); }
  __device__ static constexpr int offset(int lg) { return kBytes == 16 ? 0 : (kBytes == 8 ? 8 * (lg & 1) : 4 * lg); }
  __device__ static constexpr int read_piece(int r, int half) {
    return kBytes == 16 ? 0 : (kBytes == 8 ? 2 * (r + half) : r + 2 * half);
  }
  // the activations' chunk of lane group lg in matrix step c: 64-column half, and place in it
  __device__ static constexpr int lane_half(int lg) { return kRun == 4 ? lg >> 1 : 0; }
  __device__ static constexpr int lane_chunk(int lg) { return kRun == 4 ? 4 * (lg & 1) : (kRun == 2 ? 2 * lg : lg); }
  __device__ static constexpr int step_half(int c) { return kRun == 4 ? 0 : c >> 1; }
  __device__ static constexpr int step_chunk(int c) { return kRun == 4 ? c : (kRun == 2 ? c & 1 : 4 * (c & 1)); }
};

typedef uint32_t u32x4_by4 __attribute__((ext_vector_type(4), aligned(4)));

template <class T, class X, int BITS, int GS, int FM, int KIND>
__global__ __launch_bounds__(kThreads, FM == 1 ? 4 : (FM == 2 ? 3 : 2)) void grouped_kernel(const Args a) {
  constexpr int PLANES = KIND == kDown ? 2 : 1;
  constexpr bool kLds = BITS == 4 || BITS == 8;           // other widths: codes from memory to registers
  // columns of a step: what leaves room for two workgroups per CU
  constexpr int STEP = BITS == 4 && PLANES == 1 ? 128 : 64;
  constexpr int MS = STEP / 32;
  constexpr int kGroupSteps = GS == 0 ? 1 : GS / 32;      // matrix steps of a group
  constexpr int kHalves = kGroupSteps > MS ? kGroupSteps / MS : 1;   // steps of a group
  constexpr int kLoads = PLANES * (STEP / 64) * 2 * FM;   // direct loads of activations per step
  using L = Shared<FM, PLANES, STEP>;
  using C = Codes<kLds ? BITS : 4, GS == 0 ? 32 : GS, STEP>;
  __shared__ u32x4 as0[L::kEntries], as1[L::kEntries];
  __shared__ u32x4 bs[kLds ? 1024 : 528];                 // codes of four waves; then rows of the result
  __shared__ u32x4 ss[256];                               // eight scales of each weight row

  // Workgroups go to the eight XCDs in turn.  Each XCD takes a run of the work in the order expert,
  // weight block, tile: what runs there at a time shares both weights and activations.  (In the
  // order weight block, tile, expert each XCD went through all activations for every block.)
  const int total = *a.tile_count * a.n_blocks, run = (total + 7) / 8;
  const int id = (int)(blockIdx.x & 7) * run + (int)(blockIdx.x >> 3);
  if ((int)(blockIdx.x >> 3) >= run || id >= total) return;
  const Tile* any = a.tiles + id / a.n_blocks;             // a tile of the same expert
  const int local = id - any->expert_first * a.n_blocks;
  const int nb = __builtin_amdgcn_readfirstlane(local / any->expert_tiles);
  const Tile* mine = a.tiles + any->expert_first + (local - nb * any->expert_tiles);
  // the same in every lane, which the descriptors need to know
  struct {
    int expert, first, rows;
  } tile = {__builtin_amdgcn_readfirstlane(mine->expert), __builtin_amdgcn_readfirstlane(mine->first),
            __builtin_amdgcn_readfirstlane(mine->rows)};

  const int lane = threadIdx.x & 63, lg = lane >> 4, col = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  constexpr bool kTwo = KIND == kGated;
  // first weight row of the wave's tile j
  const auto weight_row = [&](int j) {
    return kTwo ? nb * (kBlockN / 2) + wave * 32 + 16 * (j & 1) : nb * kBlockN + wave * 64 + 16 * j;
  };
  const auto stack = [&](int j) -> const Stack& { return a.w[kTwo && j >= TN / 2 ? 1 : 0]; };
  const int group_shift = __builtin_ctz((unsigned)a.w[0].group_size), groups = a.k >> group_shift;
  // the steps of this split
  const int all_steps = (a.k + STEP - 1) / STEP;
  const int first_step = KIND == kDown ? (int)blockIdx.y * (a.split_cols / STEP) : 0;
  const int steps = KIND == kDown ? min(all_steps, first_step + (a.split_cols + STEP - 1) / STEP) : all_steps;

  // ---- codes
  __amdgpu_buffer_rsrc_t w_rs[2];
#pragma unroll
  for (int m = 0; m < 2; ++m) {
    const Stack& k = a.w[m];
    w_rs[m] = decode::make_rsrc(k.w + tile.expert * k.w_expert_stride,
                                (uint32_t)(a.n - 1) * (uint32_t)(k.w_row_stride * 4) + (uint32_t)(a.k / 32 * BITS * 4));
  }
  int w_voff[TN];                                          // rows past the last read as zeros
  int gword = 0;
  uint32_t gshift = 0u;
  if constexpr (!kLds) decode::generic_lane_offsets<BITS>(lg, gword, gshift);
#pragma unroll
  for (int j = 0; j < TN; ++j) {
    const int row_bytes = (int)(stack(j).w_row_stride * 4);
    if constexpr (kLds) {
      const int r = lane >> 2, piece = (lane & 3) ^ C::row_place(r);
      w_voff[j] = (weight_row(j) + r) * row_bytes + 16 * piece;
    } else {
      w_voff[j] = (weight_row(j) + col) * row_bytes + 4 * gword;
    }
  }
  // direct loads of the codes of block `blk` (64 bytes of each row), to the wave's part of LDS
  u32x4* const my_codes = bs + (kLds ? wave * 256 : 0);
  const auto load_codes = [&](int blk) {
    if constexpr (kLds) {
#pragma unroll
      for (int j = 0; j < TN; ++j) load_to_lds(w_rs[kTwo && j >= TN / 2], my_codes + 64 * j, w_voff[j], 64 * blk);
    }
  };
  const int code_at = wave * 4096 + 64 * col + C::offset(lg), code_piece = C::piece(lg) ^ C::row_place(col);
  u32x4 rc[TN];                                            // a step's codes of the lane
  const auto read_codes = [&](int half) {
    if constexpr (kLds) {
#pragma unroll
      for (int j = 0; j < TN; ++j)
#pragma unroll
        for (int r = 0; r < C::kReads; ++r) {
          const char* p = (const char*)bs + code_at + 1024 * j + 16 * (code_piece ^ C::read_piece(r, half));
          if constexpr (C::kBytes == 16) {
            rc[j] = *(const u32x4*)p;
          } else if constexpr (C::kBytes == 8) {
            const uint2 u = *(const uint2*)p;
            rc[j][2 * r] = u.x;
            rc[j][2 * r + 1] = u.y;
          } else {
            rc[j][r] = *(const uint32_t*)p;
          }
        }
    }
  };
  uint32_t gw[TN][kLds ? 1 : 2 * MS];                      // other widths
  const auto load_generic = [&](int j, int c, int t) {
    if constexpr (!kLds) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
        gw[j][2 * c + i] = __builtin_amdgcn_raw_buffer_load_b32(w_rs[kTwo && j >= TN / 2], w_voff[j] + 4 * c * BITS + 4 * i,
                                                                t * (STEP * BITS / 8), 0);
    }
  };

  // ---- scales: lane r loads those of the wave's weight row r, eight groups at a time, well ahead, and
  // leaves them in LDS when their first step comes.  Groups and rows past the last are zero.
  const bool narrow = (((uintptr_t)a.w[0].s | (uintptr_t)a.w[1].s | (uintptr_t)a.w[0].b | (uintptr_t)a.w[1].b) & 3) != 0 ||
                      ((a.w[0].sb_row_stride | a.w[1].sb_row_stride | a.w[0].sb_expert_stride | a.w[1].sb_expert_stride) & 1) != 0;
  const Stack& s_stack = a.w[kTwo ? lane >> 5 : 0];
  const int s_row = weight_row(lane >> 4) + col;
  const uint16_t* s_ptr = s_stack.s + tile.expert * s_stack.sb_expert_stride + (int64_t)min(s_row, a.n - 1) * s_stack.sb_row_stride;
  const uint32_t s_mask = s_row < a.n ? 0xFFFFFFFFu : 0u;
  u32x4 s_next = {0u, 0u, 0u, 0u};
  const auto load_scales = [&](int g0) {
    if (!narrow && g0 + 8 <= groups) {
      s_next = *(const u32x4_by4*)(s_ptr + g0);
    } else {
      s_next = u32x4{0u, 0u, 0u, 0u};
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (g0 + e < groups) s_next[e >> 1] |= (uint32_t)s_ptr[g0 + e] << (16 * (e & 1));
    }
  };
  const char* const my_scales = (const char*)(ss + wave * 64 + col);

  // ---- activations
  const auto x_row = [&](int m) -> int64_t {               // row of x of the tile's row m < rows
    if constexpr (KIND == kGated) return a.pairs[tile.first + m] / a.top_k;
    return (int64_t)tile.first + m;
  };
  // descriptor over all of x where rows are looked up, else over the tile's rows; rows are whole steps
  const uint16_t* x_base = KIND == kGated ? a.x : a.x + (int64_t)tile.first * a.x_stride;
  const uint32_t x_bytes = KIND == kGated ? a.x_bytes : (uint32_t)(tile.rows * a.x_stride * 2);
  const __amdgpu_buffer_rsrc_t x_rs = decode::make_rsrc(x_base, x_bytes);
  // load d of the wave: 8 rows of one half and plane; the wave's rows are the same in all of them
  constexpr int kMine = FM == 4 ? 2 : 1;                   // octets of rows of the wave
  const auto octet = [&](int u) { return FM == 1 ? wave & 1 : wave + 4 * u; };
  uint32_t x_off[kMine];                                   // of the lane's rows and chunk
#pragma unroll
  for (int u = 0; u < kMine; ++u) {
    const int m = 8 * octet(u) + (lane >> 3);
    const int chunk = (lane & 7) ^ C::x_place(m);
    x_off[u] = kPast;
    if (m < tile.rows) x_off[u] = (uint32_t)((KIND == kGated ? x_row(m) : m) * a.x_stride * 2) + 16 * chunk;
  }
  const auto load_x = [&](int t, u32x4* buf) {
#pragma unroll
    for (int d = 0; d < (kLoads + 3) / 4; ++d) {
      if (kLoads < 4 && wave >= kLoads) break;
      const int u = d % kMine, part = FM == 1 ? 2 * d + (wave >> 1) : d / kMine;
      const int half = part % (STEP / 64), p = part / (STEP / 64);
      load_to_lds(x_rs, buf + part * L::kHalf + 64 * octet(u), x_off[u], 2 * (t * STEP + 64 * half + p * (int)a.x_plane));
    }
  };
  const int x_entry = C::lane_half(lg) * L::kHalf + 8 * col, x_chunk = C::lane_chunk(lg) ^ C::x_place(col);

  f32x4 acc[TN][FM], part[TN][FM];
  const f32x4 zero4 = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int j = 0; j < TN; ++j)
#pragma unroll
    for (int i = 0; i < FM; ++i) acc[j][i] = part[j][i] = zero4;

  load_scales((first_step * STEP) >> group_shift);
  load_x(first_step, as0);
  load_codes(first_step / C::kBlockSteps);
  if constexpr (!kLds) {
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int c = 0; c < MS; ++c) load_generic(j, c, first_step);
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  lds_barrier();

  // Step t reads `cur` and loads step t + 1 into `nxt`, and into the places that it has emptied; the last
  // step loads itself once more, which nobody uses.  half: which step of the group, or of the block of
  // codes, it is.
  const auto step = [&](int t_in, const u32x4* cur, u32x4* nxt, auto half_c) __attribute__((always_inline)) {
    constexpr int half = decltype(half_c)::value;
    const int t = __builtin_amdgcn_readfirstlane(t_in);    // (else it may be kept per lane, offset and all)
    const int next = min(t + 1, steps - 1);
    load_x(next, nxt);
    const int g0 = (t * STEP) >> group_shift;              // the step's first group
    if (((t * STEP) & ((8 << group_shift) - 1)) == 0) {
      ss[wave * 64 + lane] = s_next & s_mask;
      if (g0 + 8 < groups) load_scales(g0 + 8);
    }
    read_codes(C::kBlockSteps == 2 ? half : 0);
    // scales of the groups that end in the step, as many as one read has
    constexpr int kScales = GS == 0 ? MS : (MS / kGroupSteps > 0 ? MS / kGroupSteps : 1);
    uint32_t sc[TN][(kScales + 1) / 2];
#pragma unroll
    for (int j = 0; j < TN; ++j) {
      const char* p = my_scales + 256 * j + 2 * (g0 & 7);
      if constexpr (GS == 0) {
        sc[j][0] = 0u;
#pragma unroll
        for (int c = 0; c < MS; ++c)
          sc[j][0] |= (uint32_t)*(const uint16_t*)(my_scales + 256 * j + 2 * (((t * STEP + 32 * c) >> group_shift) & 7)) << (16 * c);
      } else if constexpr (kScales == 1) {
        sc[j][0] = *(const uint16_t*)p;
      } else if constexpr (kScales == 2) {
        sc[j][0] = *(const uint32_t*)p;
      } else {
        const uint2 u = *(const uint2*)p;
        sc[j][0] = u.x;
        sc[j][kScales / 4] = u.y;
      }
    }
    typename X::v8 av[2][PLANES][FM];
    const auto read_x = [&](int c) {
#pragma unroll
      for (int p = 0; p < PLANES; ++p)
#pragma unroll
        for (int i = 0; i < FM; ++i)
          av[c & 1][p][i] = as_v8<X>(
              cur[(p * (STEP / 64) + C::step_half(c)) * L::kHalf + 128 * i + x_entry + (x_chunk ^ C::step_chunk(c))]);
    };
    read_x(0);
    if constexpr (kLds) {
      if (C::kBlockSteps == 1 || half == 1) {              // the codes are out of LDS: the next ones may come
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        load_codes(min(t / C::kBlockSteps + 1, (steps - 1) / C::kBlockSteps));
      }
    }
    // operand of tile j in matrix step c
    const auto codes = [&](int j, int c) {
      if constexpr (BITS == 4) {
        return codes4_to_v8<X>(rc[j][c]);
      } else if constexpr (BITS == 8) {
        return c % 2 ? codes8_to_v8<X>(rc[j].z, rc[j].w) : codes8_to_v8<X>(rc[j].x, rc[j].y);
      } else {
        const u32x4 q = codesN_to_v8<X, BITS>(gw[j][2 * c], gw[j][2 * c + 1], gshift);
        load_generic(j, c, next);
        return q;
      }
    };
    const auto last_of_group = [](int c) { return (half % kHalves * MS + c + 1) % kGroupSteps == 0; };
    const auto first_of_group = [](int c) { return (half % kHalves * MS + c) % kGroupSteps == 0; };
    // a finished group of tile j: its products, scaled, to the sums
    const auto add_group = [&](int j, int c) {
      const int i = GS == 0 ? c : (kScales == 1 ? 0 : c / kGroupSteps);
      const float s = T::to_f32((sc[j][i >> 1] >> (16 * (i & 1))) & 0xFFFFu);
#pragma unroll
      for (int m = 0; m < FM; ++m)
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[j][m][r] = __builtin_fmaf(s, part[j][m][r], acc[j][m][r]);
    };
    u32x4 q = codes(0, 0);
    // The products of a tile, with the unpacking of the next one's codes and the scaling of the last
    // one's group between them, one by one: the matrix core works while the vector unit does.
#pragma unroll
    for (int c = 0; c < MS; ++c) {
#pragma unroll
      for (int j = 0; j < TN; ++j) {
        __builtin_amdgcn_sched_barrier(0);
        if (j == 0 && c + 1 < MS) read_x(c + 1);
        u32x4 q_next = q;
        if (j + 1 < TN)
          q_next = codes(j + 1, c);
        else if (c + 1 < MS)
          q_next = codes(0, c + 1);
        const typename X::v8 bq = as_v8<X>(q);
#pragma unroll
        for (int p = PLANES - 1; p >= 0; --p)
#pragma unroll
          for (int i = 0; i < FM; ++i)
            part[j][i] = X::mfma(av[c & 1][p][i], bq, first_of_group(c) && p == PLANES - 1 ? zero4 : part[j][i]);
        const bool adds = j > 0 ? last_of_group(c) : (c > 0 && last_of_group(c - 1));
        if (j > 0 && last_of_group(c)) add_group(j - 1, c);
        if (j == 0 && c > 0 && last_of_group(c - 1)) add_group(TN - 1, c - 1);
        // (the mask's bits: 8 a matrix instruction, 2 a vector one)
        const int each = ((adds ? 4 * FM : 0) + 10 + FM * PLANES - 1) / (FM * PLANES);
#pragma unroll
        for (int i = 0; i < FM * PLANES; ++i) {
          __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
          if (each <= 1) __builtin_amdgcn_sched_group_barrier(0x002, 1, 0);
          else if (each == 2) __builtin_amdgcn_sched_group_barrier(0x002, 2, 0);
          else if (each == 3) __builtin_amdgcn_sched_group_barrier(0x002, 3, 0);
          else if (each <= 6) __builtin_amdgcn_sched_group_barrier(0x002, 6, 0);
          else __builtin_amdgcn_sched_group_barrier(0x002, 10, 0);
        }
        q = q_next;
      }
    }
    __builtin_amdgcn_sched_barrier(0);
    if (last_of_group(MS - 1)) add_group(TN - 1, MS - 1);
    // (the sums are taken here: else the multiply-adds sink below the next step's branches, and
    // the products that they wait for fill the registers)
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int i = 0; i < FM; ++i) asm volatile("" : "+v"(acc[j][i]));
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");       // the next step's loads, a step old
    lds_barrier();
  };
  using First = std::integral_constant<int, 0>;
  using Second = std::integral_constant<int, 1>;
  int t = first_step;
  for (; t + 1 < steps; t += 2) {
    step(t, as0, as1, First{});
    step(t + 1, as1, as0, Second{});
  }
  if (t < steps) step(t, as0, as1, First{});

  // ---- biases: 32 groups at a time, what a split has whole runs of
  {
    const uint16_t* sum_rows[FM];
#pragma unroll
    for (int i = 0; i < FM; ++i)
      sum_rows[i] = a.sums + x_row(min(16 * i + col, tile.rows - 1)) * (kPlanes * (int64_t)a.sum_groups) + 8 * lg;
    const int last = min(groups, (steps * STEP) >> group_shift);
    for (int g0 = (first_step * STEP) >> group_shift; g0 < last; g0 += kSplitGroups) {
      bf16x8 sv[kPlanes][FM];
#pragma unroll
      for (int p = 0; p < kPlanes; ++p)
#pragma unroll
        for (int i = 0; i < FM; ++i) sv[p][i] = as_v8<Bf16>(*(const u32x4*)(sum_rows[i] + p * a.sum_groups + g0));
#pragma unroll
      for (int j = 0; j < TN; ++j) {
        const Stack& k = stack(j);
        const int row = weight_row(j) + col;
        uint32_t b[4] = {0u, 0u, 0u, 0u};
        const uint16_t* p = k.b + tile.expert * k.sb_expert_stride + (int64_t)min(row, a.n - 1) * k.sb_row_stride + g0 + 8 * lg;
        const int left = groups - g0 - 8 * lg;
        if (!narrow && left >= 8) {
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
        float* o = a.out + blockIdx.y * a.out_split + (int64_t)a.pairs[tile.first + m] * a.n;
#pragma unroll
        for (int j = 0; j < TN; ++j) {
          const int n = weight_row(j) + col;
          if (n < a.n) o[n] = acc[j][i][r];
        }
      }
  } else if constexpr (KIND == kGated) {
    // 16 rows at a time through LDS, so that a thread has eight consecutive columns of a row
    float* const tile_s = (float*)bs;                      // [16][132]
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
        if (a.h_bits == 4) {                               // the order in which 4-bit codes are expanded
          hi = interleave_even_odd(hi);
          lo = interleave_even_odd(lo);
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
    uint16_t* const ys = (uint16_t*)bs;                    // [16][264]
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
  const dim3 grid((unsigned)product_blocks(a), KIND == kDown ? (unsigned)a.splits : 1u);
  if (tile_rows == 16)
    hipLaunchKernelGGL((grouped_kernel<T, X, BITS, GS, 1, KIND>), grid, dim3(kThreads), 0, stream, a);
  else if (tile_rows == 64)
    hipLaunchKernelGGL((grouped_kernel<T, X, BITS, GS, 4, KIND>), grid, dim3(kThreads), 0, stream, a);
  else
    hipLaunchKernelGGL((grouped_kernel<T, X, BITS, GS, 2, KIND>), grid, dim3(kThreads), 0, stream, a);
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
