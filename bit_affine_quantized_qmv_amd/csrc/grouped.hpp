// Launch interface of the matrix products grouped by expert, and of the expert layer built on them.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "moe.hpp"

namespace qmm {
namespace grouped {

using moe::Stack;

constexpr int kThreads = 256;
constexpr int kBlockN = 256;          // weight rows per workgroup: four waves of four 16-row tiles
constexpr int kStepK = 128;           // rows of staged activations are whole steps of this
constexpr int kPlanes = 3;            // bfloat16 parts of a group's sum of activations
constexpr int kSumPad = 32;           // groups per row of the sums, rounded up to this
constexpr int kMaxPairs = 1 << 20;    // rows of one call
constexpr int kSplitGroups = 32;      // a split of the columns is whole runs of so many groups

// What becomes of a product x W_e^T.
enum Kind {
  kPlain,      // y, rounded to dtype
  kGated,      // two products (gate, up): h = silu(g) u in two bfloat16 parts, and the sums of its groups
  kDown,       // x in two parts; float32, to the row of the (token, choice) pair
};

// Up to `rows` consecutive rows of one expert.
struct Tile {
  int32_t expert;
  int32_t first;
  int32_t rows;
  int32_t expert_first;      // the expert's first tile, and the number of its tiles
  int32_t expert_tiles;
  int32_t unused[3];
};

struct Args {
  // Activations, rows of whole steps (zeros behind k), each eight elements in the order in which the
  // weights' codes are expanded: row r at r * x_stride, its rest (kDown) x_plane further.
  const uint16_t* x;
  int64_t x_stride;
  int64_t x_plane;
  uint32_t x_bytes;          // kGated: bytes of all rows, below 2^31
  const uint16_t* sums;      // [x row][kPlanes][sum_groups]
  int32_t sum_groups;
  Stack w[2];                // kGated: gate and up; else twice the same
  int32_t n, k;
  const Tile* tiles;
  const int32_t* tile_count;
  int32_t max_tiles;
  int32_t n_blocks;
  const int32_t* pairs;      // kGated, kDown: pair (token * top_k + choice) of a row
  int32_t top_k;
  uint16_t* y;               // kPlain
  int64_t y_stride;
  uint16_t* h;               // kGated: [row][2][h_cols]
  int32_t h_cols;
  uint16_t* h_sums;          // kGated: [row][kPlanes][h_sum_groups]
  int32_t h_sum_groups;
  int32_t h_group;
  int32_t h_bits;            // width and group size of the weights that take h
  // kDown: the columns are shared out over `splits` workgroups, split_cols each (whole runs of
  // kSplitGroups groups, or all of them), which leave a result of their own each.
  int32_t splits;
  int32_t split_cols;
  float* out;                // kDown: [split][pair][n]
  int64_t out_split;         // elements from one split to the next
};

// x as the products take it, the sums of its groups, and the tiles of given offsets: one kernel.
struct PrepareArgs {
  const uint16_t* x;
  int64_t x_stride;
  uint16_t* staged;          // [rows][cols]
  int32_t cols;              // k rounded up to whole steps
  int32_t bits;
  int64_t rows;
  int32_t k;
  int32_t group;
  int32_t dtype;
  uint16_t* sums;            // [rows][kPlanes][sum_groups]
  int32_t sum_groups;
  int32_t experts;
  const int32_t* offsets;    // [experts + 1]; null: no tiles are made
  int32_t tile_rows;
  Tile* tiles;
  int32_t max_tiles;
  int32_t* tile_count;
};

// Workgroups of kThreads threads that take a row of x, 2048 columns each: its columns and what they and
// the sums are padded to.
__host__ __device__ inline int64_t blocks_per_row(const PrepareArgs& a) {
  const int64_t sums = (int64_t)a.sum_groups * a.group, n = sums > a.cols ? sums : a.cols;
  return (n + 8 * kThreads - 1) / (8 * kThreads);
}
// Workgroups of prepare_kernel, of kMake threads: those of the rows, and one for the tiles.
constexpr int kMake = 1024;
inline int64_t prepare_blocks(const PrepareArgs& a) {
  constexpr int64_t per = kMake / kThreads;
  return (a.rows * blocks_per_row(a) + per - 1) / per + 1;
}
// Workgroups along x of a product: an equal run of the work for each of the eight XCDs.
inline int64_t product_blocks(const Args& a) { return ((int64_t)a.max_tiles * a.n_blocks + 7) / 8 * 8; }
// A launch has fewer threads than this along its grid.
constexpr int64_t kLaunchThreads = 1ll << 32;

// Routing of the expert layer: each token's choices, then the rows of every expert.
struct RouteArgs {
  const uint16_t* router;
  int64_t router_stride;
  int32_t tokens;
  int32_t experts;
  int32_t top_k;
  int32_t renormalize;
  int32_t dtype;
  int32_t* pair_expert;      // [tokens * top_k]
  float* pair_share;
  int32_t* pairs;            // [tokens * top_k]: pair of each row, by expert
  int32_t tile_rows;
  Tile* tiles;
  int32_t max_tiles;
  int32_t* tile_count;
};

// The weighted sum of a token's pairs.
struct SumArgs {
  int32_t tokens;
  int32_t top_k;
  int32_t renormalize;
  int32_t hidden;            // a multiple of 4
  int32_t dtype;
  int32_t splits;
  const float* out;          // [split][tokens * top_k][hidden]
  const float* share;        // [tokens * top_k]
  uint16_t* y;               // [tokens][y_stride]
  int64_t y_stride;
};

hipError_t launch_sum(const SumArgs& a, hipStream_t stream);
hipError_t launch_prepare(const PrepareArgs& a, hipStream_t stream);
hipError_t launch_route(const RouteArgs& r, const PrepareArgs& p, hipStream_t stream);
// tile_rows: 16, 32 or 64
hipError_t launch_b4(const Args& a, Kind kind, int dtype, int tile_rows, hipStream_t stream);
hipError_t launch_b8(const Args& a, Kind kind, int dtype, int tile_rows, hipStream_t stream);
hipError_t launch_bn(const Args& a, Kind kind, int dtype, int tile_rows, hipStream_t stream);

}  // namespace grouped
}  // namespace qmm
