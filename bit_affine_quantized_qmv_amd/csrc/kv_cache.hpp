// Layout and launch interface of the 4-bit key/value cache.
//
// The cache is one array of 32-bit words [pages][heads][page words]; the words of one page of
// one head hold its K rows, then its V rows:
//     K codes  page_size * D/8 words      K (s, b)  D/gs * page_size words
//     V codes  page_size * D/8 words      V (s, b)  D/gs * page_size words
// A word of the (s, b) areas is one token's scale (low half) and bias (high half) of one
// group, [group][token], so the four consecutive tokens that a lane of an MFMA accumulator
// owns are one 16-byte load.
//
// The codes sit in the order in which the matrix cores take them, because one wave reads a
// row once per step and has no time to shuffle it:
//   K  token t's row is D/8 words of 8 consecutive codes (element e of a word at bits 4e);
//      word w (elements 8w .. 8w+7) is stored at t * D/8 + (w % 4) * D/32 + w / 4.  A lane
//      of lane group h feeds the 32-element steps c = 0 .. D/32-1 of q . k with words
//      4c + h, which are then consecutive: one load of D/8 bytes.
//   V  the products contract over tokens, so a lane feeds 8 tokens of one element.  Element
//      d = 16 i + o (o = d % 16) of token t is nibble i % 2 (low first) of the byte
//      t % 4 of word ((t / 4) * 16 + o) * D/32 + i / 2: the four bytes of a word are four
//      consecutive tokens, its two nibbles the elements of two 16-row output tiles.
//      A lane reads its row o of four tokens with one load of D/8 bytes.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/qmm.h"

namespace qmm {
namespace kv {

constexpr int kBits = 4;

// Sizes of one page of one head, in words.
__host__ __device__ constexpr int64_t code_words(int64_t page_size, int head_dim) { return page_size * (head_dim / 8); }
__host__ __device__ constexpr int64_t sb_words(int64_t page_size, int head_dim, int group) {
  return page_size * (head_dim / group);
}
__host__ __device__ constexpr int64_t side_words(int64_t page_size, int head_dim, int group) {
  return code_words(page_size, head_dim) + sb_words(page_size, head_dim, group);
}

// Word of the K code word w (elements 8w .. 8w+7) of token t in the page's K codes.
__host__ __device__ constexpr int k_word(int t, int w, int head_dim) {
  return t * (head_dim / 8) + (w % 4) * (head_dim / 32) + w / 4;
}
// Byte of elements d = 16i + o, i in {2j, 2j+1}, of token t in the page's V codes.
__host__ __device__ constexpr int v_byte(int t, int o, int j, int head_dim) {
  return (((t / 4) * 16 + o) * (head_dim / 32) + j) * 4 + t % 4;
}

// Block (entry of a block table) of the 16-token tile `tile`: tile / d with d = page_size / 16,
// by the reciprocal 2^38 / d rounded up.  With tiles below 2^26 (2^30 tokens) and d <= 2^12 the
// product stays below 2^64, and the rounding adds less than 2^38 / d to it, so that the quotient
// is exact.
constexpr int kRecipShift = 38;
__host__ __device__ constexpr uint64_t page_recip(int page_size) {
  return ((1ull << kRecipShift) + (uint64_t)(page_size / 16) - 1) / (uint64_t)(page_size / 16);
}
__host__ __device__ constexpr int block_of_tile(uint32_t tile, uint64_t recip) {
  return (int)(((uint64_t)tile * recip) >> kRecipShift);
}

struct CacheArgs {
  uint32_t* data;
  int64_t pages;
  int64_t side;         // words of one page's K (or V) side
  int32_t page_size;
  int32_t heads;
  int32_t head_dim;
  int32_t group_size;
  int32_t dtype;
};

// Validate a cache descriptor and fill `out` (host only; the data pointer when `pointers`).
constexpr int64_t kMaxInt = 0x7FFFFFFF;
int32_t check_cache(const qmm_kv_cache_t* c, bool pointers, CacheArgs* out);

struct AppendArgs {
  CacheArgs c;
  const void* x[2];     // K and V rows
  int64_t token_stride[2];
  int64_t head_stride[2];
  int64_t tokens;
  const int32_t* slots;
};

struct ReadArgs {
  CacheArgs c;
  void* out[2];         // dense [count, heads, head_dim]
  int64_t count;
  const int32_t* slots;
};

struct AttendArgs {
  CacheArgs c;
  const void* q;
  int64_t q_batch_stride, q_token_stride, q_head_stride;
  int64_t batch;
  int32_t q_len;
  int32_t q_heads;
  int32_t rep;            // query heads per cached head
  int32_t rows;           // q_len * rep: query rows that share one cached head
  const int32_t* table;   // [batch, table_stride]
  int64_t table_stride;
  int32_t max_blocks;
  const int32_t* lengths;
  int32_t max_length;
  float scale_log2;       // scale * log2(e)
  int32_t causal;
  int32_t window;         // 0: none
  int32_t chunk;          // tokens per split, a multiple of the tokens of one workgroup step
  int32_t splits;
  void* out;              // dense [batch, q_len, q_heads, head_dim]
  uint64_t page_recip;    // page_recip(page_size)
  const uint32_t* mask;   // trees: [batch, q_len, mask_words], the nodes that a query sees
  int32_t mask_words;
  const int32_t* depth;   // trees with a window: [batch, q_len]
  float* part;            // splits > 1: [batch * heads * rows][splits][head_dim] sums, then their (max, sum) pairs
};

// Append: workgroups of one call, each with the rows of one side of one head (a read's have both
// sides, so half as many); a launch has fewer than 2^32 threads along its grid.
constexpr int kCopyThreads = 256;
inline int64_t copy_blocks(const CacheArgs& c, int64_t tokens) {
  const int64_t rows = kCopyThreads / (c.head_dim / 8);
  return (tokens + rows - 1) / rows * 2 * c.heads;
}
constexpr int64_t kMaxCopyBlocks = 0xFFFFFFFFll / kCopyThreads;

hipError_t launch_append(const AppendArgs& a, hipStream_t stream);
hipError_t launch_read(const ReadArgs& a, hipStream_t stream);

// What the waves of a workgroup share out: the tokens, for 16 query rows or (trees) for two tiles
// of 16, or the query rows.
enum AttendForm { kTokensForm, kPairsForm, kRowsForm };
// Two tiles' registers fit two waves per SIMD (groups of 32 do not; 64 elements were not tried).
constexpr bool has_pairs(int head_dim, int group) { return head_dim == 128 && group >= 64; }

// Splits of the token range and tokens per split of an attention call (host only).
struct AttendPlan {
  int32_t form;           // AttendForm
  int32_t row_tiles;      // workgroups along the rows of one cached head
  int32_t chunk;
  int32_t splits;
};
AttendPlan plan_attend(int64_t batch, const CacheArgs& c, int64_t rows, int64_t range, bool tree);

hipError_t launch_attend_bf16(const AttendArgs& a, const AttendPlan& p, hipStream_t stream);
hipError_t launch_attend_fp16(const AttendArgs& a, const AttendPlan& p, hipStream_t stream);
hipError_t launch_attend_tree_bf16(const AttendArgs& a, const AttendPlan& p, hipStream_t stream);
hipError_t launch_attend_tree_fp16(const AttendArgs& a, const AttendPlan& p, hipStream_t stream);

}  // namespace kv
}  // namespace qmm
