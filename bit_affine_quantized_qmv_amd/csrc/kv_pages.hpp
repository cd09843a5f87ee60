// Launch interface of the operators on trees of drafted tokens and on pages of the cache.
#pragma once

#include "kv_cache.hpp"

namespace qmm {
namespace kv {

constexpr int kMaxNodes = 1024;

struct TreeMaskArgs {
  const int32_t* parents;    // [batch, stride]
  int64_t stride;
  int64_t batch;
  int32_t nodes;
  int32_t words;             // mask words per node
  int32_t window;            // 0: none
  uint32_t* mask;            // [batch, nodes, words]
  int32_t* depth;            // [batch, nodes] or null
};

struct TreeAcceptArgs {
  const int32_t* parents;    // [batch, .] each
  const int32_t* tokens;
  const int32_t* sampled;
  int64_t parents_stride, tokens_stride, sampled_stride;
  int64_t batch;
  int32_t nodes;
  int32_t* path;             // [batch, nodes]
  int32_t* count;            // [batch]
  int32_t* last;             // [batch]
};

struct MoveArgs {
  CacheArgs c;
  const int32_t* table;      // [batch, table_stride]: pages that are read
  int64_t table_stride;
  int64_t blocks;
  const int32_t* to;         // pages that are written
  int64_t to_stride;
  int64_t to_blocks;
  const int32_t* index;      // [batch, index_stride]
  int64_t index_stride;
  int64_t batch;
  int32_t count;
  const int32_t* origin;     // [batch] or null
  const int32_t* start;      // [batch]
  int32_t in_place;
};

struct CopyPagesArgs {
  CacheArgs c;
  const int32_t* src;
  const int32_t* dst;
  int64_t count;
  int64_t page_quads;        // 16-byte quads of a page, all heads
};

struct ForkArgs {
  int32_t* refs;             // [pages]
  int64_t pages;
  const int32_t* table;      // [batch, table_stride]
  int64_t table_stride;
  int64_t batch;
  int64_t blocks;
  const int32_t* lengths;    // [batch]
  const int32_t* parents;    // [rows]
  const int32_t* want;       // [rows] or null
  int64_t rows;
  int32_t* new_table;        // [rows, new_stride]
  int64_t new_stride;
  int64_t new_blocks;
  int32_t page_size;
  int32_t* copy_src;         // [rows]
  int32_t* copy_dst;
  int32_t* short_of;         // [1]
  // workspace
  int32_t segments;
  int32_t* need;             // [rows]: fresh pages of a row
  int32_t* cut;              // [rows]: pages of a row past new_blocks
  int32_t* open;             // [segments]: free pages of a segment of the pool
  int32_t* list;             // the first free pages, at most list_size
  int64_t list_size;
};

constexpr int kForkThreads = 256;
constexpr int kSegment = 4096;   // pages of the pool per workgroup

hipError_t launch_tree_mask(const TreeMaskArgs& a, hipStream_t stream);
hipError_t launch_tree_accept(const TreeAcceptArgs& a, hipStream_t stream);
hipError_t launch_move(const MoveArgs& a, hipStream_t stream);
hipError_t launch_copy_pages(const CopyPagesArgs& a, hipStream_t stream);
hipError_t launch_fork(const ForkArgs& a, hipStream_t stream);

}  // namespace kv
}  // namespace qmm
