// extern "C" entry points of the operators on trees of drafted tokens and on pages of the cache:
// validate, launch.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <string>

#include "capi_internal.hpp"
#include "kv_pages.hpp"

namespace qmm {
namespace kv {
namespace {

int32_t check_tree_sizes(const char* who, int64_t batch, int64_t nodes) {
  if (batch < 0 || batch > 65535 || nodes < 0 || nodes > kMaxNodes)
    return report(QMM_ERR_SHAPE, std::string(who) + ": need 0 <= batch <= 65535 and 0 <= nodes <= 1024");
  return QMM_OK;
}

bool unaligned4(const void* p) { return (uintptr_t)p % 4 != 0; }

int64_t align64(int64_t ints) { return (ints + 15) / 16 * 16; }

// Workspace of a fork, in ints: need, cut, open, list.
int64_t fork_ints(const qmm_kv_fork_t* f, int64_t* segments, int64_t* list) {
  *segments = (f->pages + kSegment - 1) / kSegment;
  *list = std::min(f->pages, f->rows * f->new_blocks);
  return 2 * align64(f->rows) + align64(*segments) + *list;
}

int32_t check_fork(const qmm_kv_fork_t* f) {
  if (!f) return report(QMM_ERR_NULL, "kv_fork: args must be non-NULL");
  if (f->page_size < 16 || f->page_size % 16 || f->page_size > 65536)
    return report(QMM_ERR_SHAPE, "kv_fork: page_size must be a multiple of 16 in [16, 65536]");
  if (f->pages < 1 || f->pages > kMaxInt / f->page_size)
    return report(QMM_ERR_SHAPE, "kv_fork: need pages >= 1 and pages * page_size < 2^31");
  if (f->batch < 0 || f->batch > 65535 || f->rows < 0 || f->rows > 65535)
    return report(QMM_ERR_SHAPE, "kv_fork: need 0 <= batch, rows <= 65535");
  if (f->blocks < 0 || f->new_blocks < 0 || f->table_stride < f->blocks || f->new_stride < f->new_blocks)
    return report(QMM_ERR_SHAPE, "kv_fork: need 0 <= blocks <= table_stride and 0 <= new_blocks <= new_stride");
  if (f->blocks > kMaxInt / f->page_size || f->new_blocks > kMaxInt / f->page_size)
    return report(QMM_ERR_SHAPE, "kv_fork: blocks * page_size and new_blocks * page_size must be below 2^31");
  if (f->rows * f->new_blocks > (1ll << 30)) return report(QMM_ERR_SHAPE, "kv_fork: rows * new_blocks must be at most 2^30");
  return QMM_OK;
}

}  // namespace
}  // namespace kv
}  // namespace qmm

using namespace qmm;

extern "C" {

int32_t qmm_tree_mask(const int32_t* parents, int64_t parents_stride, int64_t batch, int64_t nodes, int64_t window,
                      uint32_t* mask, int32_t* depth, void* stream) {
  return guarded([&]() -> int32_t {
    const int32_t rc = kv::check_tree_sizes("tree_mask", batch, nodes);
    if (rc != QMM_OK) return rc;
    if (parents_stride < nodes) return report(QMM_ERR_SHAPE, "tree_mask: parents_stride < nodes");
    if (window < 0) return report(QMM_ERR_UNSUPPORTED, "tree_mask: window must be >= 0");
    if (batch == 0 || nodes == 0) return report(QMM_OK, "");
    if (!parents || !mask) return report(QMM_ERR_NULL, "tree_mask: parents and mask must be non-NULL");
    if (kv::unaligned4(parents) || kv::unaligned4(mask) || kv::unaligned4(depth))
      return report(QMM_ERR_ALIGN, "tree_mask: parents, mask and depth must be 4-byte aligned");
    kv::TreeMaskArgs a{parents, parents_stride, batch, (int32_t)nodes, (int32_t)((nodes + 31) / 32),
                       (int32_t)std::min<int64_t>(window, kv::kMaxNodes), mask, depth};   // no path is longer
    return report_launch(kv::launch_tree_mask(a, (hipStream_t)stream));
  });
}

int32_t qmm_tree_accept(const qmm_tree_accept_t* t, int32_t* path, int32_t* count, int32_t* last, void* stream) {
  return guarded([&]() -> int32_t {
    if (!t) return report(QMM_ERR_NULL, "tree_accept: args must be non-NULL");
    const int32_t rc = kv::check_tree_sizes("tree_accept", t->batch, t->nodes);
    if (rc != QMM_OK) return rc;
    if (t->nodes < 1) return report(QMM_ERR_SHAPE, "tree_accept: need at least one node");
    if (t->parents_stride < t->nodes || t->tokens_stride < t->nodes || t->sampled_stride < t->nodes)
      return report(QMM_ERR_SHAPE, "tree_accept: strides smaller than a row");
    if (t->batch == 0) return report(QMM_OK, "");
    if (!t->parents || !t->tokens || !t->sampled || !path || !count || !last)
      return report(QMM_ERR_NULL, "tree_accept: pointers must be non-NULL");
    for (const void* p : {(const void*)t->parents, (const void*)t->tokens, (const void*)t->sampled, (const void*)path,
                          (const void*)count, (const void*)last})
      if (kv::unaligned4(p)) return report(QMM_ERR_ALIGN, "tree_accept: arrays must be 4-byte aligned");
    kv::TreeAcceptArgs a{t->parents,        t->tokens, t->sampled,        t->parents_stride, t->tokens_stride,
                         t->sampled_stride, t->batch,  (int32_t)t->nodes, path,              count,
                         last};
    return report_launch(kv::launch_tree_accept(a, (hipStream_t)stream));
  });
}

int32_t qmm_kv_move(const qmm_kv_cache_t* cache, const qmm_kv_move_t* m, void* stream) {
  return guarded([&]() -> int32_t {
    kv::MoveArgs a{};
    if (!m) return report(QMM_ERR_NULL, "kv_move: args must be non-NULL");
    const bool empty = m->batch == 0 || m->count == 0;
    const int32_t rc = kv::check_cache(cache, !empty, &a.c);
    if (rc != QMM_OK) return rc;
    if (m->batch < 0 || m->batch > 65535 || m->count < 0 || m->count > (1 << 30))
      return report(QMM_ERR_SHAPE, "kv_move: need 0 <= batch <= 65535 and 0 <= count <= 2^30");
    if (m->batch * a.c.heads >= (1 << 24)) return report(QMM_ERR_SHAPE, "kv_move: batch * heads must be below 2^24");
    if (m->blocks < 0 || m->table_stride < m->blocks || m->to_blocks < 0 || (m->to_table && m->to_stride < m->to_blocks) ||
        m->index_stride < m->count)
      return report(QMM_ERR_SHAPE, "kv_move: strides smaller than a row");
    if (empty) return report(QMM_OK, "");
    if (!m->block_table || !m->index || !m->start)
      return report(QMM_ERR_NULL, "kv_move: block_table, index and start must be non-NULL");
    for (const void* p : {(const void*)m->block_table, (const void*)m->to_table, (const void*)m->index,
                          (const void*)m->origin, (const void*)m->start})
      if (kv::unaligned4(p)) return report(QMM_ERR_ALIGN, "kv_move: arrays must be 4-byte aligned");
    a.table = m->block_table;
    a.table_stride = m->table_stride;
    a.blocks = m->blocks;
    a.in_place = m->to_table == nullptr;
    a.to = a.in_place ? m->block_table : m->to_table;
    a.to_stride = a.in_place ? m->table_stride : m->to_stride;
    a.to_blocks = a.in_place ? m->blocks : m->to_blocks;
    a.index = m->index;
    a.index_stride = m->index_stride;
    a.batch = m->batch;
    a.count = (int32_t)m->count;
    a.origin = m->origin;
    a.start = m->start;
    return report_launch(kv::launch_move(a, (hipStream_t)stream));
  });
}

int32_t qmm_kv_copy_pages(const qmm_kv_cache_t* cache, const int32_t* src, const int32_t* dst, int64_t count,
                          void* stream) {
  return guarded([&]() -> int32_t {
    kv::CopyPagesArgs a{};
    const int32_t rc = kv::check_cache(cache, count > 0, &a.c);
    if (rc != QMM_OK) return rc;
    if (count < 0 || count > kv::kMaxInt) return report(QMM_ERR_SHAPE, "kv_copy_pages: need 0 <= count < 2^31");
    if (count == 0) return report(QMM_OK, "");
    if (!src || !dst) return report(QMM_ERR_NULL, "kv_copy_pages: src and dst must be non-NULL");
    if (kv::unaligned4(src) || kv::unaligned4(dst))
      return report(QMM_ERR_ALIGN, "kv_copy_pages: src and dst must be 4-byte aligned");
    a.src = src;
    a.dst = dst;
    a.count = count;
    a.page_quads = 2 * a.c.side * a.c.heads / 4;
    return report_launch(kv::launch_copy_pages(a, (hipStream_t)stream));
  });
}

int64_t qmm_kv_fork_workspace_bytes(const qmm_kv_fork_t* args) {
  return guarded([&]() -> int64_t {
    const int32_t rc = kv::check_fork(args);
    if (rc != QMM_OK) return rc;
    report(QMM_OK, "");
    int64_t segments, list;
    return 4 * kv::fork_ints(args, &segments, &list);
  });
}

int32_t qmm_kv_fork(const qmm_kv_fork_t* f, int32_t* copy_src, int32_t* copy_dst, int32_t* short_of, void* workspace,
                    int64_t workspace_bytes, void* stream) {
  return guarded([&]() -> int32_t {
    const int32_t rc = kv::check_fork(f);
    if (rc != QMM_OK) return rc;
    if (!f->refs || !short_of || !workspace || (f->batch > 0 && (!f->lengths || (f->blocks > 0 && !f->block_table))) ||
        (f->rows > 0 && (!f->parents || !copy_src || !copy_dst || (f->new_blocks > 0 && !f->new_table))))
      return report(QMM_ERR_NULL, "kv_fork: arrays must be non-NULL");
    for (const void* p : {(const void*)f->refs, (const void*)f->block_table, (const void*)f->lengths,
                          (const void*)f->parents, (const void*)f->want, (const void*)f->new_table,
                          (const void*)copy_src, (const void*)copy_dst, (const void*)short_of, (const void*)workspace})
      if (kv::unaligned4(p)) return report(QMM_ERR_ALIGN, "kv_fork: arrays must be 4-byte aligned");
    int64_t segments, list;
    const int64_t need = 4 * kv::fork_ints(f, &segments, &list);
    if (workspace_bytes < need)
      return report(QMM_ERR_SHAPE, "kv_fork: workspace of " + std::to_string(workspace_bytes) + " bytes, needs " +
                                       std::to_string(need));
    kv::ForkArgs a{};
    a.refs = f->refs;
    a.pages = f->pages;
    a.table = f->block_table;
    a.table_stride = f->table_stride;
    a.batch = f->batch;
    a.blocks = f->blocks;
    a.lengths = f->lengths;
    a.parents = f->parents;
    a.want = f->want;
    a.rows = f->rows;
    a.new_table = f->new_table;
    a.new_stride = f->new_stride;
    a.new_blocks = f->new_blocks;
    a.page_size = f->page_size;
    a.copy_src = copy_src;
    a.copy_dst = copy_dst;
    a.short_of = short_of;
    a.segments = (int32_t)segments;
    int32_t* ws = (int32_t*)workspace;
    a.need = ws;
    ws += kv::align64(f->rows);
    a.cut = ws;
    ws += kv::align64(f->rows);
    a.open = ws;
    ws += kv::align64(segments);
    a.list = ws;
    a.list_size = list;
    return report_launch(kv::launch_fork(a, (hipStream_t)stream));
  });
}

}  // extern "C"
