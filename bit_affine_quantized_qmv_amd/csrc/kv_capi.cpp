// extern "C" entry points of the 4-bit key/value cache: validate, plan, launch.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <string>

#include "capi_internal.hpp"
#include "kv_pages.hpp"

namespace qmm {
namespace kv {

int32_t check_cache(const qmm_kv_cache_t* c, bool pointers, CacheArgs* out) {
  if (!c) return report(QMM_ERR_NULL, "kv: cache must be non-NULL");
  if (c->dtype != QMM_BF16 && c->dtype != QMM_FP16)
    return report(QMM_ERR_UNSUPPORTED, "kv: dtype must be QMM_BF16 or QMM_FP16");
  if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256)
    return report(QMM_ERR_UNSUPPORTED, "kv: head_dim=" + std::to_string(c->head_dim) + " not in {64,128,256}");
  if ((c->group_size != 32 && c->group_size != 64 && c->group_size != 128) || c->group_size > c->head_dim)
    return report(QMM_ERR_UNSUPPORTED,
                  "kv: group_size=" + std::to_string(c->group_size) + " not in {32,64,128} or larger than head_dim");
  if (c->page_size < 16 || c->page_size % 16 || c->page_size > 65536)
    return report(QMM_ERR_SHAPE, "kv: page_size must be a multiple of 16 in [16, 65536]");
  if (c->heads < 1 || c->heads > 4096) return report(QMM_ERR_SHAPE, "kv: need 1 <= heads <= 4096");
  if (c->pages < 1 || c->pages > kMaxInt / c->page_size)
    return report(QMM_ERR_SHAPE, "kv: need pages >= 1 and pages * page_size < 2^31");
  if (pointers) {
    if (!c->data) return report(QMM_ERR_NULL, "kv: cache data must be non-NULL");
    if ((uintptr_t)c->data % 16) return report(QMM_ERR_ALIGN, "kv: cache data must be 16-byte aligned");
  }
  *out = CacheArgs{c->data,     c->pages,    side_words(c->page_size, c->head_dim, c->group_size),
                   c->page_size, c->heads,    c->head_dim,
                   c->group_size, c->dtype};
  return QMM_OK;
}

namespace {

int32_t check_attend(const qmm_kv_cache_t* cache, const qmm_kv_attend_t* q, bool pointers, AttendArgs* a) {
  const int32_t rc = check_cache(cache, pointers, &a->c);
  if (rc != QMM_OK) return rc;
  if (!q) return report(QMM_ERR_NULL, "kv_attend: args must be non-NULL");
  if (q->batch < 0 || q->batch > 65535 || q->q_len < 0 || q->q_len > kMaxInt / 65536)
    return report(QMM_ERR_SHAPE, "kv_attend: need 0 <= batch <= 65535 and 0 <= q_len < 32768");
  if (q->q_heads < 1 || q->q_heads % cache->heads || q->q_heads > 65535)
    return report(QMM_ERR_SHAPE, "kv_attend: q_heads must be a positive multiple of the cache's heads (at most 65535)");
  if (q->window < 0 || (q->window > 0 && !q->causal))
    return report(QMM_ERR_UNSUPPORTED, "kv_attend: window must be >= 0 and needs causal");
  if (q->max_blocks < 0 || q->table_stride < q->max_blocks || q->max_blocks > kMaxInt / cache->page_size)
    return report(QMM_ERR_SHAPE, "kv_attend: need 0 <= max_blocks <= table_stride, max_blocks * page_size < 2^31");
  if (q->max_length < 0 || q->max_length > q->max_blocks * cache->page_size || q->max_length > (1 << 30))
    return report(QMM_ERR_SHAPE, "kv_attend: max_length must be in [0, max_blocks * page_size] and at most 2^30");
  if (q->q_batch_stride < 0 || q->q_token_stride < 0 || q->q_head_stride < 0)
    return report(QMM_ERR_LAYOUT, "kv_attend: negative q stride");
  if (q->q_batch_stride % 8 || q->q_token_stride % 8 || q->q_head_stride % 8)
    return report(QMM_ERR_ALIGN, "kv_attend: q strides must be multiples of 8 elements");
  a->q = q->q;
  a->q_batch_stride = q->q_batch_stride;
  a->q_token_stride = q->q_token_stride;
  a->q_head_stride = q->q_head_stride;
  a->batch = q->batch;
  a->q_len = (int32_t)q->q_len;
  a->q_heads = q->q_heads;
  a->rep = q->q_heads / cache->heads;
  if (q->q_len * a->rep > kMaxInt / 8) return report(QMM_ERR_SHAPE, "kv_attend: too many query rows per kv head");
  a->rows = (int32_t)(q->q_len * a->rep);
  a->table = q->block_table;
  a->table_stride = q->table_stride;
  a->max_blocks = (int32_t)q->max_blocks;
  a->lengths = q->lengths;
  a->max_length = (int32_t)q->max_length;
  a->scale_log2 = q->scale * 1.44269504088896340736f;
  a->causal = q->causal != 0;
  a->window = (int32_t)std::min<int64_t>(q->window, 1 << 30);   // positions stay below 2^30: no limit
  return QMM_OK;
}

// Tokens a wave's rows may span: everything, or the window of all the call's queries (and the
// rounding of its start down to a step).
int64_t token_range(const AttendArgs& a) {
  if (!a.window) return a.max_length;
  return std::min<int64_t>(a.max_length, (int64_t)a.window + a.q_len + 32);
}

// Floats of the split sums of `splits` splits.
int64_t part_floats(const AttendArgs& a, int64_t splits) {
  return splits <= 1 ? 0 : a.batch * a.c.heads * a.rows * splits * (a.c.head_dim + 2);
}

}  // namespace

// Rows: single tokens, drafts and short chunks take 16 query rows of one kv head per workgroup,
// whose waves share out the tokens; long chunks (prompts) take the form whose waves have 16
// rows of their own each and share the unpacked tokens.  Measured, the first form against the
// second: head_dim 128, 8192 tokens, 192 rows 60 us / 67, 256 rows 73 / 66; head_dim 64, 512
// rows 46 / 50, 1024 rows 87 / 79; head_dim 256, 800 rows 107 / 121, 2048 rows 265 / 246.
// Splits: as many as make one workgroup per CU in the prompt form and at head_dim 256 (only one
// is resident: 19 us against 35 with four, 8192 tokens), two, as many as are resident, with four
// groups per row (17 us / 20), else four, which are resident with one group per row.  With two
// groups three are, and the fourth still pays where lengths differ (32 ragged sequences, 128
// elements in groups of 64: 53 us against 63 with three); more do not (131071 tokens, one group:
// 35 us, with six 39).  Each split has at least one step of every wave (128 tokens), or 512 tokens
// in the prompt form, where a split's sums are large.
// Trees of 256 query rows and more, 128 elements in one or two groups, take the first form with two
// tiles of 16 rows per wave, two workgroups per CU: their workgroups fill the chip where 256 rows
// in one leave half of it idle (group 64, batch 16, 2048 tokens, 256 rows 98 us against 123; batch
// 1, 8192 tokens, 256 rows 42 / 59; one group, 512 rows, 131071 tokens 526 / 600; the other way
// only for a single long sequence in two groups: 65536 tokens, 256 rows 182 / 162).  With fewer
// rows they gain where lengths are alike (128 rows, batch 16, 8192 tokens 176 us / 212) and lose
// where they differ (121 / 112) or three do not fill a CU (batch 12: 118 / 100).  Trees of 64 or 256
// elements keep the prompts' limit of 1024 rows, which is low for them: 64 elements, batch 16, 512 to 8192
// tokens, 1020 rows in the first form 478 us, 1024 in the prompts' 624.
namespace {

struct Shape {
  AttendForm form;
  int32_t row_tiles;
  int64_t step, want;
};

Shape shape_of(int64_t batch, int heads, int head_dim, int group, int64_t rows, bool tree) {
  Shape s{};
  s.form = rows < (head_dim == 128 ? 256 : 1024) ? kTokensForm
           : tree && has_pairs(head_dim, group)  ? kPairsForm
                                                 : kRowsForm;
  const int64_t wg_rows = s.form == kRowsForm ? (head_dim == 256 ? 128 : 256) : (s.form == kPairsForm ? 32 : 16);
  s.row_tiles = (int32_t)((rows + wg_rows - 1) / wg_rows);
  s.step = s.form == kRowsForm ? 512 : 128;
  const int64_t per_cu = s.form == kRowsForm || head_dim == 256 ? 1 : (head_dim == 4 * group || s.form == kPairsForm ? 2 : 4);
  s.want = std::max<int64_t>(1, 256 * per_cu / std::max<int64_t>(1, batch * heads * s.row_tiles));
  return s;
}

}  // namespace

AttendPlan plan_attend(int64_t batch, const CacheArgs& c, int64_t rows, int64_t range, bool tree) {
  const Shape s = shape_of(batch, c.heads, c.head_dim, c.group_size, rows, tree);
  const int64_t steps = std::max<int64_t>(1, (range + s.step - 1) / s.step);
  const int64_t per = std::max<int64_t>(1, (steps + s.want - 1) / s.want);
  return AttendPlan{s.form, s.row_tiles, (int32_t)(per * s.step), (int32_t)((steps + per - 1) / per)};
}

// Splits that no shorter range of the same call exceeds.
static int64_t most_splits(const AttendArgs& a, bool tree) {
  const Shape s = shape_of(a.batch, a.c.heads, a.c.head_dim, a.c.group_size, a.rows, tree);
  return std::min<int64_t>(s.want, std::max<int64_t>(1, (a.max_length + s.step - 1) / s.step));
}

// check_attend for a tree: its queries are its nodes.
static int32_t check_tree(const qmm_kv_cache_t* cache, const qmm_kv_attend_t* q, bool pointers, AttendArgs* a) {
  const int32_t rc = check_attend(cache, q, pointers, a);
  if (rc != QMM_OK) return rc;
  if (!q->causal) return report(QMM_ERR_UNSUPPORTED, "kv_attend_tree: causal must be set");
  if (q->q_len > kMaxNodes)
    return report(QMM_ERR_SHAPE, "kv_attend_tree: " + std::to_string(q->q_len) + " nodes, at most " + std::to_string(kMaxNodes));
  return QMM_OK;
}

// Plans and launches a checked call; with a.mask a tree's.
static int32_t run_attend(AttendArgs& a, void* out, void* workspace, int64_t workspace_bytes, hipStream_t stream) {
  if (!a.q || !out || !a.lengths || (a.max_length > 0 && !a.table))
    return report(QMM_ERR_NULL, "kv_attend: q, out, lengths and block_table must be non-NULL");
  if ((uintptr_t)a.q % 16 || (uintptr_t)out % 16 || (uintptr_t)workspace % 16)
    return report(QMM_ERR_ALIGN, "kv_attend: q, out and workspace must be 16-byte aligned");
  if ((uintptr_t)a.table % 4 || (uintptr_t)a.lengths % 4)
    return report(QMM_ERR_ALIGN, "kv_attend: block_table and lengths must be 4-byte aligned");
  const AttendPlan p =
      plan_attend(a.batch, a.c, a.rows, token_range(a), a.mask != nullptr);
  if ((int64_t)a.c.heads * p.row_tiles > 65535)
    return report(QMM_ERR_SHAPE, "kv_attend: too many query rows per sequence");
  const int64_t need = part_floats(a, p.splits) * 4;
  if (need > 0 && !workspace) return report(QMM_ERR_NULL, "kv_attend: workspace must be non-NULL");
  if (workspace_bytes < need)
    return report(QMM_ERR_SHAPE, "kv_attend: workspace of " + std::to_string(workspace_bytes) + " bytes, needs " +
                                     std::to_string(need));
  a.page_recip = page_recip(a.c.page_size);
  a.chunk = p.chunk;
  a.splits = p.splits;
  a.out = out;
  a.part = (float*)workspace;
  if (a.mask)
    return report_launch(a.c.dtype == QMM_BF16 ? launch_attend_tree_bf16(a, p, stream)
                                               : launch_attend_tree_fp16(a, p, stream));
  return report_launch(a.c.dtype == QMM_BF16 ? launch_attend_bf16(a, p, stream) : launch_attend_fp16(a, p, stream));
}

}  // namespace kv
}  // namespace qmm

using namespace qmm;

extern "C" {

int32_t qmm_kv_append(const qmm_kv_cache_t* cache, const void* k, int64_t k_token_stride, int64_t k_head_stride,
                      const void* v, int64_t v_token_stride, int64_t v_head_stride, const int32_t* slots,
                      int64_t tokens, void* stream) {
  return guarded([&]() -> int32_t {
    kv::AppendArgs a{};
    const int32_t rc = kv::check_cache(cache, tokens > 0, &a.c);
    if (rc != QMM_OK) return rc;
    if (tokens < 0 || tokens > kv::kMaxInt) return report(QMM_ERR_SHAPE, "kv_append: need 0 <= tokens < 2^31");
    if (kv::copy_blocks(a.c, tokens) > kv::kMaxCopyBlocks)
      return report(QMM_ERR_SHAPE, "kv_append: tokens * heads * head_dim must be below 2^34");
    if (k_token_stride < 0 || k_head_stride < 0 || v_token_stride < 0 || v_head_stride < 0)
      return report(QMM_ERR_LAYOUT, "kv_append: negative stride");
    if ((k_token_stride | k_head_stride | v_token_stride | v_head_stride) % 8)
      return report(QMM_ERR_ALIGN, "kv_append: strides must be multiples of 8 elements");
    if (tokens == 0) return report(QMM_OK, "");
    if (!k || !v || !slots) return report(QMM_ERR_NULL, "kv_append: k, v and slots must be non-NULL");
    if ((uintptr_t)k % 16 || (uintptr_t)v % 16 || (uintptr_t)slots % 4)
      return report(QMM_ERR_ALIGN, "kv_append: k and v must be 16-byte, slots 4-byte aligned");
    a.x[0] = k;
    a.x[1] = v;
    a.token_stride[0] = k_token_stride;
    a.token_stride[1] = v_token_stride;
    a.head_stride[0] = k_head_stride;
    a.head_stride[1] = v_head_stride;
    a.tokens = tokens;
    a.slots = slots;
    return report_launch(kv::launch_append(a, (hipStream_t)stream));
  });
}

int32_t qmm_kv_read(const qmm_kv_cache_t* cache, const int32_t* slots, int64_t count, void* k, void* v,
                    void* stream) {
  return guarded([&]() -> int32_t {
    kv::ReadArgs a{};
    const int32_t rc = kv::check_cache(cache, count > 0, &a.c);
    if (rc != QMM_OK) return rc;
    if (count < 0 || count > kv::kMaxInt) return report(QMM_ERR_SHAPE, "kv_read: need 0 <= count < 2^31");
    if (kv::copy_blocks(a.c, count) > kv::kMaxCopyBlocks)
      return report(QMM_ERR_SHAPE, "kv_read: count * heads * head_dim must be below 2^34");
    if (count == 0) return report(QMM_OK, "");
    if (!k || !v || !slots) return report(QMM_ERR_NULL, "kv_read: k, v and slots must be non-NULL");
    if ((uintptr_t)k % 16 || (uintptr_t)v % 16 || (uintptr_t)slots % 4)
      return report(QMM_ERR_ALIGN, "kv_read: k and v must be 16-byte, slots 4-byte aligned");
    a.out[0] = k;
    a.out[1] = v;
    a.count = count;
    a.slots = slots;
    return report_launch(kv::launch_read(a, (hipStream_t)stream));
  });
}

int64_t qmm_kv_attend_workspace_bytes(const qmm_kv_cache_t* cache, const qmm_kv_attend_t* args) {
  return guarded([&]() -> int64_t {
    kv::AttendArgs a{};
    const int32_t rc = kv::check_attend(cache, args, false, &a);
    if (rc != QMM_OK) return rc;
    report(QMM_OK, "");
    return kv::part_floats(a, kv::most_splits(a, false)) * 4;
  });
}

int32_t qmm_kv_attend(const qmm_kv_cache_t* cache, const qmm_kv_attend_t* args, void* out, void* workspace,
                      int64_t workspace_bytes, void* stream) {
  return guarded([&]() -> int32_t {
    kv::AttendArgs a{};
    const bool empty = args && (args->batch == 0 || args->q_len == 0);
    const int32_t rc = kv::check_attend(cache, args, !empty, &a);
    if (rc != QMM_OK) return rc;
    if (empty) return report(QMM_OK, "");
    return kv::run_attend(a, out, workspace, workspace_bytes, (hipStream_t)stream);
  });
}

int64_t qmm_kv_attend_tree_workspace_bytes(const qmm_kv_cache_t* cache, const qmm_kv_attend_t* args) {
  return guarded([&]() -> int64_t {
    kv::AttendArgs a{};
    const int32_t rc = kv::check_tree(cache, args, false, &a);
    if (rc != QMM_OK) return rc;
    report(QMM_OK, "");
    return kv::part_floats(a, kv::most_splits(a, true)) * 4;
  });
}

int32_t qmm_kv_attend_tree(const qmm_kv_cache_t* cache, const qmm_kv_attend_t* args, const uint32_t* mask,
                           const int32_t* depth, void* out, void* workspace, int64_t workspace_bytes, void* stream) {
  return guarded([&]() -> int32_t {
    kv::AttendArgs a{};
    const bool empty = args && (args->batch == 0 || args->q_len == 0);
    const int32_t rc = kv::check_tree(cache, args, !empty, &a);
    if (rc != QMM_OK) return rc;
    if (empty) return report(QMM_OK, "");
    if (!mask || (a.window && !depth))
      return report(QMM_ERR_NULL, "kv_attend_tree: mask, and depth with a window, must be non-NULL");
    if ((uintptr_t)mask % 4 || (uintptr_t)depth % 4)
      return report(QMM_ERR_ALIGN, "kv_attend_tree: mask and depth must be 4-byte aligned");
    a.mask = mask;
    a.mask_words = (a.q_len + 31) / 32;
    a.depth = depth;
    return kv::run_attend(a, out, workspace, workspace_bytes, (hipStream_t)stream);
  });
}

}  // extern "C"
