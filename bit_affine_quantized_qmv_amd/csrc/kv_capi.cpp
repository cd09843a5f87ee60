// extern "C" entry points of the 4-bit key/value cache: validate, plan, launch.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <string>

#include "capi_internal.hpp"
#include "kv_cache.hpp"

namespace qmm {
namespace kv {
namespace {

constexpr int64_t kMaxInt = 0x7FFFFFFF;

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
namespace {

struct Shape {
  int32_t by_rows, row_tiles;
  int64_t step, want;
};

Shape shape_of(int64_t batch, int heads, int head_dim, int group, int64_t rows) {
  Shape s{};
  s.by_rows = rows >= (head_dim == 128 ? 256 : 1024);
  const int64_t wg_rows = s.by_rows ? (head_dim == 256 ? 128 : 256) : 16;
  s.row_tiles = (int32_t)((rows + wg_rows - 1) / wg_rows);
  s.step = s.by_rows ? 512 : 128;
  const int64_t per_cu = s.by_rows || head_dim == 256 ? 1 : (head_dim == 4 * group ? 2 : 4);
  s.want = std::max<int64_t>(1, 256 * per_cu / std::max<int64_t>(1, batch * heads * s.row_tiles));
  return s;
}

}  // namespace

AttendPlan plan_attend(int64_t batch, const CacheArgs& c, int64_t rows, int64_t range) {
  const Shape s = shape_of(batch, c.heads, c.head_dim, c.group_size, rows);
  const int64_t steps = std::max<int64_t>(1, (range + s.step - 1) / s.step);
  const int64_t per = std::max<int64_t>(1, (steps + s.want - 1) / s.want);
  return AttendPlan{s.by_rows, s.row_tiles, (int32_t)(per * s.step), (int32_t)((steps + per - 1) / per)};
}

// Splits that no shorter range of the same call exceeds.
static int64_t most_splits(const AttendArgs& a) {
  const Shape s = shape_of(a.batch, a.c.heads, a.c.head_dim, a.c.group_size, a.rows);
  return std::min<int64_t>(s.want, std::max<int64_t>(1, (a.max_length + s.step - 1) / s.step));
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
    return kv::part_floats(a, kv::most_splits(a)) * 4;
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
    if (!a.q || !out || !a.lengths || (a.max_length > 0 && !a.table))
      return report(QMM_ERR_NULL, "kv_attend: q, out, lengths and block_table must be non-NULL");
    if ((uintptr_t)a.q % 16 || (uintptr_t)out % 16 || (uintptr_t)workspace % 16)
      return report(QMM_ERR_ALIGN, "kv_attend: q, out and workspace must be 16-byte aligned");
    if ((uintptr_t)a.table % 4 || (uintptr_t)a.lengths % 4)
      return report(QMM_ERR_ALIGN, "kv_attend: block_table and lengths must be 4-byte aligned");
    const kv::AttendPlan p =
        kv::plan_attend(a.batch, a.c, a.rows, kv::token_range(a));
    if ((int64_t)a.c.heads * p.row_tiles > 65535)
      return report(QMM_ERR_SHAPE, "kv_attend: too many query rows per sequence");
    const int64_t need = kv::part_floats(a, p.splits) * 4;
    if (need > 0 && !workspace) return report(QMM_ERR_NULL, "kv_attend: workspace must be non-NULL");
    if (workspace_bytes < need)
      return report(QMM_ERR_SHAPE, "kv_attend: workspace of " + std::to_string(workspace_bytes) + " bytes, needs " +
                                       std::to_string(need));
    a.page_recip = kv::page_recip(a.c.page_size);
    a.chunk = p.chunk;
    a.splits = p.splits;
    a.out = out;
    a.part = (float*)workspace;
    hipStream_t s = (hipStream_t)stream;
    return report_launch(a.c.dtype == QMM_BF16 ? kv::launch_attend_bf16(a, p, s) : kv::launch_attend_fp16(a, p, s));
  });
}

}  // extern "C"
