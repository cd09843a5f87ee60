// extern "C" entry points of the products grouped by expert: validate, plan, launch.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <string>

#include "capi_internal.hpp"
#include "dispatch.hpp"
#include "grouped.hpp"

namespace qmm {
namespace grouped {
namespace {

int64_t align256(int64_t v) { return (v + 255) / 256 * 256; }
int64_t round_up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }

// Rows per tile.  Taller ones unpack a code for more rows, lower ones leave more workgroups per CU (four
// of 16 rows, three of 32, two of 64) and less of a tile empty.  Measured, 32 rows against 64, us for
// the product of 64 experts of [1024, 2048] in 4 bits: 24 rows per expert 30 / 40, 64 rows 41 / 43, 96
// rows 55 / 47, 160 rows 78 / 70; the layer of 64 experts of [704, 1408] in 8 bits: 24 rows 74 / 80, 64
// rows 120 / 136, 96 rows 149 / 141.  16 rows against 32, the gated product of 8 experts of [14336, 4096]:
// 2 rows per expert 137 / 152, 8 rows 150 / 153, 16 rows 175 / 156; of 128 experts of [704, 1408]: 3
// rows 32 / 35, 6 rows 34 / 36, 12 rows 39 / 38.
int tile_rows_of(int64_t rows, int64_t experts) {
  return rows >= 80 * experts ? 64 : (rows <= 8 * experts ? 16 : 32);
}
// Workgroups of tiles of so many rows that the chip holds.
int64_t slots_of(int tile_rows) { return tile_rows == 16 ? 1024 : (tile_rows == 32 ? 768 : 512); }
// Tiles at most: a part of a tile for each expert with rows.
int64_t max_tiles_of(int64_t rows, int64_t experts) {
  return rows / 16 + std::min(rows, experts);
}

int64_t sum_groups_of(int64_t k, int64_t group) { return round_up(k / group, kSumPad); }
// Splits of the second product's columns, of whole runs of groups: what leaves the chip's workgroup slots
// idle least.  `tiles` times `blocks` workgroups take whole rounds of the slots, and a split more costs its
// results' way through memory, about what 1024 columns of the product do.  (8 experts of [4096, 14336], one
// piece against the choice, product and sum: 2 tokens 183 us / 80, 512 348 / 264, 1024 550 / 487, 2047 967 /
// 875.)
struct Splits {
  int64_t count, cols;
};
constexpr int64_t kSplitRounds = 5;            // rounds of the slots that splits may fill
Splits splits_of(int64_t tiles, int64_t blocks, int tile_rows, int64_t k, int64_t group) {
  const int64_t run = kSplitGroups * group, runs = (k + run - 1) / run, slots = slots_of(tile_rows), all = tiles * blocks;
  Splits best{1, k};
  double least = 0.0;
  for (int64_t want = 1; want <= runs && (want == 1 || want * all <= kSplitRounds * slots); ++want) {
    const int64_t per = (runs + want - 1) / want, count = (runs + per - 1) / per;
    if (count != want) continue;
    const double cost = (double)((count * all + slots - 1) / slots * per) / runs + 1024.0 * count * all / ((double)slots * k);
    if (want == 1 || cost < least) {
      least = cost;
      if (want > 1) best = Splits{count, per * run};
    }
  }
  return best;
}
// Bytes of their results, [split][pair][n], at most: several splits have no more rows and columns than the
// tiles of those rounds.
int64_t out_bytes(int64_t pairs, int64_t n, int64_t k) {
  const int64_t runs = (k + kSplitGroups * 32 - 1) / (kSplitGroups * 32);
  return align256(4 * std::max(pairs * n, std::min(runs * pairs * n, kSplitRounds * 512 * 64 * kBlockN)));
}
// Bytes of the staged activations, and of the sums of `rows` rows, whatever the group size.
int64_t staged_bytes(int64_t rows, int64_t k) { return align256(2 * rows * round_up(k, kStepK)); }
int64_t sums_bytes(int64_t rows, int64_t k) { return align256(rows * kPlanes * 2 * round_up((k + 31) / 32, kSumPad)); }
int64_t tiles_bytes(int64_t rows, int64_t experts) {
  return align256(16) + align256(max_tiles_of(rows, experts) * (int64_t)sizeof(Tile));
}

hipError_t launch(const Args& a, Kind kind, int dtype, int tile_rows, hipStream_t s) {
  const int bits = a.w[0].bits;
  return bits == 4 ? launch_b4(a, kind, dtype, tile_rows, s)
                   : (bits == 8 ? launch_b8(a, kind, dtype, tile_rows, s) : launch_bn(a, kind, dtype, tile_rows, s));
}

// The kernels address a workgroup's weight rows, up to kBlockN past the last, with 32-bit byte offsets:
// moe::check_stack keeps N + 128 rows below 2^30 bytes, so N + 256 stay below 2^31.
static_assert(kBlockN <= 256, "rows past the last");

int32_t check_grouped(int64_t rows, const qmm_expert_stack_t* w, bool pointers, Stack* out) {
  if (!w) return report(QMM_ERR_NULL, "grouped: weights must be non-NULL");
  if (rows < 0 || rows > kMaxPairs) return report(QMM_ERR_SHAPE, "grouped: need 0 <= rows <= 2^20");
  if (w->num_experts < 1 || w->num_experts > moe::kMaxExperts)
    return report(QMM_ERR_SHAPE, "grouped: need 1 <= experts <= 512");
  if (w->w.N < 1 || w->w.N > (1 << 20) || w->w.K < 1 || w->w.K > (1 << 20))
    return report(QMM_ERR_SHAPE, "grouped: need 1 <= N, K <= 2^20");
  if (!pointers) return QMM_OK;
  return moe::check_stack("grouped", w, w->w.N, w->w.K, (int32_t)w->num_experts, w->w.dtype, out);
}

int32_t check_sizes(int64_t tokens, int64_t experts, int64_t top_k, int64_t hidden, int64_t inter) {
  if (tokens < 0 || tokens > 65535) return report(QMM_ERR_SHAPE, "moe_prompt: need 0 <= tokens <= 65535");
  if (experts < 1 || experts > moe::kMaxExperts) return report(QMM_ERR_SHAPE, "moe_prompt: need 1 <= experts <= 512");
  if (top_k < 1 || top_k > moe::kMaxTopK || top_k > experts)
    return report(QMM_ERR_SHAPE, "moe_prompt: need 1 <= top_k <= min(experts, 32)");
  if (tokens * top_k > kMaxPairs) return report(QMM_ERR_SHAPE, "moe_prompt: tokens * top_k must be at most 2^20");
  if (hidden < 1 || hidden > (1 << 20) || inter < 1 || inter > (1 << 20))
    return report(QMM_ERR_SHAPE, "moe_prompt: need 1 <= hidden, inter <= 2^20");
  return QMM_OK;
}

// Workspace of the layer, in this order.
struct LayerBytes {
  int64_t expert, share, pairs, tiles, staged, sums, h, h_sums, out;
  int64_t all() const { return expert + share + pairs + tiles + staged + sums + h + h_sums + out; }
};
LayerBytes layer_bytes(int64_t tokens, int64_t experts, int64_t top_k, int64_t hidden, int64_t inter) {
  const int64_t n = tokens * top_k, cols = round_up(inter, kStepK);
  return LayerBytes{align256(4 * n),
                    align256(4 * n),
                    align256(4 * n),
                    tiles_bytes(n, experts),
                    staged_bytes(tokens, hidden),
                    sums_bytes(tokens, hidden),
                    align256(4 * n * cols),
                    sums_bytes(n, cols),
                    out_bytes(n, hidden, inter)};
}

}  // namespace
}  // namespace grouped
}  // namespace qmm

using namespace qmm;

extern "C" {

int64_t qmm_grouped_workspace_bytes(int64_t rows, const qmm_expert_stack_t* w) {
  return guarded([&]() -> int64_t {
    const int32_t rc = grouped::check_grouped(rows, w, false, nullptr);
    if (rc != QMM_OK) return rc;
    report(QMM_OK, "");
    return grouped::tiles_bytes(rows, w->num_experts) + grouped::sums_bytes(rows, w->w.K) +
           grouped::staged_bytes(rows, w->w.K);
  });
}

int32_t qmm_grouped(const void* x, int64_t x_stride, int64_t rows, const qmm_expert_stack_t* weights,
                    const int32_t* offsets, void* y, int64_t y_stride, void* workspace, int64_t workspace_bytes,
                    void* stream) {
  return guarded([&]() -> int32_t {
    grouped::Args a{};
    const int32_t rc = grouped::check_grouped(rows, weights, true, &a.w[0]);
    if (rc != QMM_OK) return rc;
    const int64_t n = weights->w.N, k = weights->w.K;
    if (x_stride < 0 || y_stride < 0) return report(QMM_ERR_LAYOUT, "grouped: negative stride");
    if (x_stride % 8) return report(QMM_ERR_ALIGN, "grouped: x_stride must be a multiple of 8 elements");
    if (rows > 1 && y_stride < n) return report(QMM_ERR_SHAPE, "grouped: y_stride < N");
    if (rows == 0) return report(QMM_OK, "");
    if (!x || !offsets || !y || !workspace)
      return report(QMM_ERR_NULL, "grouped: x, offsets, y and workspace must be non-NULL");
    if ((uintptr_t)x % 16 || (uintptr_t)workspace % 16 || (uintptr_t)offsets % 4 || (uintptr_t)y % 2)
      return report(QMM_ERR_ALIGN, "grouped: x and workspace must be 16-byte, offsets 4-byte, y 2-byte aligned");
    const int64_t experts = weights->num_experts;
    const int64_t tiles_bytes = grouped::tiles_bytes(rows, experts), sums_bytes = grouped::sums_bytes(rows, k);
    const int64_t need = tiles_bytes + sums_bytes + grouped::staged_bytes(rows, k);
    if (workspace_bytes < need)
      return report(QMM_ERR_SHAPE, "grouped: workspace of " + std::to_string(workspace_bytes) + " bytes, needs " +
                                       std::to_string(need));
    const int tile_rows = grouped::tile_rows_of(rows, experts);
    char* ws = (char*)workspace;
    grouped::PrepareArgs p{};
    p.x = (const uint16_t*)x;
    p.x_stride = x_stride;
    p.rows = rows;
    p.k = (int32_t)k;
    p.group = weights->w.group_size;
    p.dtype = weights->w.dtype;
    p.bits = weights->w.bits;
    p.cols = (int32_t)grouped::round_up(k, grouped::kStepK);
    p.sums = (uint16_t*)(ws + tiles_bytes);
    p.staged = (uint16_t*)(ws + tiles_bytes + sums_bytes);
    p.sum_groups = (int32_t)grouped::sum_groups_of(k, p.group);
    p.experts = (int32_t)experts;
    p.offsets = offsets;
    p.tile_rows = tile_rows;
    p.tile_count = (int32_t*)ws;
    p.tiles = (grouped::Tile*)(ws + grouped::align256(16));
    p.max_tiles = (int32_t)(rows / tile_rows + std::min(rows, experts));
    a.w[1] = a.w[0];
    a.x = p.staged;
    a.x_stride = p.cols;
    a.sums = p.sums;
    a.sum_groups = p.sum_groups;
    a.n = (int32_t)n;
    a.k = (int32_t)k;
    a.tiles = p.tiles;
    a.tile_count = p.tile_count;
    a.max_tiles = p.max_tiles;
    a.n_blocks = (int32_t)((n + grouped::kBlockN - 1) / grouped::kBlockN);
    a.y = (uint16_t*)y;
    a.y_stride = y_stride;
    if (grouped::prepare_blocks(p) * grouped::kMake >= grouped::kLaunchThreads)
      return report(QMM_ERR_SHAPE, "grouped: rows * K too large for one call (up to 2^35 - 2^15, K rounded up to 4096, always fits)");
    if (grouped::product_blocks(a) * grouped::kThreads >= grouped::kLaunchThreads)
      return report(QMM_ERR_SHAPE, "grouped: rows * N too large for one call");
    hipStream_t s = (hipStream_t)stream;
    hipError_t e = grouped::launch_prepare(p, s);
    if (e == hipSuccess) e = grouped::launch(a, grouped::kPlain, p.dtype, tile_rows, s);
    return report_launch(e);
  });
}

int64_t qmm_moe_prompt_workspace_bytes(int64_t tokens, int64_t experts, int64_t top_k, int64_t hidden, int64_t inter) {
  return guarded([&]() -> int64_t {
    const int32_t rc = grouped::check_sizes(tokens, experts, top_k, hidden, inter);
    if (rc != QMM_OK) return rc;
    report(QMM_OK, "");
    return grouped::layer_bytes(tokens, experts, top_k, hidden, inter).all();
  });
}

int32_t qmm_moe_prompt(const qmm_moe_t* m, void* y, void* workspace, int64_t workspace_bytes, void* stream) {
  return guarded([&]() -> int32_t {
    if (!m) return report(QMM_ERR_NULL, "moe_prompt: args must be non-NULL");
    if (m->dtype != QMM_BF16 && m->dtype != QMM_FP16)
      return report(QMM_ERR_UNSUPPORTED, "moe_prompt: dtype must be QMM_BF16 or QMM_FP16");
    if (!m->gate || !m->up || !m->down) return report(QMM_ERR_NULL, "moe_prompt: gate, up and down must be non-NULL");
    const int64_t hidden = m->gate->w.K, inter = m->gate->w.N, experts = m->gate->num_experts;
    int32_t rc = grouped::check_sizes(m->tokens, experts, m->top_k, hidden, inter);
    if (rc != QMM_OK) return rc;
    grouped::Stack gate, up, down;
    rc = moe::check_stack("moe_prompt: gate", m->gate, inter, hidden, (int32_t)experts, m->dtype, &gate);
    if (rc == QMM_OK) rc = moe::check_stack("moe_prompt: up", m->up, inter, hidden, (int32_t)experts, m->dtype, &up);
    if (rc == QMM_OK) rc = moe::check_stack("moe_prompt: down", m->down, hidden, inter, (int32_t)experts, m->dtype, &down);
    if (rc != QMM_OK) return rc;
    if (up.bits != gate.bits || up.group_size != gate.group_size)
      return report(QMM_ERR_UNSUPPORTED, "moe_prompt: gate and up must share bits and group_size");
    if (m->x_stride < 0 || m->router_stride < 0 || m->y_stride < 0)
      return report(QMM_ERR_LAYOUT, "moe_prompt: negative stride");
    if (m->x_stride % 8) return report(QMM_ERR_ALIGN, "moe_prompt: x_stride must be a multiple of 8 elements");
    if (m->tokens > 1 && m->y_stride < hidden) return report(QMM_ERR_SHAPE, "moe_prompt: y_stride < hidden");
    if (m->tokens == 0) return report(QMM_OK, "");
    const int64_t x_bytes = 2 * m->tokens * grouped::round_up(hidden, grouped::kStepK);   // as staged
    if (x_bytes >= (1ll << 30)) return report(QMM_ERR_SHAPE, "moe_prompt: tokens * hidden must be below 2^29");
    if (!m->x || !m->router_logits || !y || !workspace)
      return report(QMM_ERR_NULL, "moe_prompt: x, router_logits, y and workspace must be non-NULL");
    if ((uintptr_t)m->x % 16 || (uintptr_t)m->router_logits % 2 || (uintptr_t)y % 2 || (uintptr_t)workspace % 16)
      return report(QMM_ERR_ALIGN, "moe_prompt: x and workspace must be 16-byte, router_logits and y 2-byte aligned");
    const int64_t n = m->tokens * m->top_k;
    const grouped::LayerBytes b = grouped::layer_bytes(m->tokens, experts, m->top_k, hidden, inter);
    if (workspace_bytes < b.all())
      return report(QMM_ERR_SHAPE, "moe_prompt: workspace of " + std::to_string(workspace_bytes) + " bytes, needs " +
                                       std::to_string(b.all()));
    char* ws = (char*)workspace;
    const auto take = [&](int64_t bytes) {
      char* p = ws;
      ws += bytes;
      return p;
    };
    const int tile_rows = grouped::tile_rows_of(n, experts);
    grouped::RouteArgs r{};
    r.router = (const uint16_t*)m->router_logits;
    r.router_stride = m->router_stride;
    r.tokens = (int32_t)m->tokens;
    r.experts = (int32_t)experts;
    r.top_k = m->top_k;
    r.renormalize = m->renormalize != 0;
    r.dtype = m->dtype;
    r.pair_expert = (int32_t*)take(b.expert);
    r.pair_share = (float*)take(b.share);
    r.pairs = (int32_t*)take(b.pairs);
    r.tile_rows = tile_rows;
    char* tiles = take(b.tiles);
    r.tile_count = (int32_t*)tiles;
    r.tiles = (grouped::Tile*)(tiles + grouped::align256(16));
    r.max_tiles = (int32_t)(n / tile_rows + std::min(n, experts));
    grouped::PrepareArgs p{};
    p.x = (const uint16_t*)m->x;
    p.x_stride = m->x_stride;
    p.rows = m->tokens;
    p.k = (int32_t)hidden;
    p.group = gate.group_size;
    p.dtype = m->dtype;
    p.bits = gate.bits;
    p.cols = (int32_t)grouped::round_up(hidden, grouped::kStepK);
    p.staged = (uint16_t*)take(b.staged);
    p.sums = (uint16_t*)take(b.sums);
    p.sum_groups = (int32_t)grouped::sum_groups_of(hidden, p.group);

    grouped::Args g{};
    g.x = p.staged;
    g.x_stride = p.cols;
    g.x_bytes = (uint32_t)x_bytes;
    g.sums = p.sums;
    g.sum_groups = p.sum_groups;
    g.w[0] = gate;
    g.w[1] = up;
    g.n = (int32_t)inter;
    g.k = (int32_t)hidden;
    g.tiles = r.tiles;
    g.tile_count = r.tile_count;
    g.max_tiles = r.max_tiles;
    g.h_cols = (int32_t)grouped::round_up(inter, grouped::kStepK);
    g.n_blocks = g.h_cols / (grouped::kBlockN / 2);
    g.pairs = r.pairs;
    g.top_k = m->top_k;
    g.h = (uint16_t*)take(b.h);
    g.h_sums = (uint16_t*)take(b.h_sums);
    g.h_group = down.group_size;
    g.h_bits = down.bits;
    g.h_sum_groups = (int32_t)grouped::sum_groups_of(g.h_cols, down.group_size);

    grouped::Args d{};
    d.x = g.h;
    d.x_stride = 2 * (int64_t)g.h_cols;
    d.x_plane = g.h_cols;
    d.sums = g.h_sums;
    d.sum_groups = g.h_sum_groups;
    d.w[0] = d.w[1] = down;
    d.n = (int32_t)hidden;
    d.k = (int32_t)inter;
    d.tiles = r.tiles;
    d.tile_count = r.tile_count;
    d.max_tiles = r.max_tiles;
    d.n_blocks = (int32_t)((hidden + grouped::kBlockN - 1) / grouped::kBlockN);
    d.pairs = r.pairs;
    d.top_k = m->top_k;
    d.out = (float*)take(b.out);
    const grouped::Splits split = grouped::splits_of(d.max_tiles, d.n_blocks, tile_rows, inter, down.group_size);
    d.splits = (int32_t)split.count;
    d.split_cols = (int32_t)split.cols;
    d.out_split = n * hidden;
    if (std::max(grouped::product_blocks(g), grouped::product_blocks(d)) * grouped::kThreads >= grouped::kLaunchThreads)
      return report(QMM_ERR_SHAPE, "moe_prompt: tokens * top_k * max(hidden, inter) too large for one call");

    const grouped::SumArgs sum{r.tokens,       m->top_k, r.renormalize, (int32_t)hidden, m->dtype, d.splits, d.out,
                               r.pair_share, (uint16_t*)y, m->y_stride};

    hipStream_t s = (hipStream_t)stream;
    hipError_t e = grouped::launch_route(r, p, s);
    if (e == hipSuccess) e = grouped::launch(g, grouped::kGated, m->dtype, tile_rows, s);
    if (e == hipSuccess) e = grouped::launch(d, grouped::kDown, m->dtype, tile_rows, s);
    if (e == hipSuccess) e = grouped::launch_sum(sum, s);
    return report_launch(e);
  });
}

}  // extern "C"
