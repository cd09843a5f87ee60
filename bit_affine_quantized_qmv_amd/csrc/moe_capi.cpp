// extern "C" entry points of the mixture-of-experts layer: validate, plan, launch.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <string>

#include "capi_internal.hpp"
#include "dispatch.hpp"
#include "moe.hpp"

namespace qmm {
namespace moe {
namespace {

static_assert(kMaxTokens == QMM_DECODE_MAX_ROWS && kMaxExperts == QMM_MOE_MAX_EXPERTS &&
                  kMaxTopK == QMM_MOE_MAX_TOP_K,
              "limits of the ABI");

int64_t align256(int64_t v) { return (v + 255) / 256 * 256; }

// Workspace regions, in this order: pair_expert, pair_share, h, out.
int64_t pair_bytes(int64_t tokens, int64_t top_k) { return align256(4 * tokens * top_k); }
int64_t h_bytes(int64_t tokens, int64_t top_k, int64_t inter) { return align256(4 * tokens * top_k * inter); }
int64_t out_bytes(int64_t tokens, int64_t top_k, int64_t hidden, int64_t splits) {
  return align256(4 * tokens * top_k * splits * hidden);
}

// Stretches of inter that different workgroups of the second kernel take: about 6144 columns
// each, of which LDS holds two tokens' operands at once.
int64_t splits_of(int64_t inter) { return std::min<int64_t>(kMaxSplits, (inter + 6143) / 6144); }

int32_t check_stack(const char* name, const qmm_expert_stack_t* k, int64_t n, int64_t cols, int32_t experts,
                    int32_t dtype, Stack* out) {
  const std::string who = std::string("moe: ") + name + ": ";
  if (!k) return report(QMM_ERR_NULL, who + "must be non-NULL");
  const qmm_weight_desc_t& w = k->w;
  std::string err;
  const int rc = check_codec(w.group_size, w.bits, w.dtype, &err);
  if (rc) return report(rc, who + err);
  if (w.dtype != dtype) return report(QMM_ERR_UNSUPPORTED, who + "x and the experts must share one dtype");
  if (w.N != n || w.K != cols)
    return report(QMM_ERR_SHAPE, who + "experts are [" + std::to_string(w.N) + ", " + std::to_string(w.K) +
                                     "], expected [" + std::to_string(n) + ", " + std::to_string(cols) + "]");
  if (cols % w.group_size) return report(QMM_ERR_SHAPE, who + "K is not a multiple of group_size");
  if (k->num_experts != experts) return report(QMM_ERR_SHAPE, who + "the stacks must have the same number of experts");
  if (w.w_row_stride < cols * w.bits / 32 || w.sb_row_stride < cols / w.group_size)
    return report(QMM_ERR_SHAPE, who + "row strides smaller than a row");
  if (k->w_expert_stride < n * w.w_row_stride || k->sb_expert_stride < n * w.sb_row_stride)
    return report(QMM_ERR_SHAPE, who + "expert strides smaller than one expert");
  // rows of one expert, and as many past the last, are addressed with 32-bit byte offsets
  if ((n + 128) * w.w_row_stride * 4 >= (1ll << 30) || (n + 128) * w.sb_row_stride * 2 >= (1ll << 30))
    return report(QMM_ERR_SHAPE, who + "one expert's codes must be smaller than 1 GiB");
  const bool wide = w.bits == 4 || w.bits == 8;   // codes loaded 16 bytes at a time, else word by word
  if (wide && (w.w_row_stride % 4 || k->w_expert_stride % 4))
    return report(QMM_ERR_ALIGN, who + "w_row_stride and w_expert_stride must be multiples of 4 words");
  if (!w.w_packed || !w.scales || !w.biases) return report(QMM_ERR_NULL, who + "pointers must be non-NULL");
  if ((uintptr_t)w.w_packed % (wide ? 16 : 4) || (uintptr_t)w.scales % 2 || (uintptr_t)w.biases % 2)
    return report(QMM_ERR_ALIGN, who + "w_packed must be 16-byte (4-byte unless 4 or 8 bits), scales and biases "
                                       "2-byte aligned");
  *out = Stack{w.w_packed,      w.w_row_stride,       k->w_expert_stride, (const uint16_t*)w.scales,
               (const uint16_t*)w.biases, w.sb_row_stride, k->sb_expert_stride, w.bits, w.group_size};
  return QMM_OK;
}

int32_t check_sizes(int64_t tokens, int64_t experts, int64_t top_k, int64_t hidden, int64_t inter) {
  if (tokens < 0 || tokens > kMaxTokens)
    return report(QMM_ERR_SHAPE, "moe: " + std::to_string(tokens) + " tokens, at most " + std::to_string(kMaxTokens));
  if (experts < 1 || experts > kMaxExperts) return report(QMM_ERR_SHAPE, "moe: need 1 <= experts <= 512");
  if (top_k < 1 || top_k > kMaxTopK || top_k > experts)
    return report(QMM_ERR_SHAPE, "moe: need 1 <= top_k <= min(experts, 32)");
  if (hidden < 1 || hidden > (1 << 20) || inter < 1 || inter > (1 << 20))
    return report(QMM_ERR_SHAPE, "moe: need 1 <= hidden, inter <= 2^20");
  return QMM_OK;
}

hipError_t launch(const MoeArgs& a, int bits, bool down, hipStream_t s) {
  return bits == 4 ? launch_b4(a, s, down) : (bits == 8 ? launch_b8(a, s, down) : launch_bn(a, s, down));
}

// Slots (spans of K that one round of loads covers) of a row.
int64_t slots_of(int64_t k, int bits, int gs) {
  const int64_t span = bits == 8 && gs == 64 ? 64 : 128;
  return (k + span - 1) / span;
}

}  // namespace
}  // namespace moe
}  // namespace qmm

using namespace qmm;

extern "C" {

int64_t qmm_moe_workspace_bytes(int64_t tokens, int64_t experts, int64_t top_k, int64_t hidden, int64_t inter) {
  return guarded([&]() -> int64_t {
    const int32_t rc = moe::check_sizes(tokens, experts, top_k, hidden, inter);
    if (rc != QMM_OK) return rc;
    report(QMM_OK, "");
    return 2 * moe::pair_bytes(tokens, top_k) + moe::h_bytes(tokens, top_k, inter) + moe::out_bytes(tokens, top_k, hidden, moe::splits_of(inter));
  });
}

int32_t qmm_moe(const qmm_moe_t* m, void* y, void* workspace, int64_t workspace_bytes, void* stream) {
  return guarded([&]() -> int32_t {
    if (!m) return report(QMM_ERR_NULL, "moe: args must be non-NULL");
    if (m->dtype != QMM_BF16 && m->dtype != QMM_FP16)
      return report(QMM_ERR_UNSUPPORTED, "moe: dtype must be QMM_BF16 or QMM_FP16");
    if (!m->gate || !m->up || !m->down) return report(QMM_ERR_NULL, "moe: gate, up and down must be non-NULL");
    const int64_t hidden = m->gate->w.K, inter = m->gate->w.N, experts = m->gate->num_experts;
    int32_t rc = moe::check_sizes(m->tokens, experts, m->top_k, hidden, inter);
    if (rc != QMM_OK) return rc;
    moe::MoeArgs a{};
    rc = moe::check_stack("gate", m->gate, inter, hidden, (int32_t)experts, m->dtype, &a.gate);
    if (rc == QMM_OK) rc = moe::check_stack("up", m->up, inter, hidden, (int32_t)experts, m->dtype, &a.up);
    if (rc == QMM_OK) rc = moe::check_stack("down", m->down, hidden, inter, (int32_t)experts, m->dtype, &a.down);
    if (rc != QMM_OK) return rc;
    if (a.up.bits != a.gate.bits || a.up.group_size != a.gate.group_size)
      return report(QMM_ERR_UNSUPPORTED, "moe: gate and up must share bits and group_size");
    if (m->x_stride < 0 || m->router_stride < 0 || m->y_stride < 0)
      return report(QMM_ERR_LAYOUT, "moe: negative stride");
    if (m->x_stride % 8) return report(QMM_ERR_ALIGN, "moe: x_stride must be a multiple of 8 elements");
    if (m->tokens > 1 && m->y_stride < hidden) return report(QMM_ERR_SHAPE, "moe: y_stride < hidden");
    if (m->tokens == 0) return report(QMM_OK, "");
    if (!m->x || !m->router_logits || !y || !workspace)
      return report(QMM_ERR_NULL, "moe: x, router_logits, y and workspace must be non-NULL");
    if ((uintptr_t)m->x % 16 || (uintptr_t)m->router_logits % 2 || (uintptr_t)y % 2 || (uintptr_t)workspace % 16)
      return report(QMM_ERR_ALIGN, "moe: x and workspace must be 16-byte, router_logits and y 2-byte aligned");
    a.x = (const uint16_t*)m->x;
    a.x_stride = m->x_stride;
    a.router = (const uint16_t*)m->router_logits;
    a.router_stride = m->router_stride;
    a.tokens = (int32_t)m->tokens;
    a.experts = (int32_t)experts;
    a.top_k = m->top_k;
    a.renormalize = m->renormalize != 0;
    a.hidden = (int32_t)hidden;
    a.inter = (int32_t)inter;
    a.dtype = m->dtype;
    a.y = (uint16_t*)y;
    a.y_stride = m->y_stride;
    const int64_t need = 2 * moe::pair_bytes(m->tokens, m->top_k) + moe::h_bytes(m->tokens, m->top_k, inter) +
                         moe::out_bytes(m->tokens, m->top_k, hidden, moe::splits_of(inter));
    if (workspace_bytes < need)
      return report(QMM_ERR_SHAPE, "moe: workspace of " + std::to_string(workspace_bytes) + " bytes, needs " +
                                       std::to_string(need));
    char* ws = (char*)workspace;
    a.pair_expert = (int32_t*)ws;
    ws += moe::pair_bytes(m->tokens, m->top_k);
    a.pair_share = (float*)ws;
    ws += moe::pair_bytes(m->tokens, m->top_k);
    a.h = (uint16_t*)ws;
    ws += moe::h_bytes(m->tokens, m->top_k, inter);
    a.out = (float*)ws;

    a.splits = (int32_t)moe::splits_of(inter);
    // Waves per tile: each with at least four slots, so that a wave's ring of loads is in use (one
    // token, 8 experts of 1024 x 2048: 24 us with one wave per tile, 20 with two or four); in the
    // second kernel one where that fills the machine, since its activations pass through LDS in
    // many chunks, each with a barrier (7 tokens, 4096 x 14336: 179 us against 199 with four).
    // Workgroups: three for every compute unit in all, which is what is resident, each with
    // several tiles (that layer: 512 workgroups 220 us, 768 199, 1024 206; 32 tokens over 128
    // experts of 704 x 1408: 108, 104, 128).
    constexpr int64_t kResident = 768;
    const int64_t used = std::min<int64_t>(experts, m->tokens * m->top_k);   // experts in use at most
    const int64_t tiles = (inter + 15) / 16, down_tiles = (hidden + 31) / 32;
    const auto parts = [](int64_t slots) { return slots >= 16 ? 4 : (slots >= 8 ? 2 : 1); };
    const auto blocks = [&](int64_t n, int64_t part, int64_t per_tile) {
      const int64_t units = (n * part + moe::kWaves - 1) / moe::kWaves;
      return (int32_t)std::min(units, std::max<int64_t>(1, kResident / (used * per_tile)));
    };
    a.parts = parts(moe::slots_of(hidden, a.gate.bits, a.gate.group_size));
    a.down_parts = down_tiles * used * a.splits >= kResident * moe::kWaves
                       ? 1
                       : parts(moe::slots_of(inter, a.down.bits, a.down.group_size) / a.splits);
    a.blocks = blocks(tiles, a.parts, 1);
    a.down_blocks = blocks(down_tiles, a.down_parts, a.splits);
    hipStream_t s = (hipStream_t)stream;
    hipError_t e = moe::launch(a, a.gate.bits, false, s);
    if (e == hipSuccess) e = moe::launch(a, a.down.bits, true, s);
    if (e == hipSuccess) e = moe::launch_sum(a, s);
    return report_launch(e);
  });
}

}  // extern "C"
