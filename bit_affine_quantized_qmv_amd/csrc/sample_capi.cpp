// extern "C" entry point of sampling: validate, launch.
#include <hip/hip_runtime.h>

#include <string>

#include "capi_internal.hpp"
#include "sample.hpp"

using namespace qmm;

static_assert(sizeof(sampling::RowSpace) == QMM_SAMPLE_WORKSPACE_BYTES(1), "workspace of one row");

extern "C" int32_t qmm_sample(const void* logits, int32_t dtype, int64_t rows, int64_t n, int64_t row_stride,
                              const qmm_sample_params_t* params, const float* u, int32_t* out_index,
                              float* out_prob, void* workspace, void* stream) {
  return guarded([&]() -> int32_t {
    if (dtype != QMM_BF16 && dtype != QMM_FP16)
      return report(QMM_ERR_UNSUPPORTED, "sample: dtype must be QMM_BF16 or QMM_FP16");
    if (rows < 0 || rows > 65535) return report(QMM_ERR_SHAPE, "sample: need 0 <= rows <= 65535");
    if (n <= 0 || n > QMM_SAMPLE_MAX_N) return report(QMM_ERR_SHAPE, "sample: need 0 < n <= QMM_SAMPLE_MAX_N");
    if (row_stride < n) return report(QMM_ERR_SHAPE, "sample: row_stride < n");
    if (!params) return report(QMM_ERR_NULL, "sample: params must be non-NULL");
    if (rows == 0) return report(QMM_OK, "");
    if (!logits || !u || !out_index || !workspace)
      return report(QMM_ERR_NULL, "sample: logits, u, out_index and workspace must be non-NULL");
    if ((uintptr_t)logits % 2 || (uintptr_t)u % 4 || (uintptr_t)out_index % 4 || (uintptr_t)out_prob % 4 ||
        (uintptr_t)workspace % 8)
      return report(QMM_ERR_ALIGN,
                    "sample: logits must be 2-byte, u and the outputs 4-byte, workspace 8-byte aligned");
    if ((uintptr_t)params->temperature % 4 || (uintptr_t)params->top_k % 4 || (uintptr_t)params->top_p % 4 ||
        (uintptr_t)params->min_p % 4)
      return report(QMM_ERR_ALIGN, "sample: the settings' arrays must be 4-byte aligned");
    sampling::SampleArgs a{};
    a.logits = logits;
    a.rows = rows;
    a.n = n;
    a.row_stride = row_stride;
    a.dtype = dtype;
    a.u = u;
    a.temperature = {params->temperature, params->temperature_all};
    a.top_k = {params->top_k, params->top_k_all};
    a.top_p = {params->top_p, params->top_p_all};
    a.min_p = {params->min_p, params->min_p_all};
    a.out_index = out_index;
    a.out_prob = out_prob;
    a.space = (sampling::RowSpace*)workspace;
    return report_launch(sampling::launch_sample(a, (hipStream_t)stream));
  });
}
