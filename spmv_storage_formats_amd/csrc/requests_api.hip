// C ABI of the operators on a step's rows (include/spmv.h): argument checks.
#include <cmath>

#include "requests.h"

using namespace spmv;

namespace {

bool aligned(const void *p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

}  // namespace

extern "C" {

spmv_status spmv_token_logprobs_workspace(int32_t V, int64_t n, int32_t top, size_t *bytes) {
    if (!bytes || V < 0 || n < 0 || top < 0 || top > kMostTop) return SPMV_ERR_INVALID_ARG;
    if (V > kMostVocab || n > kMostRows) return SPMV_ERR_TOO_LARGE;
    *bytes = logprobs_bytes(V, n, top);
    return SPMV_OK;
}

spmv_status spmv_token_logprobs(int32_t V, int64_t n, const void *logits, int64_t ld,
                                spmv_dtype dtype, const void *ids, spmv_dtype id_dtype,
                                float scale, int32_t top, float *logprobs_out, float *entropy,
                                float *stats, void *top_ids, float *top_logprobs,
                                void *workspace, size_t workspace_bytes, void *stream) {
    if (V < 0 || n < 0 || top < 0 || top > kMostTop || !float_dtype(dtype) ||
        !id_dtype_ok(id_dtype) || !(scale > 0.f) || !std::isfinite(scale))
        return SPMV_ERR_INVALID_ARG;
    if (V > kMostVocab || n > kMostRows) return SPMV_ERR_TOO_LARGE;
    if (n == 0) return SPMV_OK;
    if ((V > 0 && !logits) || (n > 1 && ld < V) || !ids || !logprobs_out ||
        (top > 0 && (!top_ids || !top_logprobs)))
        return SPMV_ERR_INVALID_ARG;
    const size_t need = logprobs_bytes(V, n, top);
    if (need > 0 && (!workspace || workspace_bytes < need || !aligned(workspace, 16)))
        return SPMV_ERR_INVALID_ARG;
    return logprobs({V, n, logits, ld, dtype, ids, id_dtype, scale, top, logprobs_out, entropy,
                     stats, top_ids, top_logprobs, workspace},
                    static_cast<hipStream_t>(stream));
}

spmv_status spmv_token_logprobs_grad(int32_t V, int64_t n, const void *logits, int64_t ld,
                                     spmv_dtype dtype, const void *ids, spmv_dtype id_dtype,
                                     float scale, const float *stats, const float *grad_logprobs,
                                     const float *entropy, const float *grad_entropy, void *out,
                                     int64_t out_ld, spmv_dtype out_dtype, void *stream) {
    if (V < 0 || n < 0 || !float_dtype(dtype) || !id_dtype_ok(id_dtype) || !(scale > 0.f) ||
        !std::isfinite(scale) || (out_dtype != dtype && out_dtype != SPMV_FP32))
        return SPMV_ERR_INVALID_ARG;
    if (V > kMostVocab || n > kMostRows) return SPMV_ERR_TOO_LARGE;
    if (n == 0 || V == 0) return SPMV_OK;
    if (!logits || !out || (n > 1 && (ld < V || out_ld < V)) || !ids || !stats ||
        (grad_entropy && !entropy) ||
        (out == logits && (out_dtype != dtype || (n > 1 && out_ld != ld))))
        return SPMV_ERR_INVALID_ARG;
    return logprobs_grad({V, n, logits, ld, dtype, ids, id_dtype, scale, stats, grad_logprobs,
                          entropy, grad_entropy, out, out_ld, out_dtype},
                         static_cast<hipStream_t>(stream));
}

}  // extern "C"
