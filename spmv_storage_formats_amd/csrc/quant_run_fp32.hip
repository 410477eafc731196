// 4-bit products of fp32 vectors, and the entry to all of them.
#include "quant_product.h"

namespace spmv {

void quant_run_fp32(const QuantArgs &a, int32_t scale_dtype, hipStream_t s) {
    launch_product<float>(a, scale_dtype, s);
}

spmv_status quant_run(const spmv_quant *q, int32_t n, const void *x, int64_t x_ld,
                      int32_t x_dtype, void *y, int64_t y_ld, int32_t y_dtype, int accumulate,
                      hipStream_t s) {
    QuantArgs a{};
    a.R = q->R;
    a.C = q->C;
    a.n = n;
    a.blocks = q->blocks;
    a.group = q->group;
    a.groups_pad = q->groups_pad;
    a.group_shift = (q->group & (q->group - 1)) ? -1 : bits_for(q->group) - 1;
    a.codes = q->codes;
    a.scales = q->scales;
    a.zeros = q->zeros;
    a.x = x;
    a.x_ld = x_ld;
    a.y = y;
    a.y_ld = y_ld;
    a.accumulate = accumulate;
    a.y_fp32 = y_dtype == SPMV_FP32;
    if (x_dtype == SPMV_FP32)
        quant_run_fp32(a, q->scale_dtype, s);
    else if (x_dtype == SPMV_FP16)
        quant_run_fp16(a, q->scale_dtype, s);
    else
        quant_run_bf16(a, q->scale_dtype, s);
    SPMV_HIP(hipGetLastError());
    return SPMV_OK;
}

}  // namespace spmv
