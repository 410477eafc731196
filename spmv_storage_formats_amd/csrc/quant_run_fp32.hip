// 4-bit products of fp32 vectors, and the entry to all of them.
#include "quant_product.h"

namespace spmv {

void quant_run_fp32(const QuantArgs &a, int32_t scale_dtype, hipStream_t s) {
    launch_product<float>(a, scale_dtype, s);
}

namespace {

// Parts of the columns of a wide product: enough for four workgroups per CU, of
// eight blocks at least, at most eight (their sums are written and read once
// more).  us per call, join included, by the number of parts:
//                              1     2     4     8    16    rule
//   1024 x 8192    bf16, 48   53.4  31.4  20.1  15.1  14.1  8   vectors
//   4096 x 4096    bf16, 48   29.3  19.7  14.5  13.3  15.7  4
//   8192 x 8192    bf16, 20   47.4  29.5  20.0  18.1  21.7  8
//   8192 x 11000   bf16, 48   73.7  44.8  30.8  31.2  36.2  8
//   16384 x 4096   bf16, 48   30.8  24.3  24.8  30.3  38.8  4
//   28672 x 8192   bf16, 64   70.0  73.8  76.1  94.2   110  3
//                  fp32, 16   70.2  56.8  54.5  52.2  61.1  5
// Of 24 such cases (20, 48 and 64 bf16 and 16 fp32 vectors over the six matrices)
// the rule is within 8 % of the best count in 21, and 9, 12 and 15 % from it at
// 4096 x 4096, whose 32 blocks would rather be cut in eight parts of four.
int32_t column_splits(const spmv_quant *q, int32_t n, int32_t x_dtype) {
    const int parts = x_dtype == SPMV_FP32 ? Unit<float>::kParts : 1;
    const int64_t cols = wide_columns(n, parts);
    if (cols <= 16) return 1;
    const int64_t passes = (static_cast<int64_t>(n) * parts + cols - 1) / cols;
    const int64_t groups = (static_cast<int64_t>(q->R) + kWideRows - 1) / kWideRows * passes;
    const int64_t want = (1024 + groups - 1) / groups;
    return static_cast<int32_t>(std::max<int64_t>(
        1, std::min<int64_t>({want, int64_t{8}, static_cast<int64_t>(q->blocks / 8)})));
}

}  // namespace

size_t quant_run_bytes(const spmv_quant *q, int32_t n, int32_t x_dtype) {
    const int32_t splits = column_splits(q, n, x_dtype);
    return splits > 1 ? static_cast<size_t>(splits) * static_cast<size_t>(n) *
                            static_cast<size_t>(q->R) * sizeof(float)
                      : 0;
}

spmv_status quant_run(const spmv_quant *q, int32_t n, const void *x, int64_t x_ld,
                      int32_t x_dtype, void *y, int64_t y_ld, int32_t y_dtype, int accumulate,
                      void *workspace, hipStream_t s) {
    QuantArgs a{};
    a.R = q->R;
    a.C = q->C;
    a.n = n;
    a.blocks = q->blocks;
    a.group = q->group;
    a.set = q->set;
    a.sets = q->sets;
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
    a.splits = column_splits(q, n, x_dtype);
    a.partial = static_cast<float *>(workspace);
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
