// 4-bit products of fp16 vectors.
#include "quant_product.h"

namespace spmv {

void quant_run_fp16(const QuantArgs &a, int32_t scale_dtype, hipStream_t s) {
    launch_product<f16>(a, scale_dtype, s);
}

}  // namespace spmv
