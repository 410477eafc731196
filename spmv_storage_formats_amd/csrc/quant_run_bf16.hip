// 4-bit products of bf16 vectors.
#include "quant_product.h"

namespace spmv {

void quant_run_bf16(const QuantArgs &a, int32_t scale_dtype, hipStream_t s) {
    launch_product<bf16>(a, scale_dtype, s);
}

}  // namespace spmv
