// Adapter kernels for fp16 rows and matrices (adapt.h).
#define SPMV_ADAPT_KERNELS
#include "adapt.h"

namespace spmv {
template struct Adapt<f16>;
}  // namespace spmv
