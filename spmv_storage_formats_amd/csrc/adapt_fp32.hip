// Adapter kernels for fp32 rows and matrices (adapt.h).
#define SPMV_ADAPT_KERNELS
#include "adapt.h"

namespace spmv {
template struct Adapt<float>;
}  // namespace spmv
