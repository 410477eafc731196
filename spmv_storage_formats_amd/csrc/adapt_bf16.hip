// Adapter kernels for bf16 rows and matrices (adapt.h).
#define SPMV_ADAPT_KERNELS
#include "adapt.h"

namespace spmv {
template struct Adapt<bf16>;
}  // namespace spmv
