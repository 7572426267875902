// scaled_f16.hip -- products of 8-bit matrices with block scales, results of type _Float16.
#include "scaled_kernels.h"

namespace tra {
template struct ScaledKernels<_Float16>;
}  // namespace tra
