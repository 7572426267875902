// scaled_bf16.hip -- products of 8-bit matrices with block scales, results of type __bf16.
#include "scaled_kernels.h"

namespace tra {
template struct ScaledKernels<__bf16>;
}  // namespace tra
