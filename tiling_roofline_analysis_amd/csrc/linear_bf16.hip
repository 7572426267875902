// linear_bf16.hip -- the fused linear operators' kernels for __bf16 elements.
#include "linear_kernels.h"

namespace tra {
template struct LinearKernels<__bf16>;
}  // namespace tra
