// linear_f16.hip -- the fused linear operators' kernels for _Float16 elements.
#include "linear_kernels.h"

namespace tra {
template struct LinearKernels<_Float16>;
}  // namespace tra
