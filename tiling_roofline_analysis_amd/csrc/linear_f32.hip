// linear_f32.hip -- the fused linear operators' kernels for float elements.
#include "linear_kernels.h"

namespace tra {
template struct LinearKernels<float>;
}  // namespace tra
