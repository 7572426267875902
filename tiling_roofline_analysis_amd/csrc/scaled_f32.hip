// scaled_f32.hip -- products of 8-bit matrices with block scales, results of type float.
#include "scaled_kernels.h"

namespace tra {
template struct ScaledKernels<float>;
}  // namespace tra
