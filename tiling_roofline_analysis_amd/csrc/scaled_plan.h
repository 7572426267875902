// scaled_plan.h -- internal interface of the products of 8-bit matrices: between their
// entry points (scaled.hip) and the kernels, which are built once per type of the result
// (scaled_f32.hip, scaled_bf16.hip, scaled_f16.hip).
#pragma once

#include "linear_internal.h"
#include "scaled_internal.h"

namespace tra {

// Formats of X's and W's values: both e4m3fn, or one of them e5m2.
enum ScaledFormats { kX4W4 = 0, kX5 = 1, kW5 = 2 };

// Few rows that the kernel quantizes itself: their bytes in LDS, filled up to whole blocks.
constexpr int kFewBytes = 16384;

// X is t.A and W is t.B[0], both k-contiguous; t.K is a multiple of 16.
struct ScaledArgs {
    TileArgs t;
    const void *SX;
    int64_t sx_row, sx_block;
    const void *SW;
    int64_t sw_row, sw_block;
    int w_shift;               // rows of W per scale: 1 << w_shift
    int x_cols;                // few rows: X is the result's type and has that many columns, or 0
};

struct ScaledPlan {
    TilePlan tile;
    ScaledFormats formats;
    int scale;
    bool make;                             // few rows: the kernel quantizes X itself
    size_t values_bytes, scales_bytes;     // workspace of a quantized X
    int64_t ldx, sx_block;                 // its layout
    size_t total;
};

template <typename T>
struct ScaledKernels {
    static hipError_t product(const ScaledPlan &plan, const ScaledArgs &p, hipStream_t stream);
};

}  // namespace tra
