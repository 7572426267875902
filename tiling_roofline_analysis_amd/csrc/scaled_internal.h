// scaled_internal.h -- what the operators on 8-bit matrices with block scales share: the
// scale of a block, the rounding of its elements, host-side views of scales.
#pragma once

#include "linear_epilogue.h"
#include "operator_args.h"

namespace tra {

constexpr int kScaleBlock = 128;       // elements of a block

namespace {

// A scale: its value, its inverse, and the bits that are stored.
struct BlockScale {
    float value, inverse;
    uint32_t bits;
};

// F = 7/8 2^9 (e4m3fn) or 7/8 2^16 (e5m2).
template <int FP8>
constexpr float kLargest = FP8 == TRA_FP8_E4M3 ? 448.0f : 57344.0f;

template <int FP8, int SCALE>
__device__ __forceinline__ BlockScale block_scale(float largest) {
    BlockScale s;
    if constexpr (SCALE == TRA_SCALE_E8M0) {
        // largest = m 2^e, 1/2 <= m < 1: the least power with largest / s <= 7/8 2^t is
        // 2^(e - t), or twice that where m > 7/8
        constexpr int t = FP8 == TRA_FP8_E4M3 ? 9 : 16;
        int e = __builtin_amdgcn_frexp_expf(largest) - t;
        e += __builtin_amdgcn_frexp_mantf(largest) > 0.875f ? 1 : 0;
        e = largest > 0.0f ? (e < -127 ? -127 : e) : 0;
        s.bits = static_cast<uint32_t>(e + 127);
        // (2^-127 is a subnormal; its inverse is not)
        s.inverse = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
        s.value = e > -127 ? __uint_as_float(static_cast<uint32_t>(e + 127) << 23)
                           : __uint_as_float(1u << 22);
    } else {
        const float v = fmaxf(largest / kLargest<FP8>, 1.17549435e-38f);
        s.value = largest > 0.0f ? v : 1.0f;
        s.inverse = 1.0f / s.value;
        s.bits = __float_as_uint(s.value);
    }
    return s;
}

// x / s, rounded to odd where it is not exact: a second rounding, to the 8-bit type, then
// gives what one rounding of the quotient would (its borders are even).  The quotient
// comes from the rounded inverse by one step of Newton's, and the sign of x - t s, which
// fma gives exactly, says on which side of t it lies.
__device__ __forceinline__ float odd_quotient(float x, const BlockScale &s) {
    const float first = x * s.inverse;
    const float t = fmaf(fmaf(-first, s.value, x), s.inverse, first);
    const float rest = fmaf(-t, s.value, x);
    const uint32_t bits = __float_as_uint(t);
    // one unit away from zero where the rest has t's sign, else towards it
    const uint32_t way = ((bits ^ __float_as_uint(rest)) >> 31) ? 0xffffffffu : 1u;
    const float odd = __uint_as_float(rest == 0.0f || (bits & 1u) ? bits : bits + way);
    // (of an infinity or NaN the rest is NaN)
    return fabsf(first) < __builtin_huge_valf() ? odd : first;
}

// N elements (a multiple of 4) of a block to 8 bits, 4 a word.
template <int FP8, int SCALE, int N>
__device__ __forceinline__ void to_fp8(const float (&x)[N], BlockScale s, uint32_t (&out)[N / 4]) {
    float t[N];
    float up = 1.0f;
    if (SCALE == TRA_SCALE_F32 && s.value < 8.6736174e-19f) {
        // 2^64 times both, so that the rest of a small element is no subnormal
        up = 1.8446744e19f;
        s.value *= up;
        s.inverse *= 5.4210109e-20f;
    }
#pragma unroll
    for (int e = 0; e < N; ++e) {
        if constexpr (SCALE == TRA_SCALE_E8M0)
            t[e] = x[e] * s.inverse;                // exact, or far below the type's least
        else
            t[e] = odd_quotient(x[e] * up, s);
    }
#pragma unroll
    for (int q = 0; q < N / 4; ++q) {
        int w = 0;
        if constexpr (FP8 == TRA_FP8_E4M3) {
            w = __builtin_amdgcn_cvt_pk_fp8_f32(t[4 * q], t[4 * q + 1], w, false);
            w = __builtin_amdgcn_cvt_pk_fp8_f32(t[4 * q + 2], t[4 * q + 3], w, true);
        } else {
            w = __builtin_amdgcn_cvt_pk_bf8_f32(t[4 * q], t[4 * q + 1], w, false);
            w = __builtin_amdgcn_cvt_pk_bf8_f32(t[4 * q + 2], t[4 * q + 3], w, true);
        }
        out[q] = static_cast<uint32_t>(w);
    }
}

// |x|, or 0 where that is not finite.
__device__ __forceinline__ float finite_size(float x) {
    const float a = fabsf(x);
    return a < __builtin_huge_valf() ? a : 0.0f;
}

// The largest of the 16 lanes' values (not negative, not NaN), in each of them.
__device__ __forceinline__ float largest_of_16(float v) {
#define TRA_DPP_MAX(ctrl) \
    v = fmaxf(v, __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), ctrl, 0xf, 0xf, true)))
    TRA_DPP_MAX(0xb1);     // lane ^ 1
    TRA_DPP_MAX(0x4e);     // lane ^ 2
    TRA_DPP_MAX(0x141);    // mirrored in its 8
    TRA_DPP_MAX(0x140);    // mirrored in its 16
#undef TRA_DPP_MAX
    return v;
}

}  // namespace

namespace host {

inline bool valid_fp8(int f) { return f == TRA_FP8_E4M3 || f == TRA_FP8_E5M2; }
inline bool valid_scale(int s) { return s == TRA_SCALE_F32 || s == TRA_SCALE_E8M0; }
inline int64_t scale_bytes(int s) { return s == TRA_SCALE_F32 ? 4 : 1; }

// Scales of `rows` x `blocks` as a row-major view, whichever of the two strides is 1;
// with neither (where both count), or with scales on top of each other, an invalid one.
inline View scale_view(const void *p, int64_t rows, int64_t blocks, int64_t ss_row,
                       int64_t ss_block, int64_t bytes) {
    if (rows <= 1) ss_row = 1;
    if (blocks <= 1) ss_block = rows;
    if (rows <= 0 || blocks <= 0) return View{p, 0, 0, 0, bytes};
    if (ss_row == 1) return View{p, blocks, rows, ss_block, bytes};
    if (ss_block == 1) return View{p, rows, blocks, ss_row, bytes};
    if (blocks == 1) return View{p, rows, 1, ss_row, bytes};
    return View{nullptr, 1, 1, 1, bytes};
}

}  // namespace host
}  // namespace tra
