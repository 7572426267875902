// scaled_kernels.h -- products of 8-bit matrices with block scales, results of type T.
// Included once by each scaled_<type>.hip.
//
// Bytes move as in linear_kernels.h: both operands k-contiguous, a K tile of 128 bytes a
// row straight into LDS, the same panels, waits, epilogue and split.  A K tile is one
// block of 128 elements, of which lane l holds row l % 16 and 32 elements of each operand:
// chunks l / 16 and 4 + l / 16 of its row.  (Which 32 does not matter, as long as both
// operands have the same: a block's sum is over all of them, and all share one scale.)
//
// 16-bit results: a block is one v_mfma_f32_16x16x128_f8f6f4.  The 8-bit matrix
// instructions of gfx950, this one and those of the generation before alike, add 8
// neighbouring products as integers, cut off 13 binary places below the largest one's
// exponent (measured: 2^16 + 2^3 is kept, 2^16 + 2^2 is not; between the groups of 8, and
// to the sum so far, they add in binary32).  That costs a sum of normal values 1e-5 of
// itself, against 2e-3 and 2e-4 by which its rounding to bfloat16 and binary16 is off in
// the mean.
// binary32 results: there it would be most of the error, so the operands are converted to
// bfloat16, exactly, and multiplied by v_mfma_f32_16x16x32_bf16, four a block, at half the
// rate.
//
// The scales come as part of the K tile: one word for each row of both panels, in one
// direct load a wave.
//   e8m0   16-bit results: the matrix unit multiplies by both scales; a lane passes its
//          row's byte
//   else   the block's sums start from zero and are added by v_fma_f32, times the product
//          of the two scales, 2^32 times as large (kUp): 4 instructions an MFMA, which run
//          beside other MFMAs
#pragma once

#include "linear_kernels.h"
#include "scaled_plan.h"

namespace tra {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));

// The two operands' formats (ScaledFormats) for the instruction: 0 e4m3fn, 1 e5m2.
template <int FORMATS>
constexpr int kFormatX = FORMATS == kX5 ? 1 : 0;
template <int FORMATS>
constexpr int kFormatW = FORMATS == kW5 ? 1 : 0;

// c + w x^T over a block, times the scales whose bytes are in sw and sx.
template <int FORMATS>
__device__ __forceinline__ f32x4 mma_scaled(i32x8 w, i32x8 x, f32x4 c, uint32_t sw, uint32_t sx) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
        w, x, c, kFormatW<FORMATS>, kFormatX<FORMATS>, 0, static_cast<int>(sw), 0,
        static_cast<int>(sx));
}

// w x^T over a block.  (Scales of zero, as constants, stand for the instruction without
// scales.)
template <int FORMATS>
__device__ __forceinline__ f32x4 mma_plain(i32x8 w, i32x8 x) {
    const f32x4 zero = {};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
        w, x, zero, kFormatW<FORMATS>, kFormatX<FORMATS>, 0, 0, 0, 0);
}

// Words 2 q and 2 q + 1 of a fragment, 8 elements, in bfloat16.
template <int FORMAT>
__device__ __forceinline__ bf16x8 widen(const i32x8 &v, int q) {
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    const uint32_t a = static_cast<uint32_t>(v[2 * q]), b = static_cast<uint32_t>(v[2 * q + 1]);
    bf16x2 t[4];
    if constexpr (FORMAT == 0) {
        t[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.0f, false);
        t[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.0f, true);
        t[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.0f, false);
        t[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.0f, true);
    } else {
        t[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(a, 1.0f, false);
        t[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(a, 1.0f, true);
        t[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(b, 1.0f, false);
        t[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(b, 1.0f, true);
    }
    return __builtin_shufflevector(__builtin_shufflevector(t[0], t[1], 0, 1, 2, 3),
                                   __builtin_shufflevector(t[2], t[3], 0, 1, 2, 3), 0, 1, 2, 3, 4,
                                   5, 6, 7);
}

// A scale's word as a binary32 number.
template <int SCALE>
__device__ __forceinline__ float scale_value(uint32_t word) {
    // 0 and 255 stand for 2^-127, a subnormal, and NaN
    if constexpr (SCALE == TRA_SCALE_E8M0)
        word = word << 23 | (word == 0 || word == 255 ? 0x400000u : 0u);
    return __uint_as_float(word);
}

// ---- scales whose product leaves binary32's range ----------------------------------------
//
// A block's sum t is 0 or between 2^-25 and 2^32 in size.  It is multiplied by the product of its
// two scales, which may lie past either end of binary32's range though t times it does not.
// So sums are taken 2^32 times as large.  A product of scales that is subnormal even then is off by
// 2^-150 at most, and t times it, brought down again, by no more: half of the least number.  Where
// a sum comes out infinite or NaN and the scales are large enough for it (results past 2^96, products
// of scales past it; else the operands are infinite or NaN themselves) the wave takes its sums once
// more with add_scaled, whose steps leave the range only where their result does: 13 to 18 times
// the time of a tile.  Otherwise it costs the look at the sums at a tile's end: 8192 x 12288 x 4096
// with binary32 scales 380 us, 368 without; with the extremes of the scales kept in the K loop
// instead, to find such products, 393.
constexpr float kUp = 4294967296.0f, kDown = 1.0f / kUp;

// d + t a b for two scales: t times their product where that is a normal number, else times the
// larger and then the smaller one.  (Of a product past the range's end the smaller one is above 1,
// so t times the larger overflows only with the result.  Of one below the least normal number t
// times the larger is normal, or both scales are below 2^-101 and the result is 0.)
__device__ __forceinline__ float add_scaled(float d, float t, float a, float b) {
    const float both = a * b;
    const bool normal = __builtin_amdgcn_classf(both, 0x108);      // of either sign
    const bool less = fabsf(a) < fabsf(b);
    return fmaf(normal ? t : t * (less ? b : a), normal ? both : less ? a : b, d);
}

// The larger size of two, NaN if either is.
__device__ __forceinline__ float larger(float a, float b) {
    return __builtin_elementwise_maximum(fabsf(a), fabsf(b));
}

// Sums of 16 x 16 tiles down by 2^32; whether some of the wave's were infinite or NaN.
template <int N, int TI, int TJ>
__device__ __forceinline__ bool bring_down(f32x4 (&c)[N][TI][TJ]) {
    float most = 0.0f;
#pragma unroll
    for (int h = 0; h < N; ++h)
#pragma unroll
        for (int i = 0; i < TI; ++i)
#pragma unroll
            for (int j = 0; j < TJ; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    most = larger(most, c[h][i][j][e]);
                    c[h][i][j][e] *= kDown;
                }
    return __builtin_amdgcn_ballot_w64(!(most < __builtin_huge_valf())) != 0;
}

// Whether scales no larger than a lane's x and w, of any lanes, can make sums infinite of finite
// values: 2^15 blocks of 2^32 each, 2^32 times as large; or one of the scales that by itself.
__device__ __forceinline__ bool far_scales(float x, float w) {
    auto of_lane = [](float v, int l) __attribute__((always_inline)) {
        return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), l));
    };
#pragma unroll 1
    for (int l = 0; l < 64; ++l) {
        x = larger(x, of_lane(x, l));
        w = larger(w, of_lane(w, l));
    }
    return __builtin_amdgcn_ballot_w64(!(x * w < 0x1p48f && larger(x, w) < 0x1p95f)) != 0;
}

// threadIdx.x & 63, which takes no register before it is asked for.
__device__ __forceinline__ int lane_id() {
    return static_cast<int>(__builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, 0u)));
}

// A barrier that no load is waited for at; and a wait for this wave's direct loads but
// the last VM (stage_sync does both).
__device__ __forceinline__ void step_sync() {
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}
template <int VM>
__device__ __forceinline__ void stage_wait() {
    static_assert(VM >= 0 && VM < 64, "vmcnt range");
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt((VM & 15) | ((VM >> 4) << 14) | (7 << 4) | (15 << 8));
}

using Bytes = uint8_t;

// Rows row0 .. + 15 of a panel: chunks l / 16 and 4 + l / 16 of each.
template <typename P>
__device__ __forceinline__ i32x8 fragment8(const char *st, int panel, int row0) {
    const u32x4 a = P::fragment(st, panel, row0, 0), b = P::fragment(st, panel, row0, 1);
    return __builtin_bit_cast(
        i32x8, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
}

// Loads a panel of k-contiguous rows, as Panel::load_direct does, but with buffers that end
// with the panel's rows inside the matrix and, one a load, begin at the load's first row:
// a lane's offset is the same in every load of an operand's panels.
template <typename P>
struct RowPanel {
    static constexpr int L = P::INS;
    static constexpr int ROWS = P::BYTES / 128 / L;      // a load's
    static_assert(ROWS % 16 == 0, "every load's chunks are swizzled alike");

    int64_t skip;              // bytes from a load's rows to the next's
    int length[L];

    // `rows` of the matrix from the panel's first row on, `ld` bytes apart.
    __device__ __forceinline__ RowPanel(int64_t rows, int64_t ld) : skip(ROWS * ld) {
#pragma unroll
        for (int i = 0; i < L; ++i) {
            const int64_t n = (rows - i * ROWS) * ld;
            length[i] = static_cast<int>(n <= 0 ? 0 : n < 0x7fffffff ? n : 0x7fffffff);
        }
    }
    static __device__ __forceinline__ uint32_t offset(int wave, int64_t ld) {
        return static_cast<uint32_t>(P::line(wave, 0)) * static_cast<uint32_t>(ld) +
               static_cast<uint32_t>(P::chunk(wave, 0) * 16);
    }
    __device__ __forceinline__ void load(int wave, const char *corner, uint32_t off, int rem,
                                         char *lds) const {
        const uint32_t at = P::chunk(wave, 0) * 16 >= rem ? P::OUTSIDE : off;
#pragma unroll
        for (int i = 0; i < L; ++i) {
            // (variables, whose types depend on no template parameter: from expressions that
            // do, the compiler's host pass drops every kernel that calls this but the first,
            // with no word before the link)
            char *to = lds + P::lds_block(wave, i);
            void *from = const_cast<char *>(corner) + i * skip;
            const int bytes = length[i];
            const __amdgpu_buffer_rsrc_t rsrc =
                __builtin_amdgcn_make_buffer_rsrc(from, (short)0, bytes, 0x00020000);
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, to, 16, at, 0, 0, 0);
        }
    }
};

// Scales of a K tile in LDS: a word for each of WAVES * 64 rows, BM of X's and then BN of
// W's (and none for the rest).  A wave loads 64 of them, of one operand.
template <int SCALE, int BM, int BN, int WAVES>
struct ScalePanel {
    static constexpr int BYTES = WAVES * 256;
    static constexpr int SIZE = SCALE == TRA_SCALE_E8M0 ? 1 : 4;
    static_assert(BM % 64 == 0 && BN % 64 == 0 && BM + BN <= WAVES * 64, "a wave has one operand");

    const char *at;        // the tile's first row's scale, of the K tile to load
    int64_t step;          // bytes from a K tile's to the next's
    uint32_t offset;       // this lane's row's

    __device__ __forceinline__ ScalePanel(const ScaledArgs &p, int wave, int64_t m0, int64_t n0,
                                          int first) {
        const int r = wave * 64 + static_cast<int>(threadIdx.x & 63);
        constexpr uint32_t OUTSIDE = Panel<Bytes, true, 64, 4>::OUTSIDE;
        if (wave * 64 < BM) {
            at = static_cast<const char *>(p.SX) + m0 * p.sx_row * SIZE;
            step = p.sx_block * SIZE;
            offset = m0 + r < p.t.M ? static_cast<uint32_t>(r * p.sx_row * SIZE) : OUTSIDE;
        } else {
            const int64_t n = n0 + (r - BM), block = n0 >> p.w_shift;
            at = static_cast<const char *>(p.SW) + block * p.sw_row * SIZE;
            step = p.sw_block * SIZE;
            offset = r - BM < BN && n < p.t.N
                         ? static_cast<uint32_t>(((n >> p.w_shift) - block) * p.sw_row * SIZE)
                         : OUTSIDE;
        }
        at += first * step;
    }

    // rem: elements of K left, as in Panel::load_direct; one load, whatever it is
    __device__ __forceinline__ void load(int wave, int rem, char *lds) {
        const __amdgpu_buffer_rsrc_t rsrc =
            __builtin_amdgcn_make_buffer_rsrc((void *)at, (short)0, rem > 0 ? 0x7fffffff : 0,
                                              0x00020000);
        // (a byte arrives as a word too)
        if constexpr (SIZE == 1)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, lds + wave * 256, 1, offset, 0, 0, 0);
        else
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, lds + wave * 256, 4, offset, 0, 0, 0);
        at += step;
    }

    // The scales of rows row0 .. + 15 (of W's: from BM on), one a lane.
    static __device__ __forceinline__ uint32_t of_rows(const char *st, int panel, int row0) {
        return *reinterpret_cast<const uint32_t *>(
            st + panel + (row0 + static_cast<int>(threadIdx.x & 15)) * 4);
    }

    // One row's, in every lane.
    static __device__ __forceinline__ uint32_t of_row(const char *st, int panel, int row) {
        return *reinterpret_cast<const uint32_t *>(st + panel + row * 4);
    }

    // The scales of the four rows whose sums a lane gets.
    static __device__ __forceinline__ u32x4 of_sums(const char *st, int panel, int row0) {
        return *reinterpret_cast<const u32x4 *>(
            st + panel + (row0 + static_cast<int>(threadIdx.x >> 4 & 3) * 4) * 4);
    }
};

// The kernel's arguments again, behind all that was before: read there, they and what follows
// from them take no registers in the K loop (where they cost scaled_wide 70 SGPRs and spills).
__device__ __forceinline__ const ScaledArgs &arguments_again() {
    auto *at = __builtin_amdgcn_kernarg_segment_ptr();
    asm volatile("" : "+s"(at));
    return *(const ScaledArgs *)at;
}

template <int SCALE>
__device__ __forceinline__ float scale_at(const void *s, int64_t at) {
    if constexpr (SCALE == TRA_SCALE_E8M0)
        return scale_value<SCALE>(static_cast<const uint8_t *>(s)[at]);
    else
        return scale_value<SCALE>(static_cast<const uint32_t *>(s)[at]);
}

__device__ __forceinline__ int64_t at_most_last(int64_t i, int64_t n) { return i < n ? i : n - 1; }

// Whether the scales of a wave's rows and columns can make sums infinite: BM / 2 rows of X from
// `row` on and, WIDE, as many BM / 2 further on; HC columns from `col` on in both halves of the
// tile's.
template <int SCALE, bool WIDE, int BM, int BN, int HC>
__device__ __forceinline__ bool far_scales(int row, int col) {
    constexpr int ROWS = WIDE ? BM / 4 : BM / 2;
    static_assert(ROWS <= 64 && 2 * HC <= 64, "a lane each");
    const ScaledArgs &p = arguments_again();
    const Part part(p.t, 0, BM * BN);
    int tm, tn;
    grouped_tile32<WIDE ? kGroupWide : kGroupTile>(part.tile, p.t.tiles_m, p.t.tiles_n, tm, tn);
    const int lane = lane_id(), r = row + lane % ROWS, c = lane % (2 * HC);
    const int64_t m = static_cast<int64_t>(tm) * BM + r;
    const int64_t n = static_cast<int64_t>(tn) * BN + c / HC * (BN / 2) + col + c % HC;
    const int64_t x0 = at_most_last(m, p.t.M) * p.sx_row;
    const int64_t x1 = at_most_last(WIDE ? m + BM / 2 : m, p.t.M) * p.sx_row;
    const int64_t w0 = (at_most_last(n, p.t.N) >> p.w_shift) * p.sw_row;
    float x = 0.0f, w = 0.0f;
#pragma unroll 1
    for (int b = part.first; b < part.first + part.count; ++b) {
        x = larger(x, scale_at<SCALE>(p.SX, x0 + b * p.sx_block));
        if (WIDE) x = larger(x, scale_at<SCALE>(p.SX, x1 + b * p.sx_block));
        w = larger(w, scale_at<SCALE>(p.SW, w0 + b * p.sw_block));
    }
    return far_scales(x, w);
}

// The 16 x 16 sums of rows m0 .. and columns n0 .., K tiles first .. + count - 1.
template <int FORMATS, int SCALE, bool WIDEN>
__device__ __forceinline__ f32x4 sums_by_parts(const ScaledArgs &p, int64_t m0, int64_t n0,
                                               int first, int count) {
    const TileArgs &a = p.t;
    const int l16 = lane_id() & 15, g = lane_id() >> 4;
    const int64_t m = at_most_last(m0 + l16, a.M);
    const char *x_at = static_cast<const char *>(a.A) + m * a.lda;
    const char *w_at = static_cast<const char *>(a.B[0]) + at_most_last(n0 + l16, a.N) * a.ldb;
    f32x4 c = {};
    for (int b = first; b < first + count; ++b) {
        u32x4 x[2] = {}, w[2] = {};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int64_t k = static_cast<int64_t>(b) * 128 + h * 64 + g * 16;
            if (k < a.K) {
                x[h] = *reinterpret_cast<const u32x4 *>(x_at + k);
                w[h] = *reinterpret_cast<const u32x4 *>(w_at + k);
            }
        }
        const float sx = scale_at<SCALE>(p.SX, m * p.sx_row + b * p.sx_block);
        float sw[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
            sw[e] = scale_at<SCALE>(p.SW, (at_most_last(n0 + 4 * g + e, a.N) >> p.w_shift) *
                                              p.sw_row + b * p.sw_block);
        const i32x8 x8 = __builtin_bit_cast(
            i32x8, __builtin_shufflevector(x[0], x[1], 0, 1, 2, 3, 4, 5, 6, 7));
        const i32x8 w8 = __builtin_bit_cast(
            i32x8, __builtin_shufflevector(w[0], w[1], 0, 1, 2, 3, 4, 5, 6, 7));
        f32x4 t = {};
        if constexpr (WIDEN) {
#pragma unroll
            for (int q = 0; q < 4; ++q)
                t = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen<kFormatW<FORMATS>>(w8, q),
                                                            widen<kFormatX<FORMATS>>(x8, q), t, 0,
                                                            0, 0);
        } else {
            t = mma_plain<FORMATS>(w8, x8);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) c[e] = add_scaled(c[e], t[e], sx, sw[e]);
    }
    return c;
}

// What epi_put has put into `lds` of a wave's sums, TI x TJ of 16 x 16 from `row` and, in both
// halves of the tile's columns, `col` on.
template <int FORMATS, int SCALE, bool WIDEN, int BM, int BN, int HC, int TI, int TJ>
__device__ __forceinline__ void sums_again(char *lds, int row, int col) {
    const ScaledArgs &p = arguments_again();
    const Part part(p.t, 0, BM * BN);
    int tm, tn;
    grouped_tile32<BM == 256 ? kGroupWide : kGroupTile>(part.tile, p.t.tiles_m, p.t.tiles_n, tm,
                                                        tn);
    const int l16 = lane_id() & 15, g = lane_id() >> 4;
#pragma unroll 1
    for (int n = 0; n < 2 * TI * TJ; ++n) {
        const int h = n / (TI * TJ), i = n / TJ % TI, j = n % TJ;
        *reinterpret_cast<f32x4 *>(lds + epi_at<HC>(i * 16 + l16, h * (HC / 4) + j * 4 + g)) =
            sums_by_parts<FORMATS, SCALE, WIDEN>(
                p, static_cast<int64_t>(tm) * BM + row + i * 16,
                static_cast<int64_t>(tn) * BN + h * (BN / 2) + col + j * 16, part.first,
                part.count);
    }
}

// ---- the tile kernel ---------------------------------------------------------------------
//
// linear_tile for one-byte elements: BM x BN of Y per workgroup of four waves in 2 x 2.
// A K tile is one MFMA step, computed in two halves, the columns of half 0 and of half
// 1; iteration s:
//   read half 1's fragments of tile s; compute half 0;
//   wait for this wave's loads of tile s + 1, meet the other waves;
//   load tile s + S into the stage of tile s;
//   read X's and half 0's fragments of tile s + 1; compute half 1.
// For products of few tiles, which latency bounds as much as the matrix units, and for
// binary32 results, whose widening keeps the vector units as busy as those: 512 x 4096 x 4096
// with e8m0 scales to bfloat16 17.0 us (1.01 PFLOP/s), to binary32 29.2 (0.59);
// 4096 x 8192 x 4096 to binary32 240 (1.15 PFLOP/s).
template <int BM, int BN, int SCALE>
struct ScaledShape {
    static constexpr int WAVES = 4, TI = BM / 32, TJ = BN / 64, HC = BN / 4;
    using PA = Panel<Bytes, true, BM, WAVES>;
    using PB = Panel<Bytes, true, BN / 2, WAVES>;
    using PS = ScalePanel<SCALE, BM, BN, WAVES>;
    static constexpr int SCALES = PA::BYTES + 2 * PB::BYTES;     // where they begin
    static constexpr int STAGE = SCALES + PS::BYTES;
    static constexpr int MINE = BM / 2 * HC * 8;
    static constexpr int per_cu(int stages) { return stages * STAGE <= 80 * 1024 ? 2 : 1; }
};

// EACH: binary32 results and e8m0 scales, one for each row of W; else 128 rows share one, as
// with binary32 scales (4096 x 8192 x 4096: 339 us with EACH in 64 x 128 tiles, 244 without in 128 x 128, whose
// VGPRs EACH would leave one workgroup a CU).
template <typename T, int FORMATS, int SCALE, bool EACH, int BM, int BN, int S>
__global__ __launch_bounds__(256, (ScaledShape<BM, BN, SCALE>::per_cu(S))) void scaled_tile(
    const ScaledArgs p) {
    using X = ScaledShape<BM, BN, SCALE>;
    using PA = typename X::PA;
    using PB = typename X::PB;
    using PS = typename X::PS;
    constexpr int TI = X::TI, TJ = X::TJ, HC = X::HC;
    constexpr bool WIDEN = std::is_same_v<T, float>;
    constexpr bool UNIT = SCALE == TRA_SCALE_E8M0 && !WIDEN;    // the matrix unit scales
    static_assert(!EACH || (SCALE == TRA_SCALE_E8M0 && WIDEN), "else the matrix unit scales");
    static_assert(S == 2 || S == 4 || S == 6, "whole pairs of stages");
    static_assert(X::STAGE >= 2 * X::MINE, "LDS");
    __shared__ __align__(1024) char st0[X::STAGE], st1[X::STAGE];
    __shared__ __align__(1024) char st2[S > 2 ? X::STAGE : 16], st3[S > 2 ? X::STAGE : 16];
    __shared__ __align__(1024) char st4[S > 4 ? X::STAGE : 16], st5[S > 4 ? X::STAGE : 16];
    auto stage = [&](auto u) __attribute__((always_inline))->char * {
        constexpr int U = decltype(u)::value % S;
        if constexpr (U == 0) return st0;
        if constexpr (U == 1) return st1;
        if constexpr (U == 2) return st2;
        if constexpr (U == 3) return st3;
        if constexpr (U == 4) return st4;
        return st5;
    };
    for_each(std::make_integer_sequence<int, S>{}, [&](auto u) __attribute__((always_inline)) {
        lds_poison(reinterpret_cast<float *>(stage(u)), X::STAGE / 4);
        return true;
    });

    const TileArgs &a = p.t;
    const Part part(a, 0, BM * BN);
    int tm, tn;
    grouped_tile32<kGroupTile>(part.tile, a.tiles_m, a.tiles_n, tm, tn);
    const int64_t m0 = static_cast<int64_t>(tm) * BM;
    const int64_t n0 = static_cast<int64_t>(tn) * BN, n1 = n0 + BN / 2;
    const int first = part.first, count = part.count;
    Walk<Bytes, true, true> walk(a, 0, m0, n0, n1, false, first, count);

    const int wave = wave_id();
    const int wm = wave >> 1, wn = wave & 1;
    PS scales(p, wave, m0, n0, first);
    // MFMAs that add to the same registers are too near each other in small tiles: two sets
    // of sums there, for odd and even K tiles, added at the end
    constexpr int SETS = UNIT && 2 * TI * TJ < 16 ? 2 : 1;
    f32x4 c[SETS][2][TI][TJ] = {};

    i32x8 x[2][TI], w[2][TJ];          // X's of odd and even tiles; W's of the halves
    uint32_t sx[2][TI], sw[2][TJ];
    u32x4 sws[2][TJ];
    auto read_x = [&](auto parity, const char *st) __attribute__((always_inline)) {
        constexpr int P = decltype(parity)::value;
#pragma unroll
        for (int i = 0; i < TI; ++i) {
            x[P][i] = fragment8<PA>(st, 0, wm * (BM / 2) + i * 16);
            sx[P][i] = PS::of_rows(st, X::SCALES, wm * (BM / 2) + i * 16);
        }
    };
    auto read_w = [&](auto half, const char *st) __attribute__((always_inline)) {
        constexpr int H = decltype(half)::value;
#pragma unroll
        for (int j = 0; j < TJ; ++j) {
            const int row = wn * HC + j * 16;
            w[H][j] = fragment8<PB>(st, PA::BYTES + H * PB::BYTES, row);
            if constexpr (EACH)
                sws[H][j] = PS::of_sums(st, X::SCALES, BM + H * (BN / 2) + row);
            else if constexpr (UNIT)
                sw[H][j] = PS::of_rows(st, X::SCALES, BM + H * (BN / 2) + row);
            else if (j == 0)
                sw[H][j] = PS::of_row(st, X::SCALES, BM + H * (BN / 2));
        }
    };
    auto compute = [&](auto half, auto parity) __attribute__((always_inline)) {
        constexpr int H = decltype(half)::value, P = decltype(parity)::value;
        f32x4 t[TI][TJ] = {};
        if constexpr (WIDEN) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                bf16x8 wide[TJ];
#pragma unroll
                for (int j = 0; j < TJ; ++j) wide[j] = widen<kFormatW<FORMATS>>(w[H][j], q);
#pragma unroll
                for (int i = 0; i < TI; ++i) {
                    const bf16x8 v = widen<kFormatX<FORMATS>>(x[P][i], q);
#pragma unroll
                    for (int j = 0; j < TJ; ++j)
                        t[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wide[j], v, t[i][j], 0, 0,
                                                                          0);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < TI; ++i) {
            const float s = UNIT ? 0.0f : scale_value<SCALE>(sx[P][i]) * (EACH ? kUp : 1.0f);
            const float both = UNIT || EACH ? 0.0f : s * (scale_value<SCALE>(sw[H][0]) * kUp);
#pragma unroll
            for (int j = 0; j < TJ; ++j) {
                f32x4 &d = c[P % SETS][H][i][j];
                if constexpr (UNIT) {
                    d = mma_scaled<FORMATS>(w[H][j], x[P][i], d, sw[H][j], sx[P][i]);
                } else {
                    if constexpr (!WIDEN) t[i][j] = mma_plain<FORMATS>(w[H][j], x[P][i]);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        d[e] = fmaf(t[i][j][e],
                                    EACH ? s * scale_value<SCALE>(sws[H][j][e]) : both, d[e]);
                }
            }
        }
    };
    constexpr int MFMAS = TI * TJ * (WIDEN ? 4 : 1);
    constexpr int READS_W = TJ * 2 + (UNIT || EACH ? TJ : 1), READS_X = TI * 3;
    constexpr std::integral_constant<int, 0> zero;
    constexpr std::integral_constant<int, 1> one;

    constexpr int IA = PA::template DINS<16>, IB = PB::template DINS<16>;
    constexpr int LOADS = IA + 2 * IB + 1;
    uint32_t oa[IA], ob0[IB], ob1[IB];
#pragma unroll
    for (int i = 0; i < IA; ++i) oa[i] = PA::template offset<16>(wave, i, a.M - m0, a.lda);
#pragma unroll
    for (int i = 0; i < IB; ++i) {
        ob0[i] = PB::template offset<16>(wave, i, a.N - n0, a.ldb);
        ob1[i] = PB::template offset<16>(wave, i, a.N - n1, a.ldb);
    }
    const int pitch_a = static_cast<int>(a.lda), pitch_b = static_cast<int>(a.ldb);
    auto issue = [&](char *st) __attribute__((always_inline)) {
        PA::template load_direct<16>(wave, walk.a, pitch_a, oa, walk.rem, st);
        PB::template load_direct<16>(wave, walk.b0, pitch_b, ob0, walk.rem, st + PA::BYTES);
        PB::template load_direct<16>(wave, walk.b1, pitch_b, ob1, walk.rem,
                                     st + PA::BYTES + PB::BYTES);
        scales.load(wave, walk.rem, st + X::SCALES);
        walk.next();
    };
    for_each(std::make_integer_sequence<int, S>{}, [&](auto u) __attribute__((always_inline)) {
        issue(stage(u));
        __builtin_amdgcn_sched_barrier(0);
        return true;
    });
    stage_sync<(S - 1) * LOADS>();
    read_x(zero, st0);
    read_w(zero, st0);
    auto iteration = [&](auto u) __attribute__((always_inline)) {
        constexpr int U = decltype(u)::value;
        constexpr std::integral_constant<int, U % 2> now;
        constexpr std::integral_constant<int, (U + 1) % 2> next;
        read_w(one, stage(u));
        compute(zero, now);
        interleave<MFMAS, READS_W, 0>();
        stage_sync<(S - 2) * LOADS>();
        issue(stage(u));
        read_x(next, stage(std::integral_constant<int, U + 1>{}));
        read_w(zero, stage(std::integral_constant<int, U + 1>{}));
        compute(one, now);
        interleave<MFMAS, READS_X + READS_W, LOADS>();
        __builtin_amdgcn_sched_barrier(0);
    };
    int s = 0;
    for (; s + S <= count; s += S)
        for_each(std::make_integer_sequence<int, S>{}, [&](auto u) __attribute__((always_inline)) {
            iteration(u);
            return true;
        });
    for_each(std::make_integer_sequence<int, S - 1>{}, [&](auto u) __attribute__((always_inline)) {
        if (s + decltype(u)::value >= count) return false;
        iteration(u);
        return true;
    });

    // Every wave has read its last fragments, and no load is in flight, before
    // the stages are reused.
    stage_sync<0>();
    char *mine = (wave < 2 ? st0 : st1) + (wave & 1) * X::MINE;
#pragma unroll
    for (int k = 1; k < SETS; ++k)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < TI; ++i)
#pragma unroll
                for (int j = 0; j < TJ; ++j) c[0][h][i][j] += c[k][h][i][j];
    bool again = false;
    if constexpr (!UNIT)
        again = bring_down(c[0]) && far_scales<SCALE, false, BM, BN, HC>(wm * (BM / 2), wn * HC);
    epi_put<HC>(mine, c[0][0], 0);
    epi_put<HC>(mine, c[0][1], 1);
    if constexpr (!UNIT) {
        if (again)
            sums_again<FORMATS, SCALE, WIDEN, BM, BN, HC, TI, TJ>(mine, wm * (BM / 2), wn * HC);
    }
    wave_sync();
    epi_rows<T, false, HC, BM / 2>(
        a, 0, part.sums == nullptr ? nullptr : part.sums + wm * (BM / 2) * BN + wn * HC, BN, mine,
        m0 + wm * (BM / 2), n0 + wn * HC, n1 + wn * HC);
}

// ---- the wide kernel -----------------------------------------------------------------------
//
// 256 x 256 of Y per workgroup of eight waves, for 16-bit results of many tiles, which the
// matrix units bound.  The panels and the two groups of waves, half a step apart, are
// linear_wide's: A0, A1, B0, B1 of 128 rows each, in two stages, an array each; a wave
// computes 64 rows of each A panel by 32 columns of each B panel; there is one wave of each
// group on every SIMD, and while the one computes the other reads fragments.  A K tile is
// two steps of 16 MFMAs (with four of 8, half as many MFMAs between two barriers, the K
// tile took 1.2 times as long).  Tile s:
//   R0  reads B0, A0, all scales;  loads A1 > s + 1;          barrier
//   C0  reads B1 behind the first MFMAs;  A0 x B0, A0 x B1;   barrier
//   R1  reads A1;  loads A0, B0, scales > s + 2;              barrier
//   C1  loads B1 > s + 2;  A1 x B1, A1 x B0;                  barrier
// The group behind does each one barrier later, so what is read in one of these may be
// loaded anew from the second one after it on; every load is issued there.  What is to
// be read in one of them has to be in LDS, of both groups' loads, at the end of the second
// one before it: behind R0, R1 and C1 a wave waits until its last 4 panels and scales, in
// the order above, are all that is in flight.
// 8192 x 12288 x 4096 with e8m0 scales, six rounds of tiles, takes 321 us with its operands in the
// cache and 334 to 339 from memory (2.43 PFLOP/s).  Of the 53 us a tile 1.31 are each K tile's, and 12
// go for its first loads and its stores, which are 7 at the memory's rate.  The matrix units are
// busy 62 to 76% of the time, at clocks that the power lowers (1.9 GHz).
// Binary32 scales: a row tile's sums are added while the next ones' MFMAs run, a step's last
// behind the next step's reads, while the other group's do.
template <typename T, int FORMATS, int SCALE>
__global__ __launch_bounds__(512, 2) void scaled_wide(const ScaledArgs p) {
    using PP = Panel<Bytes, true, 128, 8>;
    using PS = ScalePanel<SCALE, 256, 256, 8>;
    constexpr int L = PP::INS;
    constexpr bool UNIT = SCALE == TRA_SCALE_E8M0;
    static_assert(sizeof(T) == 2 && L == 2 && PP::BYTES == 64 * 64 * 4,
                  "panels of two loads a wave; a wave's sums fill one");
    __shared__ __align__(1024) char a00[PP::BYTES], a01[PP::BYTES], a10[PP::BYTES], a11[PP::BYTES];
    __shared__ __align__(1024) char b00[PP::BYTES], b01[PP::BYTES], b10[PP::BYTES], b11[PP::BYTES];
    __shared__ __align__(1024) char s0[PS::BYTES], s1[PS::BYTES];
    lds_poison(reinterpret_cast<float *>(a00), PP::BYTES / 4);
    lds_poison(reinterpret_cast<float *>(a01), PP::BYTES / 4);
    lds_poison(reinterpret_cast<float *>(a10), PP::BYTES / 4);
    lds_poison(reinterpret_cast<float *>(a11), PP::BYTES / 4);
    lds_poison(reinterpret_cast<float *>(b00), PP::BYTES / 4);
    lds_poison(reinterpret_cast<float *>(b01), PP::BYTES / 4);
    lds_poison(reinterpret_cast<float *>(b10), PP::BYTES / 4);
    lds_poison(reinterpret_cast<float *>(b11), PP::BYTES / 4);
    lds_poison(reinterpret_cast<float *>(s0), PS::BYTES / 4);
    lds_poison(reinterpret_cast<float *>(s1), PS::BYTES / 4);

    const TileArgs &a = p.t;
    const Part part(a, 0, 256 * 256);
    int tm, tn;
    grouped_tile32<kGroupWide>(part.tile, a.tiles_m, a.tiles_n, tm, tn);
    const int64_t m0 = static_cast<int64_t>(tm) * 256, n0 = static_cast<int64_t>(tn) * 256;
    const int64_t n1 = n0 + 128;
    const int first = part.first, count = part.count;
    Walk<Bytes, true, true> walk(a, 0, m0, n0, n1, false, first, count);
    const int64_t lower = 128 * a.lda;

    const int wave = wave_id();
    const int wm = wave >> 2, wn = wave & 3;
    PS scales(p, wave, m0, n0, first);
    using PR = RowPanel<PP>;
    const uint32_t oa = PR::offset(wave, a.lda), ob = PR::offset(wave, a.ldb);
    const PR pa0(a.M - m0, a.lda), pa1(a.M - m0 - 128, a.lda);
    const PR pb0(a.N - n0, a.ldb), pb1(a.N - n1, a.ldb);

    // A1 and B1 are loaded behind the others, when `walk` is a tile on.
    const char *late_a = nullptr, *late_b = nullptr;
    int late_rem = 0;
    auto load_a0_b0 = [&](char *a0, char *b0, char *sc) __attribute__((always_inline)) {
        pa0.load(wave, walk.a, oa, walk.rem, a0);
        pb0.load(wave, walk.b0, ob, walk.rem, b0);
        scales.load(wave, walk.rem, sc);
        late_a = walk.a + lower;
        late_b = walk.b1;
        late_rem = walk.rem;
        walk.next();
    };
    auto load_a1 = [&](char *st) __attribute__((always_inline)) {
        pa1.load(wave, late_a, oa, late_rem, st);
    };
    auto load_b1 = [&](char *st) __attribute__((always_inline)) {
        pb1.load(wave, late_b, ob, late_rem, st);
    };

    f32x4 c[2][2][4][2] = {};      // [A panel][B panel]
    i32x8 x[4], w[2][2];           // [row tile]; [B panel][column tile]
    // e8m0: a byte for each row tile (column tile) of each panel.  f32: X's of each row tile,
    // and W's of each B panel, in a scalar register.
    uint32_t sx[2][UNIT ? 1 : 4], sw[2];
    float both[2] = {};
    // binary32 scales: the last row tile's sums, which are added late, and their scale
    f32x4 t[2];
    float ts = 0.0f;
    auto read_scales = [&](const char *sc) __attribute__((always_inline)) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint32_t v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = PS::of_rows(sc, 0, h * 128 + wm * 64 + i * 16);
            if constexpr (UNIT) {
                sx[h][0] = v[0] | v[1] << 8 | v[2] << 16 | v[3] << 24;
                const uint32_t w0 = PS::of_rows(sc, 0, 256 + h * 128 + wn * 32);
                const uint32_t w1 = PS::of_rows(sc, 0, 256 + h * 128 + wn * 32 + 16);
                sw[h] = w0 | w1 << 8;
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) sx[h][UNIT ? 0 : i] = v[i];
                sw[h] = PS::of_row(sc, 0, 256 + h * 128);
            }
        }
    };
    auto read_a = [&](const char *st) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = fragment8<PP>(st, 0, wm * 64 + i * 16);
    };
    auto read_b = [&](auto half, const char *st) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < 2; ++j)
            w[decltype(half)::value][j] = fragment8<PP>(st, 0, wn * 32 + j * 16);
    };
    auto scale_of = [&](auto ha, int i, auto hb) __attribute__((always_inline)) {
        return __uint_as_float(sx[decltype(ha)::value][UNIT ? 0 : i]) * both[decltype(hb)::value];
    };
    auto add_to = [&](f32x4 (&sum)[2], const f32x4 (&u)[2], float s) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) sum[j][e] = fmaf(u[j][e], s, sum[j][e]);
    };
    // One MFMA of e8m0: the bytes of the scales are immediate operands.
    auto scaled = [&](auto ha, auto hb, auto ii, auto jj) __attribute__((always_inline)) {
        constexpr int HA = decltype(ha)::value, HB = decltype(hb)::value;
        constexpr int I = decltype(ii)::value, J = decltype(jj)::value;
        c[HA][HB][I][J] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
            w[HB][J], x[I], c[HA][HB][I][J], kFormatW<FORMATS>, kFormatX<FORMATS>, J,
            static_cast<int>(sw[HB]), I, static_cast<int>(sx[HA][0]));
    };
    // The 8 MFMAs of a quadrant; binary32: and the sums of all but its last row tile.
    auto quadrant = [&](auto ha, auto hb) __attribute__((always_inline)) {
        constexpr int HA = decltype(ha)::value, HB = decltype(hb)::value;
        if constexpr (UNIT) {
            for_each(std::make_integer_sequence<int, 8>{}, [&](auto n) __attribute__((always_inline)) {
                constexpr int U = decltype(n)::value;
                scaled(ha, hb, std::integral_constant<int, U / 2>{},
                       std::integral_constant<int, U % 2>{});
                return true;
            });
        } else {
            f32x4 u[4][2];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
#pragma unroll
                for (int j = 0; j < 2; ++j) u[i][j] = mma_plain<FORMATS>(w[HB][j], x[i]);
                __builtin_amdgcn_sched_barrier(0);
                if (i > 0) add_to(c[HA][HB][i - 1], u[i - 1], scale_of(ha, i - 1, hb));
            }
            t[0] = u[3][0];
            t[1] = u[3][1];
            ts = scale_of(ha, 3, hb);
        }
    };
    auto add = [&](auto ha, auto hb) __attribute__((always_inline)) {
        if constexpr (!UNIT) {
            __builtin_amdgcn_sched_barrier(0);
            add_to(c[decltype(ha)::value][decltype(hb)::value][3], t, ts);
        }
    };
    constexpr std::integral_constant<int, 0> zero;
    constexpr std::integral_constant<int, 1> one;
    constexpr int FLIGHT = 4 * L + 1;      // loads of the last 4 panels and scales
    // Tile s, in the stages a0, a1, b0, b1, sc; `a1_next` is the other A1.
    auto tile = [&](char *a0, char *a1, char *b0, char *b1, char *sc, char *a1_next)
                    __attribute__((always_inline)) {
        read_b(zero, b0);
        read_a(a0);
        read_scales(sc);
        load_a1(a1_next);
        add(one, zero);
        stage_sync<FLIGHT>();

        read_b(one, b1);
        if constexpr (!UNIT) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
                both[h] = __int_as_float(__builtin_amdgcn_readfirstlane(
                    __float_as_int(__uint_as_float(sw[h]) * kUp)));
        }
        quadrant(zero, zero);
        add(zero, zero);
        quadrant(zero, one);
        step_sync();

        read_a(a1);
        load_a0_b0(a0, b0, sc);
        add(zero, one);
        stage_sync<FLIGHT>();

        load_b1(b1);
        quadrant(one, one);
        add(one, one);
        quadrant(one, zero);
        stage_wait<FLIGHT>();
        step_sync();
    };

    load_a0_b0(a00, b00, s0);
    __builtin_amdgcn_sched_barrier(0);
    load_b1(b10);
    __builtin_amdgcn_sched_barrier(0);
    load_a1(a10);
    __builtin_amdgcn_sched_barrier(0);
    load_a0_b0(a01, b01, s1);
    __builtin_amdgcn_sched_barrier(0);
    load_b1(b11);
    // A0, B0, B1, A1 and the scales of the first tile
    stage_sync<3 * L + 1>();
    if (wm != 0) __builtin_amdgcn_s_barrier();
    if constexpr (!UNIT) t[0] = t[1] = f32x4{};
    int s = 0;
    for (; s + 2 <= count; s += 2) {
        tile(a00, a10, b00, b10, s0, a11);
        tile(a01, a11, b01, b11, s1, a10);
    }
    if (s < count) tile(a00, a10, b00, b10, s0, a11);
    add(one, zero);
    if (wm == 0) __builtin_amdgcn_s_barrier();
    stage_sync<0>();

    // One array takes a wave's sums of one A panel.
    char *mine = wave < 4 ? (wave < 2 ? (wave < 1 ? a00 : a01) : (wave < 3 ? a10 : a11))
                          : (wave < 6 ? (wave < 5 ? b00 : b01) : (wave < 7 ? b10 : b11));
    if constexpr (!UNIT) {
        bool again = bring_down(c[0]);
        again |= bring_down(c[1]);
        if (again && far_scales<SCALE, true, 256, 256, 32>(wm * 64, wn * 32)) {
            const TileArgs &q = arguments_again().t;
            const Part own(q, 0, 256 * 256);
            grouped_tile32<kGroupWide>(own.tile, q.tiles_m, q.tiles_n, tm, tn);
            const int64_t n = static_cast<int64_t>(tn) * 256 + wn * 32;
#pragma unroll 1
            for (int row = wm * 64; row < 256; row += 128) {
                sums_again<FORMATS, SCALE, false, 256, 256, 32, 4, 2>(mine, row, wn * 32);
                wave_sync();
                epi_rows<T, false, 32, 64>(
                    q, 0, own.sums == nullptr ? nullptr : own.sums + row * 256 + wn * 32, 256, mine,
                    static_cast<int64_t>(tm) * 256 + row, n, n + 128);
                wave_sync();
            }
            return;
        }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        epi_put<32>(mine, c[h][0], 0);
        epi_put<32>(mine, c[h][1], 1);
        wave_sync();
        const int row = h * 128 + wm * 64;
        epi_rows<T, false, 32, 64>(
            a, 0, part.sums == nullptr ? nullptr : part.sums + row * 256 + wn * 32, 256, mine,
            m0 + row, n0 + wn * 32, n1 + wn * 32);
        wave_sync();
    }
}

// ---- the kernel for few rows --------------------------------------------------------------
//
// M <= 16: the weights are read once and nothing else counts.  As linear_few: a workgroup
// of eight waves owns a strip of 16 columns, a wave takes a run of the blocks of K, weights
// go from memory into the MFMA's registers (lane l loads chunks l / 16 and 4 + l / 16 of
// column l % 16), and the waves' sums meet in LDS.
// MAKE: X is of type T and quantized here, by every workgroup for itself, into LDS, while
// its first weights are on their way; for a few thousand elements that takes less than a
// launch of its own.  The bits are those of tra_quantize.  EACH: as in scaled_tile.
// 1 x 12288 x 4096 with binary32 scales: 11.1 us, 4.5 TB/s of weights read.
template <typename T, int FORMATS, int SCALE, bool EACH, bool MAKE>
__global__ __launch_bounds__(512) void scaled_few(const ScaledArgs p) {
    constexpr int WAVES = 8, U = 4;    // U blocks in hand
    constexpr int SIZE = SCALE == TRA_SCALE_E8M0 ? 1 : 4;
    constexpr bool WIDEN = std::is_same_v<T, float>;
    constexpr bool UNIT = SCALE == TRA_SCALE_E8M0 && !WIDEN;
    constexpr uint32_t OUTSIDE = 0x80000000u;
    __shared__ __align__(16) float sums[WAVES][256];
    __shared__ __align__(16) char made[MAKE ? kFewBytes : 16];
    __shared__ uint32_t made_scales[MAKE ? kFewBytes / 128 : 1];
    lds_poison(&sums[0][0], WAVES * 256);
    lds_poison(reinterpret_cast<float *>(made), (MAKE ? kFewBytes : 16) / 4);
    lds_poison(reinterpret_cast<float *>(made_scales), MAKE ? kFewBytes / 128 : 1);
    const TileArgs &a = p.t;
    const int wave = wave_id(), l16 = threadIdx.x & 15, g = (threadIdx.x >> 4) & 3;
    const int M = static_cast<int>(a.M), N = static_cast<int>(a.N), K = static_cast<int>(a.K);
    const int blocks = (K + 127) / 128;
    const int n0 = xcd_remap32(blockIdx.x, gridDim.x) * 16;
    const int own = n0 + l16 < N ? l16 : N - 1 - n0;         // this lane's column of the strip
    const int m = l16 < M ? l16 : M - 1;
    const int each = (blocks + WAVES - 1) / WAVES;
    const int begin = wave * each, end = begin + each < blocks ? begin + each : blocks;

    char *w_at = const_cast<char *>(static_cast<const char *>(a.B[0])) + n0 * a.ldb;
    const __amdgpu_buffer_rsrc_t w_rsrc =
        __builtin_amdgcn_make_buffer_rsrc(w_at, (short)0, 0x7fffffff, 0x00020000);
    const uint32_t w_off = static_cast<uint32_t>(own) * static_cast<uint32_t>(a.ldb) + g * 16;
    const char *x_at = static_cast<const char *>(a.A) + m * a.lda + g * 16;
    const char *sx_at = static_cast<const char *>(p.SX) + m * p.sx_row * SIZE;
    const char *sw_at = static_cast<const char *>(p.SW);
    auto scale_at = [&](const char *at) __attribute__((always_inline)) -> uint32_t {
        if constexpr (SIZE == 1) return *reinterpret_cast<const uint8_t *>(at);
        else return *reinterpret_cast<const uint32_t *>(at);
    };
    // W's scale of the strip's column j, block b
    auto w_scale = [&](int j, int b) __attribute__((always_inline)) {
        const int n = n0 + j < N ? n0 + j : N - 1;
        return scale_at(sw_at + ((n >> p.w_shift) * p.sw_row + b * p.sw_block) * SIZE);
    };

    u32x4 w[U][2];
    uint32_t sw[U], sws[U][4];
    auto load = [&](int b0) __attribute__((always_inline)) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int b = b0 + u;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int k = b * 128 + h * 64 + g * 16;
                const uint32_t at = b < end && k < K ? w_off + b * 128 + h * 64 : OUTSIDE;
                w[u][h] = __builtin_amdgcn_raw_buffer_load_b128(w_rsrc, at, 0, 0);
            }
            const int bb = b < end ? b : end - 1;
            if constexpr (EACH) {
#pragma unroll
                for (int e = 0; e < 4; ++e) sws[u][e] = w_scale(4 * g + e, bb);
            } else {
                sw[u] = w_scale(UNIT ? l16 : 0, bb);
            }
        }
    };
    if (begin < end) load(begin);
    if constexpr (MAKE) {
        for (int i = static_cast<int>(threadIdx.x) >> 4; i < M * blocks; i += 32) {
            const int row = i / blocks, b = i - row * blocks, k = b * 128 + l16 * 8;
            float v[8], most = 0.0f;
            load_part<T, 8>(static_cast<const T *>(a.A) + row * a.lda + k, p.x_cols - k, v);
#pragma unroll
            for (int e = 0; e < 8; ++e) most = fmaxf(most, finite_size(v[e]));
            const BlockScale s = block_scale<TRA_FP8_E4M3, SCALE>(largest_of_16(most));
            uint32_t q[2];
            to_fp8<TRA_FP8_E4M3, SCALE>(v, s, q);
            __builtin_memcpy(__builtin_assume_aligned(made + i * 128 + l16 * 8, 8), q, 8);
            if (l16 == 0) made_scales[i] = s.bits;
        }
        __syncthreads();
    }

    f32x4 c = {};
    auto run = [&](auto careful) __attribute__((always_inline)) {
        constexpr bool CAREFUL = decltype(careful)::value;
        for (int b0 = begin; b0 < end; b0 += U) {
            if (CAREFUL || b0 > begin) load(b0);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int b = b0 + u < end ? b0 + u : end - 1;
                u32x4 x[2];
                uint32_t sx;
                if constexpr (MAKE) {
                    const int at = (m * blocks + b) * 128 + g * 16;
                    x[0] = *reinterpret_cast<const u32x4 *>(made + at);
                    x[1] = *reinterpret_cast<const u32x4 *>(made + at + 64);
                    sx = made_scales[m * blocks + b];
                } else {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        // (past K the weights are zeros, and so are these: they are NaN-free)
                        const int k = b * 128 + h * 64 + g * 16;
                        x[h] = u32x4{};
                        if (k < K)
                            x[h] = *reinterpret_cast<const u32x4 *>(x_at + b * 128 + h * 64);
                    }
                    sx = scale_at(sx_at + b * p.sx_block * SIZE);
                }
                if (b0 + u >= end) continue;
                const i32x8 w8 = __builtin_bit_cast(
                    i32x8, __builtin_shufflevector(w[u][0], w[u][1], 0, 1, 2, 3, 4, 5, 6, 7));
                const i32x8 x8 = __builtin_bit_cast(
                    i32x8, __builtin_shufflevector(x[0], x[1], 0, 1, 2, 3, 4, 5, 6, 7));
                if constexpr (UNIT) {
                    c = mma_scaled<FORMATS>(w8, x8, c, sw[u], sx);
                } else {
                    f32x4 t = {};
                    if constexpr (WIDEN) {
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            t = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                                widen<kFormatW<FORMATS>>(w8, q), widen<kFormatX<FORMATS>>(x8, q), t, 0,
                                0, 0);
                    } else {
                        t = mma_plain<FORMATS>(w8, x8);
                    }
                    const float s = scale_value<SCALE>(sx) * (CAREFUL ? 1.0f : kUp);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float v = scale_value<SCALE>(EACH ? sws[u][e] : sw[u]);
                        c[e] = CAREFUL ? add_scaled(c[e], t[e], s, v) : fmaf(t[e], s * v, c[e]);
                    }
                }
            }
        }
    };
    run(std::false_type{});
    if constexpr (!UNIT) {
        f32x4 sum[1][1][1] = {{{c}}};
        const bool again = bring_down(sum);
        c = sum[0][0][0];
        if (again) {
            float x = 0.0f, y = 0.0f;
            for (int b = begin; b < end; ++b) {
                const uint32_t word = MAKE ? made_scales[m * blocks + b]
                                           : scale_at(sx_at + b * p.sx_block * SIZE);
                x = larger(x, scale_value<SCALE>(word));
                y = larger(y, scale_value<SCALE>(w_scale(l16, b)));
            }
            if (far_scales(x, y)) {
                c = f32x4{};
                run(std::true_type{});
            }
        }
    }

    // Lane l holds token l % 16 of strip columns 4 (l / 16) .. + 3.
#pragma unroll
    for (int r = 0; r < 4; ++r) sums[wave][l16 * 16 + 4 * g + r] = c[r];
    __syncthreads();
    const int i = static_cast<int>(threadIdx.x), row = i / 16, n = n0 + i % 16;
    if (i < 256 && row < M && n < N) {
        float z[1] = {}, none[1];
#pragma unroll
        for (int s = 0; s < WAVES; ++s) z[0] += sums[s][i];
        finish<T, false, TRA_ACT_NONE, 1>(a.epi, 0, row, n, z, none);
    }
}

// ---- launches ----------------------------------------------------------------------------------

template <typename T, int FORMATS, int SCALE, bool EACH = false>
hipError_t launch_scaled(const TilePlan &plan, const ScaledArgs &p, hipStream_t stream) {
    if constexpr (std::is_same_v<T, float> && SCALE == TRA_SCALE_E8M0 && !EACH)
        if (p.w_shift == 0) return launch_scaled<T, FORMATS, SCALE, true>(plan, p, stream);
    const TileArgs &a = p.t;
    const unsigned tiles = static_cast<unsigned>(a.tiles_m) * static_cast<unsigned>(a.tiles_n);
    const unsigned whole = static_cast<unsigned>(a.whole);
    const dim3 grid(whole + (tiles - whole) * static_cast<unsigned>(a.splits));
    if (plan.few) {
        const dim3 strips(static_cast<unsigned>(a.tiles_n));
        if constexpr (FORMATS == kX4W4) {
            if (p.x_cols > 0) {
                scaled_few<T, FORMATS, SCALE, EACH, true><<<strips, 512, 0, stream>>>(p);
                return hipGetLastError();
            }
        }
        scaled_few<T, FORMATS, SCALE, EACH, false><<<strips, 512, 0, stream>>>(p);
        return hipGetLastError();
    }
    if constexpr (sizeof(T) == 2) {
        if (plan.bm == 256) {
            scaled_wide<T, FORMATS, SCALE><<<grid, 512, 0, stream>>>(p);
            return hipGetLastError();
        }
    }
#define TRA_TILE(BM, BN, S) \
    scaled_tile<T, FORMATS, SCALE, EACH, BM, BN, S><<<grid, 256, 0, stream>>>(p)
    if (plan.bm == 128) {
        // (never planned with EACH)
        if constexpr (!EACH) plan.deep ? TRA_TILE(128, 128, 4) : TRA_TILE(128, 128, 2);
        else return hipErrorInvalidValue;
    } else if (plan.bn == 128) {
        plan.deep ? TRA_TILE(64, 128, 4) : TRA_TILE(64, 128, 2);
    } else {
        plan.deep ? TRA_TILE(64, 64, 6) : TRA_TILE(64, 64, 4);
    }
#undef TRA_TILE
    return hipGetLastError();
}

}  // namespace

template <typename T>
hipError_t ScaledKernels<T>::product(const ScaledPlan &plan, const ScaledArgs &p,
                                     hipStream_t stream) {
    const TilePlan &t = plan.tile;
    if (plan.scale == TRA_SCALE_E8M0) {
        switch (plan.formats) {
            case kX4W4: return launch_scaled<T, kX4W4, TRA_SCALE_E8M0>(t, p, stream);
            case kX5: return launch_scaled<T, kX5, TRA_SCALE_E8M0>(t, p, stream);
            default: return launch_scaled<T, kW5, TRA_SCALE_E8M0>(t, p, stream);
        }
    }
    return plan.formats == kX5 ? launch_scaled<T, kX5, TRA_SCALE_F32>(t, p, stream)
                               : launch_scaled<T, kX4W4, TRA_SCALE_F32>(t, p, stream);
}

}  // namespace tra
