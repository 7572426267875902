// scaled.hip -- the C-ABI entry points of products of 8-bit matrices with block scales
// (tra_scaled_linear in include/tra_gemm.h): argument checks, choice of kernels, launches
// on the caller's stream.  Errors come back as status codes; nothing throws across the ABI
// and nothing is allocated: scratch is the caller's workspace.
#include "tra_gemm.h"

#include <cstdio>

#include "linear_join.h"
#include "linear_plan.h"
#include "scaled_plan.h"

namespace {

using namespace tra::host;
using tra::ceil_div;
using tra::ScaledArgs;
using tra::ScaledPlan;

constexpr int64_t kFewBytes = tra::kFewBytes;
constexpr int64_t kMaxPitch = int64_t{1} << 22;      // bytes: a tile's offsets fit 31 bits

int64_t up16(int64_t n) { return ceil_div(n, 16) * 16; }

// How the kernels go, in microseconds (TileClass): 16-bit results with binary32 and e8m0
// scales; binary32 results with a scale for 128 rows of W, and with one for each.
constexpr TileClass kClasses[4][4] = {
    {{256, 256, 1, 1.52, 1.63, 8.0},
     {128, 128, 2, 0.65, 0.49, 5.0},
     {64, 128, 2, 0.41, 0.34, 4.0},
     {64, 64, 2, 0.284, 0.215, 3.5}},
    {{256, 256, 1, 1.34, 1.34, 4.5},
     {128, 128, 2, 0.45, 0.425, 5.0},
     {64, 128, 2, 0.34, 0.33, 3.8},
     {64, 64, 2, 0.242, 0.205, 3.2}},
    {{128, 128, 2, 1.03, 0.87, 9.0},
     {64, 128, 2, 0.635, 0.53, 6.0},
     {64, 64, 2, 0.466, 0.333, 5.0},
     {0, 0, 0, 0.0, 0.0, 0.0}},
    // (128 x 128, one a CU for its VGPRs: 1.29, twice what 64 x 128 takes)
    {{64, 128, 2, 0.85, 0.62, 4.5},
     {64, 64, 2, 0.56, 0.37, 4.0},
     {0, 0, 0, 0.0, 0.0, 0.0},
     {0, 0, 0, 0.0, 0.0, 0.0}}};

// The row of kClasses.
int classes_of(const tra_scaled_args &a) {
    const bool e8m0 = a.scale == TRA_SCALE_E8M0;
    if (a.dtype == TRA_DTYPE_F32) return e8m0 && a.w_block_rows == 1 ? 3 : 2;
    return e8m0 ? 1 : 0;
}

bool x_given(const tra_scaled_args &a) { return a.x_dtype == TRA_X_SCALED; }

ScaledPlan plan_scaled(const tra_scaled_args &a) {
    ScaledPlan s{};
    const int64_t K = up16(a.K), b = elem_bytes(a.dtype);
    const PlanSizes z{a.M, a.N, K, 1, 1, false, 1, static_cast<double>(b), false, true};
    double us = 0.0;
    s.tile = plan_classes(kClasses[classes_of(a)], 4, z, us);
    // Few rows: the weights' bytes at the rate that the strips of 16 columns can ask for.
    if (a.M <= 16) {
        const double strips = static_cast<double>(ceil_div(a.N, 16));
        const double few_us = 2.8 + static_cast<double>(K) * a.N * (1.0 + a.M / 80.0) /
                                        std::min(4.9e6, strips * 2.6e4);
        if (few_us < us) {
            s.tile = tra::TilePlan{};
            s.tile.few = true;
            s.tile.whole = static_cast<int>(strips);
            s.tile.bm = s.tile.bn = 16;
            s.tile.splits = 1;
            // X quantized by every workgroup, 32 blocks at a time, or by a launch before: a CU's
            // rounds of 32 take about 0.6 us each with binary32 scales, the launch 2.5 (4 x 2048
            // x 2048: 5.7 against 7.5 us; 4 x 12288 x 4096, 12 rounds: 18.8 against 15.5).
            const int64_t x_blocks = a.M * ceil_div(a.K, 128);
            s.make = a.x_dtype == a.dtype && a.x_fp8 == TRA_FP8_E4M3 && a.K > 0 &&
                     x_blocks * 128 <= kFewBytes &&
                     ceil_div(x_blocks, 32) * ceil_div(s.tile.whole, kCUs) <= 4;
        }
    }
    s.tile.form = tra::kFormKK;
    s.tile.direct = 16;
    s.formats = a.x_fp8 == TRA_FP8_E5M2   ? tra::kX5
                : a.w_fp8 == TRA_FP8_E5M2 ? tra::kW5
                                          : tra::kX4W4;
    s.scale = a.scale;
    if (!x_given(a) && !s.make) {
        s.ldx = K;
        s.sx_block = a.M;
        s.values_bytes = align_up(static_cast<size_t>(a.M) * static_cast<size_t>(K));
        s.scales_bytes = align_up(static_cast<size_t>(a.M) *
                                  static_cast<size_t>(ceil_div(a.K, 128) * scale_bytes(a.scale)));
    }
    s.total = s.values_bytes + s.scales_bytes + s.tile.partial_bytes;
    return s;
}

// Values the kernels may load: 16-byte aligned rows, offsets that fit.
bool values_ok(const View &v) {
    return v.empty() || (v.valid() && rows16(v.p, v.rows > 1 ? v.ld : 0, 1));
}

tra_status check_scaled(const tra_scaled_args *p) {
    if (p == nullptr) return TRA_ERR_INVALID_ARG;
    const tra_scaled_args &a = *p;
    if (!valid_dtype(a.dtype) || (!x_given(a) && !valid_dtype(a.x_dtype)) || !valid_fp8(a.x_fp8) ||
        !valid_fp8(a.w_fp8) || !valid_scale(a.scale) ||
        (a.w_block_rows != 1 && a.w_block_rows != tra::kScaleBlock) || a.M < 0 || a.N < 0 || a.K < 0)
        return TRA_ERR_INVALID_ARG;
    if (a.scale == TRA_SCALE_F32 && a.w_block_rows == 1) return TRA_ERR_INVALID_ARG;
    if (a.w_fp8 == TRA_FP8_E5M2 &&
        (a.x_fp8 == TRA_FP8_E5M2 || a.scale == TRA_SCALE_F32 || !x_given(a)))
        return TRA_ERR_INVALID_ARG;
    if (a.M == 0 || a.N == 0) return TRA_OK;
    if (a.M > kMaxSize || a.N > kMaxSize || a.K > kMaxSize) return TRA_ERR_UNSUPPORTED;
    const int64_t b = elem_bytes(a.dtype), sb = scale_bytes(a.scale);
    const int64_t K = up16(a.K), KB = ceil_div(a.K, 128), NB = ceil_div(a.N, a.w_block_rows);
    const View X = x_given(a) ? View{a.X, a.M, K, a.ldx, 1}
                              : View{a.X, a.M, a.K, a.ldx, elem_bytes(a.x_dtype)};
    const View W{a.W, a.N, K, a.ldw, 1};
    const View SX = x_given(a) ? scale_view(a.SX, a.M, KB, a.sx_row, a.sx_block, sb) : View{};
    const View SW = scale_view(a.SW, NB, KB, a.sw_row, a.sw_block, sb);
    const View bias{a.bias, a.bias != nullptr, a.N, a.N, b};
    const View R{a.R, a.R != nullptr ? a.M : 0, a.N, a.ldr, b};
    const View Y{a.Y, a.M, a.N, a.ldy, b};
    const View in[] = {X, W, SX, SW, bias, R};
    for (const View &v : in)
        if (!v.valid()) return TRA_ERR_INVALID_ARG;
    if (!values_ok(W) || (x_given(a) && !values_ok(X)) || !Y.valid()) return TRA_ERR_INVALID_ARG;
    // R in place: the lane that reads an element of R writes it, and no other.
    for (const View &v : in) {
        const bool in_place = &v == &in[5] && same(R, Y);
        if (share(v, Y) && !in_place) return TRA_ERR_INVALID_ARG;
    }
    // offsets of a tile's rows, of values and of scales
    if (K >= kMaxPitch || (a.N > 1 && a.ldw >= kMaxPitch) ||
        (x_given(a) && a.M > 1 && a.ldx >= kMaxPitch) || (NB > 1 && a.sw_row * sb >= kMaxPitch) ||
        (x_given(a) && a.M > 1 && a.sx_row * sb >= kMaxPitch))
        return TRA_ERR_UNSUPPORTED;
    if (!x_given(a) && ceil_div(a.M, 128) * KB > tra::kMaxGridLanes / 256)
        return TRA_ERR_UNSUPPORTED;
    return TRA_OK;
}

hipError_t run_product(int dtype, const ScaledPlan &s, const ScaledArgs &p, hipStream_t st) {
    switch (dtype) {
        case TRA_DTYPE_F32: return tra::ScaledKernels<float>::product(s, p, st);
        case TRA_DTYPE_BF16: return tra::ScaledKernels<__bf16>::product(s, p, st);
        default: return tra::ScaledKernels<_Float16>::product(s, p, st);
    }
}

hipError_t run_join(int dtype, const ScaledPlan &s, const ScaledArgs &p, hipStream_t st) {
    switch (dtype) {
        case TRA_DTYPE_F32: return tra::launch_join<float>(s.tile, p.t, st);
        case TRA_DTYPE_BF16: return tra::launch_join<__bf16>(s.tile, p.t, st);
        default: return tra::launch_join<_Float16>(s.tile, p.t, st);
    }
}

tra_status scaled_linear(const tra_scaled_args *p, void *stream) {
    tra_status st = check_scaled(p);
    if (st != TRA_OK || p->M == 0 || p->N == 0) return st;
    const tra_scaled_args &a = *p;
    const ScaledPlan s = plan_scaled(a);
    if (!workspace_ok(a.workspace, a.workspace_bytes, s.total)) return TRA_ERR_INVALID_ARG;
    char *ws = static_cast<char *>(a.workspace);
    ScaledArgs d{};
    d.t.A = a.X;
    d.t.lda = a.ldx;
    d.SX = a.SX;
    d.sx_row = a.sx_row;
    d.sx_block = a.sx_block;
    d.t.B[0] = d.t.B[1] = a.W;
    d.t.ldb = a.ldw;
    d.SW = a.SW;
    d.sw_row = a.sw_row;
    d.sw_block = a.sw_block;
    d.w_shift = a.w_block_rows == 1 ? 0 : 7;
    d.t.M = a.M;
    d.t.N = a.N;
    d.t.K = up16(a.K);
    d.t.segs = d.t.batch = 1;
    d.t.epi.bias = a.bias;
    d.t.epi.R = a.R;
    d.t.epi.ldr = a.ldr;
    d.t.epi.Y[0] = a.Y;
    d.t.epi.ldy = a.ldy;
    d.t.epi.act = TRA_ACT_NONE;
    if ((st = finish_tile_args(
             s.tile, 128, d.t,
             reinterpret_cast<float *>(ws + s.values_bytes + s.scales_bytes))) != TRA_OK)
        return st;
    if (s.make) {
        d.x_cols = static_cast<int>(a.K);
    } else if (!x_given(a) && a.K > 0) {
        tra_quantize_args q{};
        q.dtype = a.x_dtype;
        q.fp8 = a.x_fp8;
        q.scale = a.scale;
        q.block_rows = 1;
        q.M = a.M;
        q.K = a.K;
        q.X = a.X;
        q.ldx = a.ldx;
        d.t.A = q.Q = ws;
        d.t.lda = q.ldq = s.ldx;
        d.SX = q.S = ws + s.values_bytes;
        d.sx_row = q.ss_row = 1;
        d.sx_block = q.ss_block = s.sx_block;
        if ((st = tra_quantize(&q, stream)) != TRA_OK) return st;
    }
    const hipStream_t hs = static_cast<hipStream_t>(stream);
    hipError_t err = run_product(a.dtype, s, d, hs);
    if (err == hipSuccess && s.tile.splits > 1) err = run_join(a.dtype, s, d, hs);
    return status_of(err);
}

}  // namespace

extern "C" {

tra_status tra_scaled_linear(const tra_scaled_args *args, void *stream) {
    return scaled_linear(args, stream);
}

tra_status tra_scaled_linear_workspace_size(const tra_scaled_args *args, size_t *bytes) {
    const tra_status st = check_scaled(args);
    if (st != TRA_OK || bytes == nullptr) return st != TRA_OK ? st : TRA_ERR_INVALID_ARG;
    *bytes = args->M == 0 || args->N == 0 ? 0 : plan_scaled(*args).total;
    return TRA_OK;
}

tra_status tra_scaled_linear_describe(const tra_scaled_args *args, char *buf, size_t len) {
    const tra_status st = check_scaled(args);
    if (st != TRA_OK) return st;
    if (buf == nullptr) return len == 0 ? TRA_OK : TRA_ERR_INVALID_ARG;
    if (len == 0) return TRA_OK;
    if (args->M == 0 || args->N == 0) {
        std::snprintf(buf, len, "kernel=none");
        return TRA_OK;
    }
    const ScaledPlan s = plan_scaled(*args);
    const tra::TilePlan &t = s.tile;
    // quantizes: 0 nothing, 1 in the kernel, 2 in a launch before it
    std::snprintf(buf, len,
                  "kernel=%s tile=%dx%d deep=%d whole=%d splits=%d quantizes=%d workspace_bytes=%zu",
                  t.few ? "scaled_few" : t.bm == 256 ? "scaled_wide" : "scaled_tile", t.bm, t.bn,
                  t.deep, t.whole, t.splits, s.make ? 1 : x_given(*args) ? 0 : 2, s.total);
    return TRA_OK;
}

}  // extern "C"
