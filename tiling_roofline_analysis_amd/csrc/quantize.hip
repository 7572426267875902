// quantize.hip -- matrices to 8-bit floating point with a scale for each block of 128
// (tra_quantize in include/tra_gemm.h).
//
// A workgroup takes a tile of 128 x 128: the blocks of every form lie in it as a whole, so
// X is read once, whichever forms are asked for.  A lane holds 8 rows by 8 columns of
// the tile: a row's block is 16 lanes' (their largest by DPP), a column's is the tile's
// 16 groups of lanes' (theirs through LDS), and a lane's 8 rows of one column are 8
// consecutive bytes of the transposed form, which is put together in LDS and leaves in
// lines of 128 bytes.  Memory bounds it: 8192 x 4096 bf16 to both forms with e8m0 scales 29 us
// (4.6 TB/s); with binary32 scales, whose exact quotients cost five steps an element, also
// the vector units (rows of 8192 x 8192 bf16: 48 us, with e8m0 scales 35).
#include "tra_gemm.h"

#include "scaled_internal.h"

namespace tra {
namespace {

struct QuantizeArgs {
    int64_t M, K, tiles_k;
    const void *X;
    int64_t ldx;
    uint8_t *Q;
    int64_t ldq;
    void *S;
    int64_t ss_row, ss_block;
    uint8_t *QT;
    int64_t ldqt;
    void *ST;
    int64_t sts_row, sts_block;
};

template <int SCALE>
__device__ __forceinline__ void store_scale(void *S, int64_t at, uint32_t bits) {
    if constexpr (SCALE == TRA_SCALE_E8M0)
        static_cast<uint8_t *>(S)[at] = static_cast<uint8_t>(bits);
    else
        static_cast<uint32_t *>(S)[at] = bits;
}

__device__ __forceinline__ int64_t up16(int64_t n) { return (n + 15) / 16 * 16; }

// The 8 bytes of column k, rows 8 g .. + 7, of the transposed tile in LDS.  A write's
// lanes have 16 columns 8 apart: the pieces of a column's 128 bytes are XORed by k / 8.
__device__ __forceinline__ int piece(int k, int g) { return k * 128 + ((g ^ (k >> 3)) << 3); }

template <typename T, int FP8, int SCALE, int ROWS>
__global__ __launch_bounds__(256) void quantize_tile(const QuantizeArgs p) {
    __shared__ __align__(16) uint8_t tile[128 * 128];
    __shared__ float part[16][128];
    __shared__ float most[128];
    lds_poison(reinterpret_cast<float *>(tile), 128 * 32);
    lds_poison(&part[0][0], 16 * 128);
    lds_poison(most, 128);
    const int t = static_cast<int>(threadIdx.x), c = t & 15, g = t >> 4;
    const int64_t tm = blockIdx.x / p.tiles_k, tk = blockIdx.x - tm * p.tiles_k;
    const int64_t m0 = tm * 128, k0 = tk * 128;
    const int64_t k = k0 + c * 8, m = m0 + g * 8;

    float x[8][8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const T *row = static_cast<const T *>(p.X) + (m + i) * p.ldx + k;
        load_part<T, 8>(row, m + i < p.M ? p.K - k : 0, x[i]);
    }

    BlockScale s;
    if constexpr (ROWS != 1) {
        float a = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) a = fmaxf(a, finite_size(x[i][j]));
        a = largest_of_16(a);
        if (c == 0) most[g] = a;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 16; ++i) a = fmaxf(a, most[i]);
        s = block_scale<FP8, SCALE>(a);
        if (t == 0) {
            if (p.Q != nullptr) store_scale<SCALE>(p.S, tm * p.ss_row + tk * p.ss_block, s.bits);
            if (p.QT != nullptr)
                store_scale<SCALE>(p.ST, tk * p.sts_row + tm * p.sts_block, s.bits);
        }
    }

    if (p.Q != nullptr) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            // (the 16 lanes of a row go the same way; of a few rows' tile most do nothing)
            if (m + i >= p.M) continue;
            if constexpr (ROWS == 1) {
                float a = 0.0f;
#pragma unroll
                for (int j = 0; j < 8; ++j) a = fmaxf(a, finite_size(x[i][j]));
                s = block_scale<FP8, SCALE>(largest_of_16(a));
                if (c == 0) most[g * 8 + i] = __uint_as_float(s.bits);
            }
            uint32_t w[2];
            to_fp8<FP8, SCALE>(x[i], s, w);
            if (k < up16(p.K))
                __builtin_memcpy(__builtin_assume_aligned(p.Q + (m + i) * p.ldq + k, 8), w, 8);
        }
        if constexpr (ROWS == 1) {
            __syncthreads();
            if (t < 128 && m0 + t < p.M)
                store_scale<SCALE>(p.S, (m0 + t) * p.ss_row + tk * p.ss_block,
                                   __float_as_uint(most[t]));
        }
    }

    if (p.QT != nullptr) {
        if constexpr (ROWS == 1) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                float a = 0.0f;
#pragma unroll
                for (int i = 0; i < 8; ++i) a = fmaxf(a, finite_size(x[i][j]));
                part[g][c * 8 + j] = a;
            }
            __syncthreads();
            if (t < 128) {
                float a = 0.0f;
#pragma unroll
                for (int i = 0; i < 16; ++i) a = fmaxf(a, part[i][t]);
                part[0][t] = a;
                if (k0 + t < p.K)
                    store_scale<SCALE>(p.ST, (k0 + t) * p.sts_row + tm * p.sts_block,
                                       block_scale<FP8, SCALE>(a).bits);
            }
            __syncthreads();
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            float y[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = x[i][j];
            if constexpr (ROWS == 1) s = block_scale<FP8, SCALE>(part[0][c * 8 + j]);
            uint32_t w[2];
            to_fp8<FP8, SCALE>(y, s, w);
            __builtin_memcpy(tile + piece(c * 8 + j, g), w, 8);
        }
        __syncthreads();
        // 16 bytes a lane: two pieces of a column
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int n = i * 32 + (t >> 3), two = (t & 7) * 2;
            u32x4 v;
            __builtin_memcpy(&v, tile + piece(n, two), 8);
            __builtin_memcpy(reinterpret_cast<char *>(&v) + 8, tile + piece(n, two + 1), 8);
            if (k0 + n < p.K && m0 + two * 8 < up16(p.M))
                *reinterpret_cast<u32x4 *>(p.QT + (k0 + n) * p.ldqt + m0 + two * 8) = v;
        }
    }
}

// Rows alone, a block for each 16 lanes, blocks of one column of them next to each other:
// for matrices whose tiles would leave CUs idle.  A lane of the tile kernel rounds 64
// elements one after the other, which takes 2 to 6 us however few there are: 16 x 512 bf16 to
// binary32 scales 9.1 us in tiles, 2.6 this way, 1024 x 4096 8.2 and 5.6.  With e8m0 scales
// the two are alike from 512 tiles on (2048 x 4096 bf16 6.5 us in tiles, 7.1 this way,
// 4096 x 8192 19.7 and 22.3), with binary32 scales from 2048 on (2048 x 4096 10.1 and 9.3,
// 4096 x 4096 17.6 and 15.5, 8192 x 8192 48 and 50).
template <typename T, int FP8, int SCALE>
__global__ __launch_bounds__(256) void quantize_rows(const QuantizeArgs p) {
    const int64_t id = static_cast<int64_t>(blockIdx.x) * 16 + (threadIdx.x >> 4);
    if (id >= p.M * p.tiles_k) return;
    const int64_t b = id / p.M, m = id - b * p.M;
    const int c = static_cast<int>(threadIdx.x & 15);
    const int64_t k = b * 128 + c * 8;
    float x[8], most = 0.0f;
    load_part<T, 8>(static_cast<const T *>(p.X) + m * p.ldx + k, p.K - k, x);
#pragma unroll
    for (int e = 0; e < 8; ++e) most = fmaxf(most, finite_size(x[e]));
    const BlockScale s = block_scale<FP8, SCALE>(largest_of_16(most));
    uint32_t w[2];
    to_fp8<FP8, SCALE>(x, s, w);
    if (k < up16(p.K))
        __builtin_memcpy(__builtin_assume_aligned(p.Q + m * p.ldq + k, 8), w, 8);
    if (c == 0) store_scale<SCALE>(p.S, m * p.ss_row + b * p.ss_block, s.bits);
}

template <typename T, int FP8, int SCALE>
hipError_t launch_rows(int block_rows, unsigned tiles, const QuantizeArgs &a, hipStream_t s) {
    if (block_rows == 1 && a.QT == nullptr &&
        tiles < (SCALE == TRA_SCALE_F32 ? 2048u : 512u)) {
        const unsigned groups = static_cast<unsigned>(ceil_div(a.M * a.tiles_k, 16));
        quantize_rows<T, FP8, SCALE><<<dim3(groups), 256, 0, s>>>(a);
        return hipGetLastError();
    }
    if (block_rows == 1)
        quantize_tile<T, FP8, SCALE, 1><<<dim3(tiles), 256, 0, s>>>(a);
    else
        quantize_tile<T, FP8, SCALE, 128><<<dim3(tiles), 256, 0, s>>>(a);
    return hipGetLastError();
}

template <typename T>
hipError_t launch_quantize(const tra_quantize_args &q, unsigned tiles, const QuantizeArgs &a,
                           hipStream_t s) {
    const bool e8m0 = q.scale == TRA_SCALE_E8M0;
    if (q.fp8 == TRA_FP8_E4M3)
        return e8m0 ? launch_rows<T, TRA_FP8_E4M3, TRA_SCALE_E8M0>(q.block_rows, tiles, a, s)
                    : launch_rows<T, TRA_FP8_E4M3, TRA_SCALE_F32>(q.block_rows, tiles, a, s);
    return e8m0 ? launch_rows<T, TRA_FP8_E5M2, TRA_SCALE_E8M0>(q.block_rows, tiles, a, s)
                : launch_rows<T, TRA_FP8_E5M2, TRA_SCALE_F32>(q.block_rows, tiles, a, s);
}

}  // namespace
}  // namespace tra

namespace {

using namespace tra::host;
using tra::ceil_div;

int64_t up16(int64_t n) { return ceil_div(n, 16) * 16; }

tra_status check_quantize(const tra_quantize_args *p) {
    if (p == nullptr) return TRA_ERR_INVALID_ARG;
    const tra_quantize_args &a = *p;
    if (!valid_dtype(a.dtype) || !valid_fp8(a.fp8) || !valid_scale(a.scale) ||
        (a.block_rows != 1 && a.block_rows != tra::kScaleBlock) || a.M < 0 || a.K < 0)
        return TRA_ERR_INVALID_ARG;
    if (a.M == 0 || a.K == 0) return TRA_OK;
    if (a.Q == nullptr && a.QT == nullptr) return TRA_ERR_INVALID_ARG;
    if (a.M > kMaxSize || a.K > kMaxSize ||
        ceil_div(a.M, 128) * ceil_div(a.K, 128) > tra::kMaxGridLanes / 256)
        return TRA_ERR_UNSUPPORTED;
    const View X{a.X, a.M, a.K, a.ldx, elem_bytes(a.dtype)};
    if (!X.valid()) return TRA_ERR_INVALID_ARG;
    const int64_t sb = scale_bytes(a.scale), br = a.block_rows;
    View out[4] = {};
    if (a.Q != nullptr) {
        out[0] = View{a.Q, a.M, up16(a.K), a.ldq, 1};
        out[1] = scale_view(a.S, ceil_div(a.M, br), ceil_div(a.K, 128), a.ss_row, a.ss_block, sb);
    }
    if (a.QT != nullptr) {
        out[2] = View{a.QT, a.K, up16(a.M), a.ldqt, 1};
        out[3] = scale_view(a.ST, ceil_div(a.K, br), ceil_div(a.M, 128), a.sts_row, a.sts_block, sb);
    }
    for (int i = 0; i < 4; ++i) {
        if (!out[i].valid() || share(out[i], X)) return TRA_ERR_INVALID_ARG;
        if (i % 2 == 0 && !out[i].empty() && !rows16(out[i].p, out[i].ld, 1))
            return TRA_ERR_INVALID_ARG;
        for (int j = 0; j < i; ++j)
            if (share(out[i], out[j])) return TRA_ERR_INVALID_ARG;
    }
    return TRA_OK;
}

}  // namespace

extern "C" {

tra_status tra_quantize(const tra_quantize_args *args, void *stream) {
    const tra_status st = check_quantize(args);
    if (st != TRA_OK || args->M == 0 || args->K == 0) return st;
    const tra_quantize_args &a = *args;
    tra::QuantizeArgs d{a.M,  a.K,      ceil_div(a.K, 128),
                        a.X,  a.ldx,    static_cast<uint8_t *>(a.Q),
                        a.ldq, a.S,     a.ss_row,
                        a.ss_block,     static_cast<uint8_t *>(a.QT),
                        a.ldqt, a.ST,   a.sts_row,
                        a.sts_block};
    const unsigned tiles = static_cast<unsigned>(ceil_div(a.M, 128) * d.tiles_k);
    const hipStream_t s = static_cast<hipStream_t>(stream);
    switch (a.dtype) {
        case TRA_DTYPE_F32: return status_of(tra::launch_quantize<float>(a, tiles, d, s));
        case TRA_DTYPE_BF16: return status_of(tra::launch_quantize<__bf16>(a, tiles, d, s));
        default: return status_of(tra::launch_quantize<_Float16>(a, tiles, d, s));
    }
}

}  // extern "C"
