// linear_internal.h -- internal interface of the fused linear operators:
// between their C-ABI entry points (linear.hip) and the kernels, which are
// built once per element type (linear_f32.hip, linear_bf16.hip,
// linear_f16.hip).  Not part of the ABI.
#pragma once

#include <hip/hip_runtime.h>

#include <cstddef>
#include <cstdint>

#include "tra_gemm.h"

namespace tra {

// What happens to a product's elements on their way to memory:
//   y = act(z + bias) + R              (plain)
//   y = act(z) * u                     (gated: z and u from the two weights)
// with z (and u) also kept in binary32 when Z is set.
struct EpiArgs {
    const void *bias;      // N elements, or null
    const void *R;         // residual, or null
    int64_t ldr;
    void *Y[2];            // by batch index
    int64_t ldy;
    float *Z;              // kept pre-activations: z at column n, u at column N + n; or null
    int64_t ldz;
    const float *undo;     // binary16 gradients: what their sums are multiplied by, or null
    int64_t M, N;
    int act;
};

// One product  P = op(A) x op(B)  on tiles, A's rows and B's columns being
// the rows and columns of P, contracted over K.  An operand is "k-contiguous"
// when consecutive k are adjacent in memory (row m of A at A + m * lda), else
// its rows (columns of P) are adjacent (slice k of A at A + k * lda).
// With `segs` = 2 the contraction runs over two pairs of operands:
// (A, B[0]) and (A + a_seg, B[1]).  Gated: B[0] gives z, B[1] gives u.  With
// `batch` = 2, batch 1 uses A + a_batch and B[0] + b_batch.
struct TileArgs {
    const void *A;
    int64_t lda;
    const void *B[2];
    int64_t ldb;
    int64_t a_seg, a_batch, b_batch;    // elements
    int64_t M, N, K;                    // K of one segment
    int segs, batch;
    int tiles_m, tiles_n;
    int seg_tiles;                      // K tiles of one segment
    int k_tiles;                        // K tiles in all
    // Tiles 0 .. whole - 1 of each batch are computed whole.  Each of the others is
    // split along K into `splits` parts of tiles_per_split K tiles, whose sums go to
    // partial: [batch][tile - whole][split][bm][bn] (gated: bn / 2 of z, then of u).
    int whole;
    int splits, tiles_per_split;
    float *partial;
    EpiArgs epi;
};

// Forms of the operands: {A, B} k-contiguous or not.  Every product the
// operators need is one of these three.
enum TileForm {
    kFormKK = 0,     // X W^T: W stored N x K; dZ W^T: W stored K x N
    kFormKN = 1,     // X W:   W stored K x N; dZ W:   W stored N x K
    kFormNN = 2      // X^T dZ, dZ^T X: both contracted over rows
};

struct TilePlan {
    TileForm form;
    bool gated;
    bool few;              // the kernel for few rows; bn: columns per workgroup
    int bm, bn;            // tile of P (gated: bn / 2 columns of each of z, u)
    int direct;            // bytes a lane of loads straight into LDS, or 0: through registers
    bool deep;             // direct: one workgroup a CU, with more stages
    int whole;             // tiles of a batch not split along K (all when splits is 1)
    int splits;
    size_t partial_bytes;  // workspace of the split
};

// Stages of LDS that the tile kernel of a plan keeps (launch_tile): with direct loads of
// 16 bytes two workgroups' worth, or, deep, one workgroup's.
inline int plan_stages(const TilePlan &t) {
    if (t.few) return 0;
    if (t.bm == 256 || t.direct == 0) return 2;
    if (t.direct == 4) return 3;
    return t.bm == 128 ? (t.deep ? 4 : 2) : t.deep ? 6 : 3;
}

// Tile rows swept together by the tile kernels (grouped_tile32), by tile height.
constexpr int kGroupTile = 8, kGroupWide = 4;

// Gradient of the epilogue, element by element: dZ = dY * act'(Z), or, gated,
// dG | dU = dH * u * act'(g) | dH * act(g) from the kept [g | u]; and the
// column sums of dZ (the bias gradient) over chunks of rows.
struct SlopeArgs {
    const void *dY;
    int64_t lddy;
    const float *Z;        // null when act is TRA_ACT_NONE (plain only)
    int64_t ldz;
    void *dZ;              // null: only the column sums are wanted
    int64_t lddz;
    float *colsum;         // [row chunk][N], or null
    // Binary16 with dZ: the largest finite |dZ| of each workgroup, and what the
    // products' sums are multiplied by to undo dZ's scale.
    float *largest, *undo;
    int64_t M, N;
    int rows_per_chunk;
    int act;
};

template <typename T>
struct LinearKernels {
    static hipError_t tile(const TilePlan &plan, const TileArgs &a, hipStream_t stream);
};

}  // namespace tra
