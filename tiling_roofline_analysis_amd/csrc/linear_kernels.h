// linear_kernels.h -- kernels of the fused linear operators, for one element
// type T (float, __bf16 or _Float16).  Included once by each linear_<type>.hip.
//
// The product runs on 16 x 16 MFMA tiles whose K step is one 16-byte chunk per
// lane: 8 elements of 16 bits (v_mfma_f32_16x16x32) or 4 floats (four
// v_mfma_f32_16x16x4_f32).  A lane holds row l % 16 and chunk l / 16 of each
// operand, so all three types move the same bytes through the same addresses
// and only the instruction differs.  The weight operand goes in the first
// place, which makes a lane's four results four consecutive columns of one row.
// All sums are binary32.
#pragma once

#include <type_traits>

#include "linear_epilogue.h"

namespace tra {
namespace {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

#define TRA_LDS(type) __attribute__((address_space(3))) type

template <typename T>
constexpr int kSlice = 128 / sizeof(T);    // K tile: 8 chunks, two MFMA steps

__device__ __forceinline__ int wave_id() {
    return __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x >> 6));
}

// The end of a stage: this wave's direct loads older than its last VM are in
// LDS and its LDS reads are done; then the workgroup barrier.  (__syncthreads
// would wait for every load in flight.)  s_waitcnt's gfx9 encoding: vmcnt in
// bits 3:0 and 15:14, expcnt 6:4 (not waited for), lgkmcnt 11:8.  The empty asm
// keeps the compiler from moving memory accesses across it.
template <int VM>
__device__ __forceinline__ void stage_sync() {
    static_assert(VM >= 0 && VM < 64, "vmcnt range");
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt((VM & 15) | ((VM >> 4) << 14) | (7 << 4));
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}

// ---- MFMA ----------------------------------------------------------------------

// One chunk of K: c += w x^T on a 16 x 16 tile; lane l holds row l % 16, chunk
// l / 16 of each operand, and gets column l % 16, rows 4 (l / 16) .. + 3 of c.
template <typename T>
__device__ __forceinline__ f32x4 mma16(u32x4 w, u32x4 x, f32x4 c) {
    if constexpr (std::is_same_v<T, __bf16>)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, w),
                                                       __builtin_bit_cast(bf16x8, x), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, w),
                                                      __builtin_bit_cast(f16x8, x), c, 0, 0, 0);
}

// All tiles of one chunk step: TI row tiles of x times TJ column tiles of w.
// binary32: four steps of 4; the step is the outer loop, so that consecutive
// MFMAs add to different tiles.
template <typename T, int TI, int TJ>
__device__ __forceinline__ void mma_step(const u32x4 (&x)[TI], const u32x4 (&w)[TJ],
                                         f32x4 (&c)[TI][TJ]) {
    if constexpr (std::is_same_v<T, float>) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int i = 0; i < TI; ++i)
#pragma unroll
                for (int j = 0; j < TJ; ++j)
                    c[i][j] = __builtin_amdgcn_mfma_f32_16x16x4f32(
                        __uint_as_float(w[j][e]), __uint_as_float(x[i][e]), c[i][j], 0, 0, 0);
    } else {
#pragma unroll
        for (int i = 0; i < TI; ++i)
#pragma unroll
            for (int j = 0; j < TJ; ++j) c[i][j] = mma16<T>(w[j], x[i], c[i][j]);
    }
}

// ---- operands in LDS --------------------------------------------------------------
//
// A panel is ROWS rows (of A, or columns of P for B) by one K tile, ROWS * 128
// bytes, moved as 1 KB blocks: lane l of a wave supplies bytes 16 l .. + 15 of a
// block.  k-contiguous (KC): 128 bytes per row, else ROWS elements per k.
// Inside each line the 16-byte chunks are XORed so that the fragment reads of
// one instruction spread over all 64 banks (256 bytes):
//   KC    16 rows at one chunk: rows r, r + 1 fill the two halves of 256 bytes,
//         chunk ^ (r >> 1);
//   else  16 bits: 32 lanes of a transposing read take 32 bytes from each of
//         the 8 slices k = 0..3, 8..11; 32 bits: 64 bytes from each of the
//         slices k = 0, 4, 8, 12.
// Which global chunk a lane moves follows from that; a line's bytes still
// come from consecutive lanes.
template <typename T, bool KC, int ROWS, int WAVES>
struct Panel {
    static constexpr int BYTES = ROWS * 128;
    static constexpr int LINE = KC ? 128 : ROWS * static_cast<int>(sizeof(T));
    static constexpr int CPL = LINE / 16;             // chunks per line
    static constexpr int LPB = 1024 / LINE;           // lines per block
    static constexpr int INS = BYTES / 1024 / WAVES;  // blocks per wave
    static_assert(LINE <= 1024 && BYTES % (1024 * WAVES) == 0, "every wave moves whole blocks");

    static __device__ __forceinline__ int swizzle(int line) {
        if constexpr (KC) return (line >> 1) & 7;
        if constexpr (sizeof(T) == 4) return ((line >> 2) & 3) << 2;
        if constexpr (LINE == 128) return (((line >> 1) & 1) | (((line >> 3) & 1) << 1)) << 1;
        return ((line & 3) | (((line >> 3) & 1) << 2)) << 1;
    }

    // Line and chunk (inside its line) that this lane moves in its wave's
    // block i.
    static __device__ __forceinline__ int line(int i) {
        return (wave_id() + i * WAVES) * LPB + static_cast<int>(threadIdx.x & 63) / CPL;
    }
    static __device__ __forceinline__ int chunk(int i) {
        return (static_cast<int>(threadIdx.x & 63) % CPL) ^ swizzle(line(i));
    }
    static __device__ __forceinline__ int lds_block(int i) { return (wave_id() + i * WAVES) * 1024; }

    // -- direct loads (buffer_load_dwordx4 .. lds): rows and K tile are whole
    // chunks, bytes outside read as zero because their offset lies past the
    // buffer's length.
    static constexpr uint32_t OUTSIDE = 0x80000000u;

    // Offset of this lane's chunk of block i from the panel's corner, or
    // OUTSIDE where the panel's `rows` rows inside the matrix end before it.
    static __device__ __forceinline__ uint32_t offset(int i, int64_t rows, int64_t ld) {
        const int r = KC ? line(i) : chunk(i) * kChunk<T>;
        const uint32_t at = static_cast<uint32_t>(line(i)) * static_cast<uint32_t>(ld * sizeof(T)) +
                            static_cast<uint32_t>(chunk(i)) * 16u;
        return r < rows ? at : OUTSIDE;
    }

    // Loads the panel at `base` (its corner, wave-uniform) into `lds`.  `rem`
    // slices of K are inside (none when rem <= 0: zeros, and no memory is read).
    // Always INS loads and no branch, so that the number of loads in flight is
    // the same on every path: where it is not, the compiler waits for all of them
    // before a fragment read.
    static __device__ __forceinline__ void load_direct(const char *base, int64_t ld,
                                                       const uint32_t (&off)[INS], int64_t rem,
                                                       char *lds) {
        int length = 0x7fffffff;
        if constexpr (!KC) {
            // slices past the last lie past the buffer's end
            if (rem < kSlice<T>)
                length = rem > 0 ? static_cast<int>(rem * ld * static_cast<int64_t>(sizeof(T))) : 0;
        }
        const __amdgpu_buffer_rsrc_t rsrc =
            __builtin_amdgcn_make_buffer_rsrc((void *)base, (short)0, length, 0x00020000);
#pragma unroll
        for (int i = 0; i < INS; ++i) {
            const uint32_t at = KC && chunk(i) * kChunk<T> >= rem ? OUTSIDE : off[i];
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, lds + lds_block(i), 16, at, 0, 0, 0);
        }
    }

    // -- through registers: any alignment.  A panel that lies inside loads
    // 16 bytes a lane at element alignment; else element by element.
    static __device__ __forceinline__ void fetch(const char *base, int64_t ld, int64_t rows,
                                                 int64_t rem, u32x4 (&reg)[INS]) {
        if (rows >= ROWS && rem >= kSlice<T>) {
#pragma unroll
            for (int i = 0; i < INS; ++i)
                __builtin_memcpy(&reg[i],
                                 base + line(i) * (ld * static_cast<int64_t>(sizeof(T))) +
                                     chunk(i) * 16,
                                 16);
        } else {
#pragma unroll
            for (int i = 0; i < INS; ++i) {
                const int64_t lines = KC ? rows : rem;
                const int64_t left = (KC ? rem : rows) - chunk(i) * kChunk<T>;
                const T *p = reinterpret_cast<const T *>(base) + line(i) * ld +
                             chunk(i) * kChunk<T>;
                T t[kChunk<T>];
#pragma unroll
                for (int e = 0; e < kChunk<T>; ++e)
                    t[e] = line(i) < lines && e < left ? p[e] : static_cast<T>(0.0f);
                __builtin_memcpy(&reg[i], t, 16);
            }
        }
    }
    static __device__ __forceinline__ void store(const u32x4 (&reg)[INS], char *lds) {
#pragma unroll
        for (int i = 0; i < INS; ++i)
            *reinterpret_cast<u32x4 *>(lds + lds_block(i) + (threadIdx.x & 63) * 16) = reg[i];
    }

    // -- fragments: rows row0 .. + 15 (a multiple of 16), MFMA step `step`, of the
    // panel `panel` bytes into the stage `st`.  Each address is one offset from
    // the stage's array: past a few steps of pointer arithmetic the compiler
    // forgets which array a read is from, and waits for every direct load in
    // flight before it.
    static __device__ __forceinline__ u32x4 fragment(const char *st, int panel, int row0,
                                                     int step) {
        const int l16 = threadIdx.x & 15, g = (threadIdx.x >> 4) & 3;
        if constexpr (KC) {
            const int at = panel + (row0 + l16) * 128 + (((4 * step + g) ^ (l16 >> 1)) << 4);
            return *reinterpret_cast<const u32x4 *>(st + at);
        } else if constexpr (sizeof(T) == 4) {
            u32x4 v;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int k = 16 * step + 4 * g + e;
                const int c = ((row0 + l16) >> 2) ^ (g << 2);
                const int at = panel + k * LINE + c * 16 + (l16 & 3) * 4;
                v[e] = *reinterpret_cast<const uint32_t *>(st + at);
            }
            return v;
        } else {
            // ds_read_b64_tr_b16: 16 lanes address 4 slices of 16 elements,
            // 8 bytes a lane; lane i gets element i of each.
            u32x4 v;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int k = 32 * step + 8 * g + 4 * h + (l16 >> 2);
                const int c = ((row0 >> 3) + ((l16 & 3) >> 1)) ^ swizzle(k);
                const int at = panel + k * LINE + c * 16 + (l16 & 1) * 8;
                const s16x4 q =
                    __builtin_amdgcn_ds_read_tr16_b64_v4i16((TRA_LDS(s16x4) *)(st + at));
                const u32x2 d = __builtin_bit_cast(u32x2, q);
                v[2 * h] = d[0];
                v[2 * h + 1] = d[1];
            }
            return v;
        }
    }
};

// ---- epilogue through LDS -------------------------------------------------------------
//
// A wave owns 64 rows x (32 columns of half 0, 32 of half 1) of sums at a time.
// It lays them out in 16 KB of LDS of its own and reads them back a chunk of
// columns per lane, so that bias, residual and result move 16 bytes a lane and
// whole lines a row, and the activation's code stands once, in a rolled loop.
constexpr int kEpiBytes = 64 * 256;

template <int TI>
__device__ __forceinline__ void epi_put(char *lds, const f32x4 (&c)[TI][2], int half) {
    const int l16 = threadIdx.x & 15, g = (threadIdx.x >> 4) & 3;
#pragma unroll
    for (int i = 0; i < TI; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int row = i * 16 + l16, c16 = half * 8 + j * 4 + g;
            *reinterpret_cast<f32x4 *>(lds + row * 256 + ((c16 ^ (row & 15)) << 4)) = c[i][j];
        }
}

// V sums of one row, from column `col` of the wave's 64 on.
template <int V>
__device__ __forceinline__ void epi_get(const char *lds, int row, int col, float (&v)[V]) {
#pragma unroll
    for (int q = 0; q < V / 4; ++q) {
        const f32x4 t =
            *reinterpret_cast<const f32x4 *>(lds + row * 256 + (((col / 4 + q) ^ (row & 15)) << 4));
#pragma unroll
        for (int e = 0; e < 4; ++e) v[4 * q + e] = t[e];
    }
}

// Rows m0 .. m0 + ROWS - 1; columns n0 .. + 31 (half 0) and n1 .. + 31 (half 1:
// of the same matrix, or, gated, of u, with n1 == n0).
template <typename T, bool GATED, int ROWS>
__device__ __forceinline__ void epi_rows(const TileArgs &p, int batch, int split, const char *lds,
                                         int64_t m0, int64_t n0, int64_t n1) {
    constexpr int V = kChunk<T>;
    constexpr int VPR = (GATED ? 32 : 64) / V;   // chunks per row
    constexpr int RPI = 64 / VPR;                // rows per iteration
    const int lane = threadIdx.x & 63;
    const int col = (lane % VPR) * V;
    const int64_t n = GATED || col < 32 ? n0 + col : n1 + (col - 32);
    if (n >= p.N) return;
#pragma unroll 2
    for (int t = 0; t < ROWS / RPI; ++t) {
        const int row = t * RPI + lane / VPR;
        const int64_t m = m0 + row;
        if (m >= p.M) break;
        float z[V], u[V];
        epi_get(lds, row, col, z);
        if constexpr (GATED) epi_get(lds, row, 32 + col, u);
        if (p.partial != nullptr) {
            const int64_t np = GATED ? 2 * p.N : p.N;
            float *out = p.partial +
                         ((static_cast<int64_t>(split) * p.batch + batch) * p.M + m) * np + n;
            store_row<float, V>(out, p.N - n, p.vec_p, z);
            if constexpr (GATED) store_row<float, V>(out + p.N, p.N - n, p.vec_p, u);
        } else {
            finish<T, GATED, V>(p.epi, batch, m, n, z, u);
        }
    }
}

// ---- the tile kernel --------------------------------------------------------------------
//
// BM x 128 of P per workgroup of four waves in 2 x 2; a wave computes BM / 2
// rows by 32 columns of each half of the tile's columns.  Half 1 is the next 64
// columns, or, gated, the same 64 columns of the second weight: z and u of an
// element sit in the same lane and H is finished without a trip to memory.
//
// S stages of LDS hold a K tile of both operands each.  DIRECT: iteration s
// waits for its own loads of tile s, meets the other waves, issues the loads of
// tile s + S - 1 into the stage whose tile s - 1 every wave has finished, and
// computes tile s.  Otherwise (S = 2) tile s + 1 waits in registers while tile s
// is computed, and is stored behind it.

template <typename T, bool AKC, bool BKC, int BM, bool GATED>
struct TileShape {
    static constexpr int BN = 128, WAVES = 4, TI = BM / 32;
    using PA = Panel<T, AKC, BM, WAVES>;
    using PB = Panel<T, BKC, BN / 2, WAVES>;
    static constexpr int STAGE = PA::BYTES + 2 * PB::BYTES;
    static constexpr int LOADS = PA::INS + 2 * PB::INS;
};

// Where the operands of this workgroup's tile start.
template <typename T, bool AKC, bool BKC>
struct Corner {
    const char *a, *b0, *b1;
    int64_t lda, ldb;      // bytes

    __device__ __forceinline__ Corner(const TileArgs &p, int batch, int64_t m0, int64_t n0,
                                      int64_t n1, bool gated) {
        constexpr int64_t E = sizeof(T);
        lda = p.lda * E;
        ldb = p.ldb * E;
        a = static_cast<const char *>(p.A) + (batch ? p.a_batch * E : 0) + m0 * (AKC ? lda : E);
        const char *b = static_cast<const char *>(p.B[0]) + (batch ? p.b_batch * E : 0);
        b0 = b + n0 * (BKC ? ldb : E);
        b1 = (gated ? static_cast<const char *>(p.B[1]) : b) + n1 * (BKC ? ldb : E);
    }
};

// The K tile s: slices left in its segment, and its byte distance from the
// corner of each operand.
template <typename T, bool AKC, bool BKC>
struct KTile {
    int64_t rem, da, db;
    __device__ __forceinline__ KTile(const TileArgs &p, int64_t lda, int64_t ldb, int s) {
        constexpr int64_t E = sizeof(T);
        const bool second = s >= p.seg_tiles;
        const int64_t k0 = static_cast<int64_t>(second ? s - p.seg_tiles : s) * kSlice<T>;
        rem = p.K - k0;
        da = k0 * (AKC ? E : lda) + (second ? p.a_seg * E : 0);
        db = k0 * (BKC ? E : ldb);
        if (second) db += static_cast<const char *>(p.B[1]) - static_cast<const char *>(p.B[0]);
    }
};

template <typename T, bool AKC, bool BKC, int BM, int S, bool DIRECT, bool GATED>
__global__ __launch_bounds__(256, 2) void linear_tile(const TileArgs p) {
    using X = TileShape<T, AKC, BKC, BM, GATED>;
    using PA = typename X::PA;
    using PB = typename X::PB;
    constexpr int TI = X::TI;
    static_assert(DIRECT || S == 2, "register staging keeps two stages");
    static_assert(S >= 2 && S <= 4 && X::STAGE >= 2 * kEpiBytes * BM / 128, "LDS");
    // One array per stage, so that the compiler can tell a fragment read from
    // the direct loads in flight into the other stages.
    __shared__ __align__(1024) char st0[X::STAGE], st1[X::STAGE];
    __shared__ __align__(1024) char st2[S > 2 ? X::STAGE : 16], st3[S > 3 ? X::STAGE : 16];
    lds_poison(reinterpret_cast<float *>(st0), X::STAGE / 4);
    lds_poison(reinterpret_cast<float *>(st1), X::STAGE / 4);
    if constexpr (S > 2) lds_poison(reinterpret_cast<float *>(st2), X::STAGE / 4);
    if constexpr (S > 3) lds_poison(reinterpret_cast<float *>(st3), X::STAGE / 4);

    const int batch = blockIdx.y;
    const int tiles = p.tiles_m * p.tiles_n;
    const int id = xcd_remap32(blockIdx.x, gridDim.x);
    const int split = id / tiles;
    int tm, tn;
    grouped_tile32<8>(id - split * tiles, p.tiles_m, p.tiles_n, tm, tn);
    constexpr int NB = GATED ? 64 : 128;
    const int64_t m0 = static_cast<int64_t>(tm) * BM;
    const int64_t n0 = static_cast<int64_t>(tn) * NB, n1 = GATED ? n0 : n0 + 64;
    const Corner<T, AKC, BKC> at(p, batch, m0, n0, n1, GATED);
    const int64_t rows_a = p.M - m0, rows_b0 = p.N - n0, rows_b1 = p.N - n1;

    const int first = split * p.tiles_per_split;
    const int left = p.k_tiles - first;
    const int count = left < p.tiles_per_split ? left : p.tiles_per_split;

    const int wave = wave_id();
    const int wm = wave >> 1, wn = wave & 1;
    f32x4 c0[TI][2] = {}, c1[TI][2] = {};

    auto compute = [&](const char *st) __attribute__((always_inline)) {
#pragma unroll
        for (int step = 0; step < 2; ++step) {
            u32x4 x[TI], w0[2], w1[2];
#pragma unroll
            for (int i = 0; i < TI; ++i)
                x[i] = PA::fragment(st, 0, wm * (BM / 2) + i * 16, step);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                w0[j] = PB::fragment(st, PA::BYTES, wn * 32 + j * 16, step);
                w1[j] = PB::fragment(st, PA::BYTES + PB::BYTES, wn * 32 + j * 16, step);
            }
            mma_step<T, TI, 2>(x, w0, c0);
            mma_step<T, TI, 2>(x, w1, c1);
        }
    };

    if constexpr (DIRECT) {
        uint32_t oa[PA::INS], ob0[PB::INS], ob1[PB::INS];
#pragma unroll
        for (int i = 0; i < PA::INS; ++i) oa[i] = PA::offset(i, rows_a, p.lda);
#pragma unroll
        for (int i = 0; i < PB::INS; ++i) {
            ob0[i] = PB::offset(i, rows_b0, p.ldb);
            ob1[i] = PB::offset(i, rows_b1, p.ldb);
        }
        // Tiles past the last are "loaded" too, as zeros from nowhere, which keeps
        // the count of loads in flight.
        auto issue = [&](int s, char *st) __attribute__((always_inline)) {
            const KTile<T, AKC, BKC> t(p, at.lda, at.ldb, first + s);
            const int64_t rem = s < count ? t.rem : 0;
            PA::load_direct(at.a + t.da, p.lda, oa, rem, st);
            PB::load_direct(at.b0 + t.db, p.ldb, ob0, rem, st + PA::BYTES);
            PB::load_direct(at.b1 + t.db, p.ldb, ob1, rem, st + PA::BYTES + PB::BYTES);
        };
        auto iteration = [&](int s, const char *st, char *next) __attribute__((always_inline)) {
            stage_sync<(S - 2) * X::LOADS>();
            issue(s + S - 1, next);
            __builtin_amdgcn_sched_barrier(0);
            compute(st);
        };
        // The waits count loads in tile order: none may be moved past another's.
        issue(0, st0);
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (S > 2) issue(1, st1);
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (S > 3) issue(2, st2);
        for (int s = 0; s < count; s += S) {
            iteration(s, st0, S == 2 ? st1 : S == 3 ? st2 : st3);
            if (s + 1 >= count) break;
            iteration(s + 1, st1, st0);
            if constexpr (S > 2) {
                if (s + 2 >= count) break;
                iteration(s + 2, st2, st1);
            }
            if constexpr (S > 3) {
                if (s + 3 >= count) break;
                iteration(s + 3, st3, st2);
            }
        }
    } else {
        u32x4 ra[PA::INS], rb0[PB::INS], rb1[PB::INS];
        auto fetch = [&](int s) __attribute__((always_inline)) {
            const KTile<T, AKC, BKC> t(p, at.lda, at.ldb, first + s);
            PA::fetch(at.a + t.da, p.lda, rows_a, t.rem, ra);
            PB::fetch(at.b0 + t.db, p.ldb, rows_b0, t.rem, rb0);
            PB::fetch(at.b1 + t.db, p.ldb, rows_b1, t.rem, rb1);
        };
        auto store = [&](char *st) __attribute__((always_inline)) {
            PA::store(ra, st);
            PB::store(rb0, st + PA::BYTES);
            PB::store(rb1, st + PA::BYTES + PB::BYTES);
        };
        auto iteration = [&](int s, const char *st, char *next) __attribute__((always_inline)) {
            __syncthreads();
            if (s + 1 < count) fetch(s + 1);
            compute(st);
            if (s + 1 < count) store(next);
        };
        if (count > 0) {
            fetch(0);
            store(st0);
        }
        for (int s = 0; s < count; s += 2) {
            iteration(s, st0, st1);
            if (s + 1 < count) iteration(s + 1, st1, st0);
        }
    }

    // Every wave has read its last fragments before the stages are reused: a
    // wave's BM / 2 rows of sums take its share of them, 64 (or 32) rows at a
    // time in st0 or st1.  No load is in flight into them either.
    stage_sync<0>();
    constexpr int MINE = kEpiBytes * BM / 128;
    char *mine = (wave < 2 ? st0 : st1) + (wave & 1) * MINE;
    epi_put<TI>(mine, c0, 0);
    epi_put<TI>(mine, c1, 1);
    epi_rows<T, GATED, BM / 2>(p, batch, split, mine, m0 + wm * (BM / 2), n0 + wn * 32,
                               n1 + wn * 32);
}

// ---- launches ----------------------------------------------------------------------------------

template <typename T, bool AKC, bool BKC, bool GATED>
hipError_t launch_tile(const TilePlan &plan, const TileArgs &a, hipStream_t stream) {
    const dim3 grid(static_cast<unsigned>(a.tiles_m) * static_cast<unsigned>(a.tiles_n) *
                        static_cast<unsigned>(a.splits),
                    static_cast<unsigned>(a.batch));
    if (plan.bm == 64) {
        if (plan.direct)
            linear_tile<T, AKC, BKC, 64, 3, true, GATED><<<grid, 256, 0, stream>>>(a);
        else
            linear_tile<T, AKC, BKC, 64, 2, false, GATED><<<grid, 256, 0, stream>>>(a);
    } else {
        if (plan.direct)
            linear_tile<T, AKC, BKC, 128, 2, true, GATED><<<grid, 256, 0, stream>>>(a);
        else
            linear_tile<T, AKC, BKC, 128, 2, false, GATED><<<grid, 256, 0, stream>>>(a);
    }
    return hipGetLastError();
}

}  // namespace

template <typename T>
hipError_t LinearKernels<T>::tile(const TilePlan &plan, const TileArgs &a, hipStream_t stream) {
    switch (plan.form) {
        case kFormKK:
            return plan.gated ? launch_tile<T, true, true, true>(plan, a, stream)
                              : launch_tile<T, true, true, false>(plan, a, stream);
        case kFormKN:
            return plan.gated ? launch_tile<T, true, false, true>(plan, a, stream)
                              : launch_tile<T, true, false, false>(plan, a, stream);
        default: return launch_tile<T, false, false, false>(plan, a, stream);
    }
}

}  // namespace tra
