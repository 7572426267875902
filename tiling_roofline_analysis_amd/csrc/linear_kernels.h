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
#include <utility>

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

// A chunk's elements from `over` on, moved to its front, with zeros behind: over from 0
// (as it is) to all of them.  In 32-bit steps only: as a shift of 128 bits it becomes
// 64-bit shifts whose amount is in a VGPR, and where that is the last VGPR the kernel
// has, gfx950 has taken v0 for it now and then (linear_few with 80 VGPRs shifted the
// last chunk of K by its lane number, in one workgroup of some process's first calls).
template <typename T>
__device__ __forceinline__ u32x4 drop_elements(u32x4 v, int over) {
    constexpr int PER = 4 / static_cast<int>(sizeof(T));     // elements of a dword
    if constexpr (PER == 2) {
        const uint32_t bits = over & 1 ? 16 : 0;
        v = u32x4{__builtin_amdgcn_alignbit(v[1], v[0], bits),
                  __builtin_amdgcn_alignbit(v[2], v[1], bits),
                  __builtin_amdgcn_alignbit(v[3], v[2], bits),
                  __builtin_amdgcn_alignbit(0, v[3], bits)};
    }
    const bool one = over & PER, two = over & (2 * PER), all = over & (4 * PER);
    const uint32_t low = one ? v[1] : v[0], high = one ? v[3] : v[2];
    const uint32_t mid = one ? v[2] : v[1], top = one ? 0u : v[3];
    return u32x4{all ? 0u : two ? high : low, all ? 0u : two ? top : mid,
                 all || two ? 0u : high, all || two ? 0u : top};
}

__device__ __forceinline__ int wave_id() {
    return __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x >> 6));
}

// The end of a stage: this wave's direct loads older than its last VM are in
// LDS and its LDS reads are done; then the workgroup barrier.  (__syncthreads
// would wait for every load in flight.)  s_waitcnt's gfx9 encoding: vmcnt in
// bits 3:0 and 15:14, expcnt 6:4 (not waited for), lgkmcnt 11:8.  The empty asm
// keeps the compiler from moving memory accesses across it.
template <int VM, bool LOADS = true>
__device__ __forceinline__ void stage_sync() {
    static_assert(VM >= 0 && VM < 64, "vmcnt range");
    __builtin_amdgcn_sched_barrier(0);
    // (not LOADS: vmcnt is not waited for)
    __builtin_amdgcn_s_waitcnt(LOADS ? (VM & 15) | ((VM >> 4) << 14) | (7 << 4) : 0xc07f);
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}

// Between LDS accesses of one wave's lanes to what its other lanes wrote or have read.
// A wave's LDS instructions run in order, so it needs no wait and is no instruction;
// it keeps the compiler, which looks at one lane's addresses, from reordering them.
__device__ __forceinline__ void wave_sync() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
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

// All tiles of one chunk step: TI row tiles of x by the TJ column tiles of each
// half, into set `SET` of the sums (16 bits) or, binary32 being four steps of 4, into
// the sets in turn.  A wave needs about 16 MFMAs between two that add to the same
// registers (one wave a SIMD issuing v_mfma_f32_16x16x4_f32 alone reaches 155
// TFLOP/s over 16 tiles, 120 over 8 and 104 over 4), so small tiles keep several
// sets of sums, which are added at the end.
template <typename T, int TI, int TJ>
constexpr int kSets = 2 * TI * TJ >= 16 ? 1 : 2 * TI * TJ >= 8 ? 2 : sizeof(T) == 4 ? 4 : 2;

template <typename T, int SET, int TI, int TJ, int SETS>
__device__ __forceinline__ void mma_step(const u32x4 (&x)[TI], const u32x4 (&w)[2][TJ],
                                         f32x4 (&c)[SETS][2][TI][TJ]) {
    constexpr int STEPS = std::is_same_v<T, float> ? 4 : 1;
#pragma unroll
    for (int e = 0; e < STEPS; ++e)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < TI; ++i)
#pragma unroll
                for (int j = 0; j < TJ; ++j) {
                    f32x4 &d = c[(STEPS > 1 ? e : SET) % SETS][h][i][j];
                    if constexpr (std::is_same_v<T, float>)
                        d = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(w[h][j][e]),
                                                                 __uint_as_float(x[i][e]), d, 0, 0,
                                                                 0);
                    else
                        d = mma16<T>(w[h][j], x[i], d);
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
//         slices k = 0, 4, 8, 12 (two of which meet on one bank where a line
//         is 128 bytes).
// Which global chunk a lane moves follows from that; a line's bytes still
// come from consecutive lanes.
template <typename T, bool KC, int ROWS, int WAVES>
struct Panel {
    static constexpr int BYTES = ROWS * 128;
    static constexpr int LINE = KC ? 128 : ROWS * static_cast<int>(sizeof(T));
    static constexpr int CPL = LINE / 16;             // chunks per line
    static constexpr int LPB = 1024 / LINE;           // lines per block
    static constexpr int INS = BYTES / 1024 / WAVES;  // blocks per wave
    static_assert(LINE >= (sizeof(T) == 4 ? 128 : 64) && LINE <= 1024, "swizzle, block");
    static_assert(BYTES % (1024 * WAVES) == 0, "every wave moves whole blocks");

    static __device__ __forceinline__ int swizzle(int line) {
        if constexpr (KC) return (line >> 1) & 7;
        if constexpr (sizeof(T) == 4) return ((line >> 2) & (CPL / 4 - 1) & 3) << 2;
        if constexpr (LINE == 64) return ((line >> 3) & 1) << 1;
        if constexpr (LINE == 128) return (((line >> 1) & 1) | (((line >> 3) & 1) << 1)) << 1;
        return ((line & 3) | (((line >> 3) & 1) << 2)) << 1;
    }

    // Line and chunk (inside its line) that this lane moves in block i of wave
    // `wave`.
    static __device__ __forceinline__ int line(int wave, int i) {
        return (wave + i * WAVES) * LPB + static_cast<int>(threadIdx.x & 63) / CPL;
    }
    static __device__ __forceinline__ int chunk(int wave, int i) {
        return (static_cast<int>(threadIdx.x & 63) % CPL) ^ swizzle(line(wave, i));
    }
    static __device__ __forceinline__ int lds_block(int wave, int i) {
        return (wave + i * WAVES) * 1024;
    }

    // -- direct loads (buffer_load .. lds), G bytes a lane: 16 where lines are
    // whole, aligned chunks, else 4 (binary32).  What lies outside reads as zero,
    // because its offset lies past the buffer's length.  A load moves 64 G bytes.
    // 4 bytes a lane, four times the instructions, against register staging, which
    // shifts and stores every chunk: 64 x 128 tiles of 3000 x 2049 x 1531 230 -> 192
    // us, of the weight gradient 4097 x 2049 over 4000 rows 734 -> 564.
    static constexpr uint32_t OUTSIDE = 0x80000000u;

    template <int G>
    static constexpr int DINS = INS * (16 / G);       // loads per wave

    // Line that this lane moves a piece of in load i, and the piece's first element
    // in it.
    template <int G>
    static __device__ __forceinline__ int direct_line(int wave, int i) {
        return ((wave + i * WAVES) * 64 + static_cast<int>(threadIdx.x & 63)) * G / LINE;
    }
    template <int G>
    static __device__ __forceinline__ int direct_elem(int wave, int i) {
        constexpr int PER = LINE / G, SUB = 16 / G;
        const int at = ((wave + i * WAVES) * 64 + static_cast<int>(threadIdx.x & 63)) % PER;
        const int c = (at / SUB) ^ swizzle(direct_line<G>(wave, i));
        return (c * SUB + at % SUB) * (G / static_cast<int>(sizeof(T)));
    }

    // Offset of this lane's piece in load i from the panel's corner, or OUTSIDE
    // where the panel's `rows` rows inside the matrix end before it.
    template <int G>
    static __device__ __forceinline__ uint32_t offset(int wave, int i, int64_t rows, int64_t ld) {
        const int n = direct_line<G>(wave, i), e = direct_elem<G>(wave, i);
        const uint32_t at = static_cast<uint32_t>(n) * static_cast<uint32_t>(ld * sizeof(T)) +
                            static_cast<uint32_t>(e) * static_cast<uint32_t>(sizeof(T));
        return (KC ? n : e) < rows ? at : OUTSIDE;
    }

    // Loads the panel at `base` (its corner, wave-uniform) into `lds`; lines are
    // `pitch` bytes apart.  `rem` slices of K are inside (none when rem <= 0:
    // zeros, and no memory is read).  Always the same loads and no branch, so that
    // the number of loads in flight is the same on every path: where it is not, the
    // compiler waits for all of them before a fragment read.
    template <int G>
    static __device__ __forceinline__ void load_direct(int wave, const char *base, int pitch,
                                                       const uint32_t (&off)[DINS<G>], int rem,
                                                       char *lds) {
        // not KC: slices past the last lie past the buffer's end
        const int length = KC || rem >= kSlice<T> ? 0x7fffffff : (rem > 0 ? rem : 0) * pitch;
        const __amdgpu_buffer_rsrc_t rsrc =
            __builtin_amdgcn_make_buffer_rsrc((void *)base, (short)0, length, 0x00020000);
#pragma unroll
        for (int i = 0; i < DINS<G>; ++i) {
            const uint32_t at = KC && direct_elem<G>(wave, i) >= rem ? OUTSIDE : off[i];
            char *to = lds + (wave + i * WAVES) * 64 * G;
            if constexpr (G == 16)
                __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, to, 16, at, 0, 0, 0);
            else
                __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, to, 4, at, 0, 0, 0);
        }
    }

    // -- through registers: any alignment, 16 bytes a lane at element alignment.
    // Every load is in bounds: a row past the matrix reads the last row (its
    // results are not stored), a slice past K the last slice, and a chunk that
    // crosses the end of its line is read where it ends with the line.  Such a
    // chunk is shifted into place, and what lies past K zeroed, when it is
    // stored: nothing waits for the loads before that.
    struct Source {
        int64_t at[INS];       // bytes from the panel's corner
        bool edge;             // not KC: the panel crosses the matrix's last column
    };

    static __device__ __forceinline__ void source(Source &f, int wave, int64_t rows, int64_t ld) {
        constexpr int E = kChunk<T>;
        f.edge = !KC && rows < ROWS;
#pragma unroll
        for (int i = 0; i < INS; ++i) {
            const int64_t n = line(wave, i), c = chunk(wave, i) * E;
            if constexpr (KC)
                f.at[i] = ((n < rows ? n : rows - 1) * ld + c) * static_cast<int64_t>(sizeof(T));
            else
                f.at[i] = (n * ld + (c + E <= rows ? c : rows - E)) * static_cast<int64_t>(sizeof(T));
        }
    }

    static __device__ __forceinline__ void fetch(int wave, const char *base, int64_t ld, int rem,
                                                 const Source &f, u32x4 (&reg)[INS]) {
        constexpr int E = kChunk<T>;
        int64_t at[INS];
#pragma unroll
        for (int i = 0; i < INS; ++i) at[i] = f.at[i];
        if (rem < kSlice<T>) {
#pragma unroll
            for (int i = 0; i < INS; ++i) {
                const int over = (KC ? chunk(wave, i) * E + E : line(wave, i) + 1) - rem;
                if (over > 0) at[i] -= over * (KC ? 1 : ld) * static_cast<int64_t>(sizeof(T));
            }
        }
#pragma unroll
        for (int i = 0; i < INS; ++i) __builtin_memcpy(&reg[i], base + at[i], 16);
    }

    static __device__ __forceinline__ void store(int wave, const u32x4 (&reg)[INS], int64_t rows,
                                                 int rem, const Source &f, char *lds) {
        constexpr int64_t E = kChunk<T>;
        if (rem < kSlice<T> || f.edge) {
#pragma unroll
            for (int i = 0; i < INS; ++i) {
                // elements by which the chunk was read too early
                int64_t over = chunk(wave, i) * E + E - (KC ? rem : rows);
                over = over < 0 ? 0 : over < E ? over : E;
                u32x4 v = drop_elements<T>(reg[i], static_cast<int>(over));
                if (!KC && line(wave, i) >= rem) v = u32x4{};
                put(wave, i, v, lds);
            }
        } else {
#pragma unroll
            for (int i = 0; i < INS; ++i) put(wave, i, reg[i], lds);
        }
    }

    static __device__ __forceinline__ void put(int wave, int i, u32x4 v, char *lds) {
        *reinterpret_cast<u32x4 *>(lds + lds_block(wave, i) + (threadIdx.x & 63) * 16) = v;
    }

    // -- element by element, at once: for lines shorter than a chunk.
    static __device__ __forceinline__ void copy_elements(int wave, const char *base, int64_t ld,
                                                         int64_t rows, int rem, char *lds) {
        constexpr int E = kChunk<T>;
        const T *p = reinterpret_cast<const T *>(base);
#pragma unroll
        for (int i = 0; i < INS; ++i) {
            T t[E];
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const int64_t x = chunk(wave, i) * E + e;
                const int64_t k = KC ? x : line(wave, i), r = KC ? line(wave, i) : x;
                const int64_t kk = k < rem ? k : rem - 1, rr = r < rows ? r : rows - 1;
                const T v = p[KC ? rr * ld + kk : kk * ld + rr];
                t[e] = k < rem ? v : static_cast<T>(0.0f);
            }
            u32x4 v;
            __builtin_memcpy(&v, t, 16);
            put(wave, i, v, lds);
        }
    }

    // LDS reads of a fragment (of 32-bit words the compiler pairs two)
    static constexpr int READS = KC ? 1 : 2;

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
                const int c = ((row0 + l16) >> 2) ^ swizzle(k);
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
// A wave lays its sums out in LDS of its own, HC columns of half 0 beside HC of
// half 1, and reads them back a chunk of columns per lane, so that bias,
// residual and result move 16 bytes a lane and whole lines a row, and the
// activation's code stands once, in a rolled loop.  The 16-byte pieces of a row
// are XORed by the row so that neither side meets bank conflicts.
template <int HC>
__device__ __forceinline__ int epi_at(int row, int piece) {
    static_assert(HC == 32 || HC == 16, "rows of 256 or 128 bytes");
    return HC == 32 ? row * 256 + ((piece ^ (row & 15)) << 4)
                    : row * 128 + ((piece ^ ((row >> 1) & 7)) << 4);
}

template <int HC, int TI, int TJ>
__device__ __forceinline__ void epi_put(char *lds, const f32x4 (&c)[TI][TJ], int half) {
    const int l16 = threadIdx.x & 15, g = (threadIdx.x >> 4) & 3;
#pragma unroll
    for (int i = 0; i < TI; ++i)
#pragma unroll
        for (int j = 0; j < TJ; ++j)
            *reinterpret_cast<f32x4 *>(
                lds + epi_at<HC>(i * 16 + l16, half * (HC / 4) + j * 4 + g)) = c[i][j];
}

// V sums of one row, from column `col` of the wave's 2 HC on.
template <int HC, int V>
__device__ __forceinline__ void epi_get(const char *lds, int row, int col, float (&v)[V]) {
#pragma unroll
    for (int q = 0; q < V / 4; ++q) {
        const f32x4 t = *reinterpret_cast<const f32x4 *>(lds + epi_at<HC>(row, col / 4 + q));
#pragma unroll
        for (int e = 0; e < 4; ++e) v[4 * q + e] = t[e];
    }
}

// Rows m0 .. m0 + ROWS - 1; columns n0 .. + HC - 1 (half 0) and n1 .. (half 1:
// of the same matrix, or, gated, of u, with n1 == n0).  Where every lane's chunk
// is inside or outside as a whole, several rows are in hand at a time, with no
// branch between a row's read and its store but those of the row's end: branches
// and waits row by row took 8 us of a 128 x 128 tile in binary32.
// Not a whole tile: the sums go to `sums` (this wave's rows and columns; rows
// `pitch` long, half 1 half a row on) as they are.
template <typename T, bool GATED, int HC, int ROWS>
__device__ __forceinline__ void epi_rows(const TileArgs &p, int batch, float *sums, int pitch,
                                         const char *lds, int64_t m0, int64_t n0, int64_t n1) {
    constexpr int V = kChunk<T>;
    constexpr int VPR = (GATED ? HC : 2 * HC) / V;   // chunks per row
    constexpr int RPI = 64 / VPR;                    // rows per step
    constexpr int STEPS = ROWS / RPI, ROOM = GATED || V == 8 ? 2 : 4;
    constexpr int U = STEPS < ROOM ? STEPS : ROOM;     // rows in hand: 32 VGPRs or fewer
    static_assert(ROWS % RPI == 0 && STEPS % U == 0, "whole rounds");
    const int lane = threadIdx.x & 63;
    const int col = (lane % VPR) * V;
    const int64_t n = GATED || col < HC ? n0 + col : n1 + (col - HC);
    if (n >= p.N) return;
    const EpiArgs &e = p.epi;
    const int first = lane / VPR;
    const int rows = static_cast<int>(p.M - m0 < ROWS ? p.M - m0 : ROWS);

    if (sums != nullptr) {
        float *out = sums + first * pitch + (GATED || col < HC ? col : pitch / 2 + (col - HC));
#pragma unroll 4
        for (int t = 0; t < STEPS; ++t) {
            const int row = t * RPI + first;
            if (row >= rows) break;
            float z[V];
            epi_get<HC>(lds, row, col, z);
            store_row<float, V>(out, z);
            if constexpr (GATED) {
                epi_get<HC>(lds, row, HC + col, z);
                store_row<float, V>(out + pitch / 2, z);
            }
            out += RPI * pitch;
        }
        return;
    }
    if (p.N % V != 0 && n1 + HC > p.N) {
        for (int t = 0; t < STEPS; ++t) {
            const int row = t * RPI + first;
            if (row >= rows) break;
            float z[V], u[V];
            epi_get<HC>(lds, row, col, z);
            if constexpr (GATED) epi_get<HC>(lds, row, HC + col, u);
            with_act(e.act, [&](auto act) __attribute__((always_inline)) {
                finish<T, GATED, decltype(act)::value, V>(e, batch, m0 + row, n, z, u);
            });
        }
        return;
    }
    float undo = 1.0f;
    if constexpr (kScaled<T> && !GATED) {
        if (e.undo != nullptr) undo = *e.undo;
    }
    float b[V] = {};
    if (!GATED && e.bias != nullptr) load_row<T, V>(static_cast<const T *>(e.bias) + n, b);
    T *y = static_cast<T *>(batch == 0 ? e.Y[0] : e.Y[1]) + (m0 + first) * e.ldy + n;
    const T *r = static_cast<const T *>(e.R) + (m0 + first) * e.ldr + n;
    float *keep = e.Z + (m0 + first) * e.ldz + n;
#pragma unroll 1
    for (int t = 0; t < STEPS; t += U) {
        float z[U][V], u[U][V], add[U][V] = {};
        if (!GATED && e.R != nullptr) {
#pragma unroll
            for (int k = 0; k < U; ++k)
                if ((t + k) * RPI + first < rows) load_row<T, V>(r + k * RPI * e.ldr, add[k]);
        }
#pragma unroll
        for (int k = 0; k < U; ++k) {
            epi_get<HC>(lds, (t + k) * RPI + first, col, z[k]);
            if constexpr (GATED) epi_get<HC>(lds, (t + k) * RPI + first, HC + col, u[k]);
        }
        if constexpr (!GATED) {
#pragma unroll
            for (int k = 0; k < U; ++k)
#pragma unroll
                for (int i = 0; i < V; ++i) z[k][i] = kScaled<T> ? z[k][i] * undo + b[i] : z[k][i] + b[i];
        }
        if (e.Z != nullptr) {
#pragma unroll
            for (int k = 0; k < U; ++k)
                if ((t + k) * RPI + first < rows) {
                    store_row<float, V>(keep + k * RPI * e.ldz, z[k]);
                    if constexpr (GATED) store_row<float, V>(keep + k * RPI * e.ldz + p.N, u[k]);
                }
        }
        with_act(e.act, [&](auto act) __attribute__((always_inline)) {
#pragma unroll
            for (int k = 0; k < U; ++k)
#pragma unroll
                for (int i = 0; i < V; ++i) z[k][i] = activate<decltype(act)::value>(z[k][i]);
        });
#pragma unroll
        for (int k = 0; k < U; ++k) {
#pragma unroll
            for (int i = 0; i < V; ++i) z[k][i] = GATED ? z[k][i] * u[k][i] : z[k][i] + add[k][i];
            if ((t + k) * RPI + first < rows) store_row<T, V>(y + k * RPI * e.ldy, z[k]);
        }
        y += U * RPI * e.ldy;
        r += U * RPI * e.ldr;
        keep += U * RPI * e.ldz;
    }
}

// ---- the tile kernel --------------------------------------------------------------------
//
// BM x BN of P per workgroup of four waves in 2 x 2; a wave computes BM / 2
// rows by BN / 4 columns of each half of the tile's columns.  Half 1 is the next
// BN / 2 columns, or, gated, the same columns of the second weight: z and u of an
// element sit in the same lane and H is finished without a trip to memory.
//
// S stages of LDS hold a K tile of both operands each.  A K tile is two MFMA
// steps, and the fragments of a step are read while the step before it is
// computed, so that one wave a SIMD keeps its matrix unit busy.  Iteration s:
//   read step 1 of tile s; compute step 0;
//   wait for this wave's loads of tile s + 1, meet the other waves: tile s + 1 is
//   in LDS, and every wave has read tile s;
//   DIRECT: load tile s + S into the stage of tile s;
//   read step 0 of tile s + 1; compute step 1.
// Without DIRECT (S = 2) tile s + 1 waits in registers until it is stored,
// before the meeting, into the stage of tile s - 1.
// Measured: 1024^3 in binary32 with bias, GELU and residual 21.3 us (64 x 64 tiles,
// one a CU; with both steps of tile s read after the meeting, in a block of their
// own, 31 us), per K tile 0.50 us against 0.43 of MFMAs at the datasheet's rate;
// 128 x 128 tiles in binary32 1.77 us per K tile, 151 TFLOP/s; 16 bits, two a CU,
// 0.83 us per two K tiles, 1.3 PFLOP/s, bounded by LDS reads and barriers.

template <typename T, bool AKC, bool BKC, int BM, int BN>
struct TileShape {
    static constexpr int WAVES = 4, TI = BM / 32, TJ = BN / 64, HC = BN / 4;
    using PA = Panel<T, AKC, BM, WAVES>;
    using PB = Panel<T, BKC, BN / 2, WAVES>;
    static constexpr int STAGE = PA::BYTES + 2 * PB::BYTES;
    static constexpr int MINE = BM / 2 * HC * 8;     // a wave's sums in the epilogue
    // Workgroups a CU by LDS: two, where the stages leave room.
    static constexpr int per_cu(int stages) { return stages * STAGE <= 80 * 1024 ? 2 : 1; }
};

// A workgroup's way along K: the corners of its panels at the current K tile, and
// the slices left.  The steps are few scalar instructions, since with one wave a
// SIMD every one of them delays the MFMAs (addresses worked out anew for each tile
// took half the time of a 64 x 64 tile in binary32).
template <typename T, bool AKC, bool BKC>
struct Walk {
    const char *a, *b0, *b1;
    int64_t step_a, step_b;    // bytes per K tile
    int64_t jump_a, jump_b;    // from the first segment's last tile to the second
    int rem;                   // slices left in this segment; then none
    int then;                  // slices of the second segment that follow

    // K tiles first .. first + count - 1 of the concatenated segments.
    __device__ __forceinline__ Walk(const TileArgs &p, int batch, int64_t m0, int64_t n0,
                                    int64_t n1, bool gated, int first, int count) {
        constexpr int64_t E = sizeof(T);
        constexpr int L = kSlice<T>;
        a = static_cast<const char *>(p.A) + (batch ? p.a_batch * E : 0) +
            m0 * (AKC ? p.lda * E : E);
        const char *b = static_cast<const char *>(p.B[0]) + (batch ? p.b_batch * E : 0);
        b0 = b + n0 * (BKC ? p.ldb * E : E);
        b1 = (gated ? static_cast<const char *>(p.B[1]) : b) + n1 * (BKC ? p.ldb * E : E);
        step_a = L * (AKC ? E : p.lda * E);
        step_b = L * (BKC ? E : p.ldb * E);
        const int64_t to_a = p.a_seg * E;
        const int64_t to_b =
            static_cast<const char *>(p.B[1]) - static_cast<const char *>(p.B[0]);
        jump_a = to_a - (p.seg_tiles - 1) * step_a;
        jump_b = to_b - (p.seg_tiles - 1) * step_b;
        const int K = static_cast<int>(p.K);
        int in = p.seg_tiles - first;          // tiles in the first segment
        int at = first;
        if (in <= 0 && count > 0) {            // none: this part lies in the second
            a += to_a;
            b0 += to_b;
            b1 += to_b;
            at = -in;
            in = count;
            then = 0;
        } else {
            const int more = count - in;
            then = more <= 0 ? 0 : more * L < K ? more * L : K;
            in = more <= 0 ? count : in;
        }
        a += at * step_a;
        b0 += at * step_b;
        b1 += at * step_b;
        rem = K - at * L < in * L ? K - at * L : in * L;
    }

    __device__ __forceinline__ void next() {
        rem -= kSlice<T>;
        // no branch: the tile's loads are to mix with its MFMAs
        const bool jump = (rem <= 0) & (then > 0);
        a += jump ? jump_a : step_a;
        b0 += jump ? jump_b : step_b;
        b1 += jump ? jump_b : step_b;
        rem = jump ? then : rem;
        then = jump ? 0 : then;
    }
};

// What a workgroup computes: a whole tile, or one part of a split one.
struct Part {
    int tile;
    int first, count;      // K tiles
    float *sums;           // of a part: bm x bn, else null

    __device__ __forceinline__ Part(const TileArgs &p, int batch, int area) {
        const int tiles = p.tiles_m * p.tiles_n, bid = static_cast<int>(blockIdx.x);
        if (bid < p.whole) {
            tile = xcd_remap32(bid, p.whole);
            first = 0;
            count = p.k_tiles;
            sums = nullptr;
        } else {
            const int split_tiles = tiles - p.whole;
            const int id = xcd_remap32(bid - p.whole, static_cast<int>(gridDim.x) - p.whole);
            const int split = id / split_tiles, at = id - split * split_tiles;
            tile = p.whole + at;
            first = split * p.tiles_per_split;
            const int left = p.k_tiles - first;
            count = left < p.tiles_per_split ? left : p.tiles_per_split;
            sums = p.partial +
                   ((static_cast<int64_t>(batch) * split_tiles + at) * p.splits + split) * area;
        }
    }
};

// Orders what stands since the last scheduling barrier: after each MFMA a share
// of the LDS reads (all within the first half of the MFMAs, so that they are done
// by the end) and of the loads.  A wave issues them while its MFMA runs; in a
// block of their own they would leave the matrix unit idle, and left alone the
// compiler sinks the reads below the MFMAs, to where their results are waited for.
template <int MFMAS, int READS, int LOADS>
__device__ __forceinline__ void interleave() {
    constexpr int HALF = MFMAS / 2 > 0 ? MFMAS / 2 : 1;
#pragma unroll
    for (int i = 0; i < MFMAS; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        constexpr int R = (READS + HALF - 1) / HALF, L = (LOADS + MFMAS - 1) / MFMAS;
        if (i * R < READS) __builtin_amdgcn_sched_group_barrier(0x100, R, 0);
        if (i * L < LOADS) __builtin_amdgcn_sched_group_barrier(0x010, L, 0);
    }
}

// f(0), f(1), .. (as constants) until one returns false; whether none did.
template <int... U, typename F>
__device__ __forceinline__ bool for_each(std::integer_sequence<int, U...>, F f) {
    return (f(std::integral_constant<int, U>{}) && ...);
}

template <typename T, bool AKC, bool BKC, int BM, int BN, int S, int DIRECT, bool GATED>
__global__ __launch_bounds__(256, (TileShape<T, AKC, BKC, BM, BN>::per_cu(S))) void linear_tile(const TileArgs p) {
    using X = TileShape<T, AKC, BKC, BM, BN>;
    using PA = typename X::PA;
    using PB = typename X::PB;
    constexpr int TI = X::TI, TJ = X::TJ, HC = X::HC;
    static_assert(DIRECT == 16 || (DIRECT == 4 && sizeof(T) == 4) || (DIRECT == 0 && S == 2),
                  "bytes of a direct load; register staging keeps two stages");
    static_assert(S >= 2 && S <= 6 && X::STAGE >= 2 * X::MINE, "LDS");
    // One array per stage, so that the compiler can tell a fragment read from
    // the direct loads in flight into the other stages.
    __shared__ __align__(1024) char st0[X::STAGE], st1[X::STAGE];
    __shared__ __align__(1024) char st2[S > 2 ? X::STAGE : 16], st3[S > 3 ? X::STAGE : 16];
    __shared__ __align__(1024) char st4[S > 4 ? X::STAGE : 16], st5[S > 5 ? X::STAGE : 16];
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

    const int batch = blockIdx.y;
    const Part part(p, batch, BM * BN);
    int tm, tn;
    grouped_tile32<kGroupTile>(part.tile, p.tiles_m, p.tiles_n, tm, tn);
    constexpr int NB = GATED ? BN / 2 : BN;
    const int64_t m0 = static_cast<int64_t>(tm) * BM;
    const int64_t n0 = static_cast<int64_t>(tn) * NB, n1 = GATED ? n0 : n0 + BN / 2;
    const int64_t rows_a = p.M - m0, rows_b0 = p.N - n0, rows_b1 = p.N - n1;

    const int first = part.first, count = part.count;

    Walk<T, AKC, BKC> walk(p, batch, m0, n0, n1, GATED, first, count);

    const int wave = wave_id();
    const int wm = wave >> 1, wn = wave & 1;
    constexpr int SETS = kSets<T, TI, TJ>;
    f32x4 c[SETS][2][TI][TJ] = {};

    u32x4 x[2][TI], w[2][2][TJ];
    auto read = [&](auto step, const char *st) __attribute__((always_inline)) {
        constexpr int P = decltype(step)::value;
#pragma unroll
        for (int i = 0; i < TI; ++i)
            x[P][i] = PA::fragment(st, 0, wm * (BM / 2) + i * 16, P);
#pragma unroll
        for (int j = 0; j < TJ; ++j) {
            w[P][0][j] = PB::fragment(st, PA::BYTES, wn * HC + j * 16, P);
            w[P][1][j] = PB::fragment(st, PA::BYTES + PB::BYTES, wn * HC + j * 16, P);
        }
    };
    // LDS instructions of one step's fragments, MFMAs of a step
    constexpr int READS = PA::READS * TI + 2 * PB::READS * TJ;
    constexpr int MFMAS = 2 * TI * TJ * (sizeof(T) == 4 ? 4 : 1);
    constexpr std::integral_constant<int, 0> step0;
    constexpr std::integral_constant<int, 1> step1;

    if constexpr (DIRECT != 0) {
        constexpr int IA = PA::template DINS<DIRECT>, IB = PB::template DINS<DIRECT>;
        constexpr int LOADS = IA + 2 * IB;
        uint32_t oa[IA], ob0[IB], ob1[IB];
#pragma unroll
        for (int i = 0; i < IA; ++i) oa[i] = PA::template offset<DIRECT>(wave, i, rows_a, p.lda);
#pragma unroll
        for (int i = 0; i < IB; ++i) {
            ob0[i] = PB::template offset<DIRECT>(wave, i, rows_b0, p.ldb);
            ob1[i] = PB::template offset<DIRECT>(wave, i, rows_b1, p.ldb);
        }
        const int pitch_a = static_cast<int>(p.lda * static_cast<int64_t>(sizeof(T)));
        const int pitch_b = static_cast<int>(p.ldb * static_cast<int64_t>(sizeof(T)));
        // Tiles past the last are "loaded" too, as zeros from nowhere, which keeps
        // the count of loads in flight.  The waits count loads in tile order: none
        // may be moved past another's.
        auto issue = [&](char *st) __attribute__((always_inline)) {
            PA::template load_direct<DIRECT>(wave, walk.a, pitch_a, oa, walk.rem, st);
            PB::template load_direct<DIRECT>(wave, walk.b0, pitch_b, ob0, walk.rem, st + PA::BYTES);
            PB::template load_direct<DIRECT>(wave, walk.b1, pitch_b, ob1, walk.rem,
                                             st + PA::BYTES + PB::BYTES);
            walk.next();
        };
        for_each(std::make_integer_sequence<int, S>{}, [&](auto u) __attribute__((always_inline)) {
            issue(stage(u));
            __builtin_amdgcn_sched_barrier(0);
            return true;
        });
        stage_sync<(S - 1) * LOADS>();
        read(step0, st0);
        auto iteration = [&](auto u) __attribute__((always_inline)) {
            constexpr int U = decltype(u)::value;
            read(step1, stage(u));
            mma_step<T, 0>(x[0], w[0], c);
            interleave<MFMAS, READS, 0>();
            stage_sync<(S - 2) * LOADS>();
            issue(stage(u));
            read(step0, stage(std::integral_constant<int, U + 1>{}));
            mma_step<T, 1>(x[1], w[1], c);
            interleave<MFMAS, READS, LOADS>();
            __builtin_amdgcn_sched_barrier(0);
        };
        // Whole rounds of the ring, then what is left: a way out of the middle of
        // the loop, which the compiler might join to its head, would make it wait
        // for every load there.
        int s = 0;
        for (; s + S <= count; s += S)
            for_each(std::make_integer_sequence<int, S>{},
                     [&](auto u) __attribute__((always_inline)) {
                         iteration(u);
                         return true;
                     });
        for_each(std::make_integer_sequence<int, S - 1>{},
                 [&](auto u) __attribute__((always_inline)) {
                     if (s + decltype(u)::value >= count) return false;
                     iteration(u);
                     return true;
                 });
    } else {
        typename PA::Source fa;
        typename PB::Source fb0, fb1;
        PA::source(fa, wave, rows_a, p.lda);
        PB::source(fb0, wave, rows_b0, p.ldb);
        PB::source(fb1, wave, rows_b1, p.ldb);
        u32x4 ra[PA::INS], rb0[PB::INS], rb1[PB::INS];
        int rem = 0;       // slices of the tile in registers
        auto fetch = [&]() __attribute__((always_inline)) {
            rem = walk.rem;
            PA::fetch(wave, walk.a, p.lda, rem, fa, ra);
            PB::fetch(wave, walk.b0, p.ldb, rem, fb0, rb0);
            PB::fetch(wave, walk.b1, p.ldb, rem, fb1, rb1);
            walk.next();
        };
        auto store = [&](char *st) __attribute__((always_inline)) {
            PA::store(wave, ra, rows_a, rem, fa, st);
            PB::store(wave, rb0, rows_b0, rem, fb0, st + PA::BYTES);
            PB::store(wave, rb1, rows_b1, rem, fb1, st + PA::BYTES + PB::BYTES);
        };
        auto iteration = [&](const char *st, char *next) __attribute__((always_inline)) {
            read(step1, st);
            mma_step<T, 0>(x[0], w[0], c);
            interleave<MFMAS, READS, 0>();
            __builtin_amdgcn_sched_barrier(0);
            store(next);
            stage_sync<0, false>();
            fetch();
            __builtin_amdgcn_sched_barrier(0);
            read(step0, next);
            mma_step<T, 1>(x[1], w[1], c);
            interleave<MFMAS, READS, 0>();
            __builtin_amdgcn_sched_barrier(0);
        };
        if ((AKC ? p.K : p.M) < kChunk<T> || (BKC ? p.K : p.N) < kChunk<T>) {
            for (int s = 0; s < count; ++s) {
                __syncthreads();
                PA::copy_elements(wave, walk.a, p.lda, rows_a, walk.rem, st0);
                PB::copy_elements(wave, walk.b0, p.ldb, rows_b0, walk.rem, st0 + PA::BYTES);
                PB::copy_elements(wave, walk.b1, p.ldb, rows_b1, walk.rem,
                                  st0 + PA::BYTES + PB::BYTES);
                walk.next();
                __syncthreads();
                read(step0, st0);
                read(step1, st0);
                mma_step<T, 0>(x[0], w[0], c);
                mma_step<T, 1>(x[1], w[1], c);
            }
        } else if (count > 0) {
            fetch();
            store(st0);
            fetch();
            stage_sync<0>();
            read(step0, st0);
            for (int s = 0; s < count; s += 2) {
                iteration(st0, st1);
                if (s + 1 < count) iteration(st1, st0);
            }
        }
    }

    // Every wave has read its last fragments, and no load is in flight, before
    // the stages are reused: a wave's sums take their share of st0 or st1.
    stage_sync<0>();
    char *mine = (wave < 2 ? st0 : st1) + (wave & 1) * X::MINE;
#pragma unroll
    for (int a = 1; a < SETS; ++a)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < TI; ++i)
#pragma unroll
                for (int j = 0; j < TJ; ++j) c[0][h][i][j] += c[a][h][i][j];
    epi_put<HC>(mine, c[0][0], 0);
    epi_put<HC>(mine, c[0][1], 1);
    wave_sync();
    epi_rows<T, GATED, HC, BM / 2>(
        p, batch, part.sums == nullptr ? nullptr : part.sums + wm * (BM / 2) * BN + wn * HC, BN,
        mine, m0 + wm * (BM / 2), n0 + wn * HC, n1 + wn * HC);
}

// ---- the kernel for few rows --------------------------------------------------------------
//
// M <= 16 (tokens being decoded): the weights are read once and nothing else
// counts, so they go from memory straight into the MFMA's registers, with no LDS
// and no second launch.  A workgroup of eight waves owns a strip of columns as
// wide as 64 bytes of a weight row (16 columns where the weights are
// k-contiguous) and shares K out over its waves; the sums meet in LDS.
//   k-contiguous   lane l loads chunk l / 16 of column l % 16: an operand as it
//                  stands;
//   else           lane l loads 4 bytes (two columns, or one in binary32) of each
//                  of 8 (4) slices, and v_perm makes two operands of them.
// Loads take any alignment, in bounds: columns past the last read the last, and
// what lies past K is zeroed.
// Measured: 1 x 2048 x 2048 bf16 5.3 us of device time (64 x 64 tiles split 4 ways,
// and their join: 8.0); gated 1 x 12288 x 4096 bf16 37 us, 5.4 TB/s of weights.
template <typename T, bool BKC>
struct FewShape {
    static constexpr int WAVES = 8;
    static constexpr int V = BKC ? 1 : 4 / static_cast<int>(sizeof(T));   // columns per lane
    static constexpr int COLS = 16 * V;
    static constexpr int STEP = 4 * kChunk<T>;     // slices per MFMA step
    static constexpr int U = 4;                    // steps loaded at a time
    static constexpr int ROUND = U * STEP;         // slices per wave and round
};

// The chunk at slices k .. of a line of K >= one chunk of elements, zero past
// its end.
template <typename T>
__device__ __forceinline__ u32x4 chunk_to_end(const T *line, int k, int K) {
    constexpr int E = kChunk<T>;
    const int over = k + E - K;
    u32x4 v;
    __builtin_memcpy(&v, line + (over > 0 ? K - E : k), 16);
    return drop_elements<T>(v, over <= 0 ? 0 : over < E ? over : E);
}

template <typename T, bool BKC, bool GATED>
__global__ __launch_bounds__(512) void linear_few(const TileArgs p) {
    using F = FewShape<T, BKC>;
    constexpr int E = kChunk<T>, V = F::V, U = F::U, W = GATED ? 2 : 1;
    __shared__ __align__(16) float sums[F::WAVES][W * V][256];
    lds_poison(&sums[0][0][0], F::WAVES * W * V * 256);
    const int wave = wave_id(), l16 = threadIdx.x & 15, g = (threadIdx.x >> 4) & 3;
    const int M = static_cast<int>(p.M), N = static_cast<int>(p.N), K = static_cast<int>(p.K);
    const int n0 = xcd_remap32(blockIdx.x, gridDim.x) * F::COLS;
    const T *xrow = static_cast<const T *>(p.A) + (l16 < M ? l16 : M - 1) * p.lda;
    // k-contiguous: this lane's column; else its first, moved back by one where
    // two columns would cross the last
    const int want = n0 + l16 * V, col = want + V <= N ? want : N - V;
    f32x4 c[W][V] = {};

    for (int seg = 0; seg < p.segs; ++seg) {
        const T *x = xrow + seg * p.a_seg;
        const T *w[W];
        for (int h = 0; h < W; ++h)
            w[h] = static_cast<const T *>(p.B[GATED ? h : seg]) + (BKC ? col * p.ldb : col);

        // Rounds of U steps: `whole` where all of them lie inside K.
        auto round = [&](int k0, auto whole) __attribute__((always_inline)) {
            constexpr bool WHOLE = decltype(whole)::value;
            u32x4 a[U], b[W][V][U];
#pragma unroll
            for (int h = 0; h < W; ++h)
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int k = k0 + u * F::STEP + g * E;
                    if constexpr (BKC) {
                        if constexpr (WHOLE)
                            __builtin_memcpy(&b[h][0][u], w[h] + k, 16);
                        else
                            b[h][0][u] = chunk_to_end(w[h], k, K);
                    } else {
                        uint32_t t[E];
#pragma unroll
                        for (int e = 0; e < E; ++e) {
                            const int kk = WHOLE || k + e < K ? k + e : K - 1;
                            __builtin_memcpy(&t[e], w[h] + kk * p.ldb, 4);
                        }
#pragma unroll
                        for (int e = 0; e < E; ++e) {
                            if (V == 2 && want > col) t[e] >>= 16;
                            if (!WHOLE && k + e >= K) t[e] = 0;
                        }
                        if constexpr (V == 1) {
                            b[h][0][u] = u32x4{t[0], t[1], t[2], t[3]};
                        } else {
#pragma unroll
                            for (int q = 0; q < 4; ++q) {
                                // low halves, then high halves, of slices 2q, 2q + 1
                                b[h][0][u][q] = __builtin_amdgcn_perm(t[2 * q + 1], t[2 * q],
                                                                      0x05040100);
                                b[h][V - 1][u][q] = __builtin_amdgcn_perm(t[2 * q + 1], t[2 * q],
                                                                          0x07060302);
                            }
                        }
                    }
                }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int k = k0 + u * F::STEP + g * E;
                if constexpr (WHOLE)
                    __builtin_memcpy(&a[u], x + k, 16);
                else
                    a[u] = chunk_to_end(x, k, K);
            }
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int h = 0; h < W; ++h)
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        if constexpr (std::is_same_v<T, float>) {
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                c[h][v] = __builtin_amdgcn_mfma_f32_16x16x4f32(
                                    __uint_as_float(b[h][v][u][e]), __uint_as_float(a[u][e]),
                                    c[h][v], 0, 0, 0);
                        } else {
                            c[h][v] = mma16<T>(b[h][v][u], a[u], c[h][v]);
                        }
                    }
        };
        int k0 = wave * F::ROUND;
        for (; k0 + F::ROUND <= K; k0 += F::WAVES * F::ROUND)
            round(k0, std::integral_constant<bool, true>{});
        if (k0 < K) round(k0, std::integral_constant<bool, false>{});
    }

    // Lane l holds token l % 16 of strip rows 4 (l / 16) .. + 3.
#pragma unroll
    for (int h = 0; h < W; ++h)
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                sums[wave][h * V + v][l16 * 16 + 4 * g + r] = c[h][v][r];
    __syncthreads();
    for (int i = threadIdx.x; i < 256 * V; i += 512) {
        const int m = i / F::COLS, j = i - m * F::COLS, n = n0 + j;
        if (m >= M || n >= N) continue;
        float z[1] = {}, u[1] = {};
#pragma unroll
        for (int s = 0; s < F::WAVES; ++s) {
            z[0] += sums[s][j % V][m * 16 + j / V];
            if constexpr (GATED) u[0] += sums[s][V + j % V][m * 16 + j / V];
        }
        with_act(p.epi.act, [&](auto act) __attribute__((always_inline)) {
            finish<T, GATED, decltype(act)::value, 1>(p.epi, 0, m, n, z, u);
        });
    }
}

// ---- the wide kernel -----------------------------------------------------------------------
//
// 256 x 256 of P per workgroup of eight waves, for 16-bit products of many tiles,
// which the matrix units bound.  A K tile is four panels of 128 rows or columns:
// A0, A1, B0, B1 (gated: B0 of the one weight, B1 of the other); a wave computes 64
// rows of each A panel by 32 columns of each B panel, as four quadrants of 16
// MFMAs.  Two stages of each panel, an array each, take 128 KB of LDS.
//
// The waves of the lower rows run half a phase behind those of the upper: there is
// one of each on every SIMD, and while the one computes a quadrant the other
// reads the fragments of its next.  (Two groups of four waves that take turns at
// the matrix units, a barrier apart, each with a tile in four quadrants, is a publicly
// described schedule for large products on this architecture, known as ping-pong; the
// phases, panels and waits below are worked out here.)  A phase is
//   read this quadrant's fragments and load one panel of a later tile; barrier;
//   16 MFMAs; barrier.
// Phases of tile s, with the panels loaded ("> s + 2": of tile s + 2):
//   0  reads B0, A0, loads A1 > s + 1;  A0 B0      2  reads A1, loads B0 > s + 2;  A1 B1
//   1  reads B1,     loads A0 > s + 2;  A0 B1      3  loads B1 > s + 2;            A1 B0
// A panel is loaded into the stage that held it two tiles before, one phase or
// more after both groups of waves have read it: reads are waited for before the
// barrier that follows them, and the group behind reads one barrier later.  In
// phase 3 a wave waits until only its last three panels are in flight: all of tile
// s + 1 is then in LDS two barriers on, when the first group reads it.
// Measured: gated 8192 x 12288 x 4096 bf16 1130 us, 1.45 PFLOP/s, its matrix units
// busy 79% of the cycles (128 x 128 tiles: 1490 us); 1.42 us per K tile with all
// CUs at work, 1.28 with fewer than a tile a CU, so power, more than the schedule,
// bounds it; the stores of a tile, 7 us, are not hidden.
template <typename T, bool AKC, bool BKC, bool GATED>
__global__ __launch_bounds__(512, 2) void linear_wide(const TileArgs p) {
    using PA = Panel<T, AKC, 128, 8>;
    using PB = Panel<T, BKC, 128, 8>;
    constexpr int L = PA::INS;
    static_assert(sizeof(T) == 2 && L == 2 && PB::INS == 2 && PA::BYTES == 64 * 64 * 4,
                  "panels of two loads a wave; a wave's sums fill one");
    __shared__ __align__(1024) char a00[PA::BYTES], a01[PA::BYTES], a10[PA::BYTES], a11[PA::BYTES];
    __shared__ __align__(1024) char b00[PB::BYTES], b01[PB::BYTES], b10[PB::BYTES], b11[PB::BYTES];
    lds_poison(reinterpret_cast<float *>(a00), PA::BYTES / 4);
    lds_poison(reinterpret_cast<float *>(a01), PA::BYTES / 4);
    lds_poison(reinterpret_cast<float *>(a10), PA::BYTES / 4);
    lds_poison(reinterpret_cast<float *>(a11), PA::BYTES / 4);
    lds_poison(reinterpret_cast<float *>(b00), PB::BYTES / 4);
    lds_poison(reinterpret_cast<float *>(b01), PB::BYTES / 4);
    lds_poison(reinterpret_cast<float *>(b10), PB::BYTES / 4);
    lds_poison(reinterpret_cast<float *>(b11), PB::BYTES / 4);

    const int batch = blockIdx.y;
    const Part part(p, batch, 256 * 256);
    int tm, tn;
    grouped_tile32<kGroupWide>(part.tile, p.tiles_m, p.tiles_n, tm, tn);
    const int64_t m0 = static_cast<int64_t>(tm) * 256;
    const int64_t n0 = static_cast<int64_t>(tn) * (GATED ? 128 : 256), n1 = GATED ? n0 : n0 + 128;
    const int first = part.first, count = part.count;
    Walk<T, AKC, BKC> walk(p, batch, m0, n0, n1, GATED, first, count);
    const int64_t lower = 128 * (AKC ? p.lda : 1) * static_cast<int64_t>(sizeof(T));

    const int wave = wave_id();
    const int wm = wave >> 2, wn = wave & 3;
    uint32_t oa0[L], oa1[L], ob0[L], ob1[L];
#pragma unroll
    for (int i = 0; i < L; ++i) {
        oa0[i] = PA::template offset<16>(wave, i, p.M - m0, p.lda);
        oa1[i] = PA::template offset<16>(wave, i, p.M - m0 - 128, p.lda);
        ob0[i] = PB::template offset<16>(wave, i, p.N - n0, p.ldb);
        ob1[i] = PB::template offset<16>(wave, i, p.N - n1, p.ldb);
    }
    const int pitch_a = static_cast<int>(p.lda * static_cast<int64_t>(sizeof(T)));
    const int pitch_b = static_cast<int>(p.ldb * static_cast<int64_t>(sizeof(T)));

    // A1 is loaded one tile behind the others: where its tile starts
    const char *late = nullptr;
    int late_rem = 0;
    auto load_a0 = [&](char *st) __attribute__((always_inline)) {
        PA::template load_direct<16>(wave, walk.a, pitch_a, oa0, walk.rem, st);
    };
    auto load_b0 = [&](char *st) __attribute__((always_inline)) {
        PB::template load_direct<16>(wave, walk.b0, pitch_b, ob0, walk.rem, st);
    };
    auto load_b1 = [&](char *st) __attribute__((always_inline)) {
        PB::template load_direct<16>(wave, walk.b1, pitch_b, ob1, walk.rem, st);
        late = walk.a + lower;
        late_rem = walk.rem;
        walk.next();
    };
    auto load_a1 = [&](char *st) __attribute__((always_inline)) {
        PA::template load_direct<16>(wave, late, pitch_a, oa1, late_rem, st);
    };

    f32x4 c[2][2][4][2] = {};      // [A panel][B panel]
    u32x4 x[2][4], w[2][2][2];     // [step][row tile]; [B panel][step][column tile]
    auto read_a = [&](const char *st) __attribute__((always_inline)) {
#pragma unroll
        for (int step = 0; step < 2; ++step)
#pragma unroll
            for (int i = 0; i < 4; ++i) x[step][i] = PA::fragment(st, 0, wm * 64 + i * 16, step);
    };
    auto read_b = [&](auto half, const char *st) __attribute__((always_inline)) {
#pragma unroll
        for (int step = 0; step < 2; ++step)
#pragma unroll
            for (int j = 0; j < 2; ++j)
                w[decltype(half)::value][step][j] = PB::fragment(st, 0, wn * 32 + j * 16, step);
    };
    // The barrier behind the reads and loads, the MFMAs, the barrier behind them.
    // VM: loads that may still be in flight (63: any).
    auto compute = [&](auto vm, auto ha, auto hb) __attribute__((always_inline)) {
        constexpr int HA = decltype(ha)::value, HB = decltype(hb)::value;
        stage_sync<decltype(vm)::value>();
#pragma unroll
        for (int step = 0; step < 2; ++step)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    c[HA][HB][i][j] = mma16<T>(w[HB][step][j], x[step][i], c[HA][HB][i][j]);
        __builtin_amdgcn_sched_barrier(0);
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
    };
    constexpr std::integral_constant<int, 0> zero;
    constexpr std::integral_constant<int, 1> one;
    constexpr std::integral_constant<int, 3 * L> three_panels;
    constexpr std::integral_constant<int, 63> any;
    // Tile s, in the stages a0, a1, b0, b1; `a1_next` is the other A1.
    auto tile = [&](char *a0, char *a1, char *b0, char *b1, char *a1_next)
                    __attribute__((always_inline)) {
        read_b(zero, b0);
        read_a(a0);
        load_a1(a1_next);
        compute(any, zero, zero);
        read_b(one, b1);
        load_a0(a0);
        compute(any, zero, one);
        read_a(a1);
        load_b0(b0);
        compute(any, one, one);
        load_b1(b1);
        compute(three_panels, one, zero);
    };

    load_a0(a00);
    __builtin_amdgcn_sched_barrier(0);
    load_b0(b00);
    __builtin_amdgcn_sched_barrier(0);
    load_b1(b10);
    __builtin_amdgcn_sched_barrier(0);
    load_a1(a10);
    __builtin_amdgcn_sched_barrier(0);
    load_a0(a01);
    __builtin_amdgcn_sched_barrier(0);
    load_b0(b01);
    __builtin_amdgcn_sched_barrier(0);
    load_b1(b11);
    stage_sync<3 * L>();
    if (wm != 0) __builtin_amdgcn_s_barrier();
    int s = 0;
    for (; s + 2 <= count; s += 2) {
        tile(a00, a10, b00, b10, a11);
        tile(a01, a11, b01, b11, a10);
    }
    if (s < count) tile(a00, a10, b00, b10, a11);
    if (wm == 0) __builtin_amdgcn_s_barrier();
    stage_sync<0>();

    // One array takes a wave's sums of one A panel.
    char *mine = wave < 4 ? (wave < 2 ? (wave < 1 ? a00 : a01) : (wave < 3 ? a10 : a11))
                          : (wave < 6 ? (wave < 5 ? b00 : b01) : (wave < 7 ? b10 : b11));
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        epi_put<32>(mine, c[h][0], 0);
        epi_put<32>(mine, c[h][1], 1);
        wave_sync();
        const int row = h * 128 + wm * 64;
        epi_rows<T, GATED, 32, 64>(
            p, batch, part.sums == nullptr ? nullptr : part.sums + row * 256 + wn * 32, 256, mine,
            m0 + row, n0 + wn * 32, n1 + wn * 32);
        wave_sync();
    }
}

// ---- launches ----------------------------------------------------------------------------------

template <typename T, bool AKC, bool BKC, bool GATED>
hipError_t launch_tile(const TilePlan &plan, const TileArgs &a, hipStream_t stream) {
    const unsigned tiles = static_cast<unsigned>(a.tiles_m) * static_cast<unsigned>(a.tiles_n);
    const unsigned whole = static_cast<unsigned>(a.whole);
    const dim3 grid(whole + (tiles - whole) * static_cast<unsigned>(a.splits),
                    static_cast<unsigned>(a.batch));
    if constexpr (AKC) {
        if (plan.few) {
            linear_few<T, BKC, GATED>
                <<<dim3(static_cast<unsigned>(a.tiles_n)), 512, 0, stream>>>(a);
            return hipGetLastError();
        }
    }
    if constexpr (sizeof(T) == 2) {
        if (plan.bm == 256) {
            linear_wide<T, AKC, BKC, GATED><<<grid, 512, 0, stream>>>(a);
            return hipGetLastError();
        }
    }
    // Direct loads of 16 bytes: two workgroups a CU, or, where the grid gives a CU no
    // more than one, stages enough that a second does not fit (the dispatcher would
    // put two on one CU and leave another idle).
#define TRA_TILE(BM, BN, S, DIRECT) \
    linear_tile<T, AKC, BKC, BM, BN, S, DIRECT, GATED><<<grid, 256, 0, stream>>>(a)
    constexpr bool F32 = sizeof(T) == 4;
    const int size = plan.bm == 128 ? 2 : plan.bn == 128 ? 1 : 0;
    if (plan.direct == 16) {
        if (size == 2) plan.deep ? TRA_TILE(128, 128, 4, 16) : TRA_TILE(128, 128, 2, 16);
        if (size == 1) plan.deep ? TRA_TILE(64, 128, 6, 16) : TRA_TILE(64, 128, 3, 16);
        if (size == 0) plan.deep ? TRA_TILE(64, 64, 6, 16) : TRA_TILE(64, 64, 3, 16);
    } else if constexpr (F32) {
        if (size == 2 || (size == 1 && plan.direct == 0)) return hipErrorInvalidValue;
        if (plan.direct == 0)
            TRA_TILE(64, 64, 2, 0);
        else if (size == 1)
            TRA_TILE(64, 128, 3, 4);
        else
            TRA_TILE(64, 64, 3, 4);
    } else {
        if (size == 2) TRA_TILE(128, 128, 2, 0);
        if (size == 1) TRA_TILE(64, 128, 2, 0);
        if (size == 0) TRA_TILE(64, 64, 2, 0);
    }
#undef TRA_TILE
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
