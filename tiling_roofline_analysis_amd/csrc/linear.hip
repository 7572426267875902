// linear.hip -- the C-ABI entry points of the fused linear operators (declared
// in include/tra_gemm.h): argument checks, choice of kernels, launches on the
// caller's stream; and the small kernels around the products, which join a
// split's partial sums and take the gradient of the epilogue.  Errors come back
// as status codes; nothing throws across the ABI and nothing is allocated: scratch
// is the caller's workspace.
#include "tra_gemm.h"

#include <algorithm>
#include <cstdio>
#include <cstring>

#include "linear_epilogue.h"

namespace tra {
namespace {

// ---- joining a split, gradients of the epilogue ----------------------------------------------

// One chunk of columns of a split tile per lane: the partial sums in split order,
// then the epilogue.
template <typename T, bool GATED>
__global__ __launch_bounds__(256) void linear_join(const TileArgs p, int bm, int bn, int blocks) {
    constexpr int V = kChunk<T>;
    const int cols = GATED ? bn / 2 : bn, per_row = cols / V;
    const int at = static_cast<int>(blockIdx.x) / blocks;
    const int item = (static_cast<int>(blockIdx.x) - at * blocks) * 256 + threadIdx.x;
    const int row = item / per_row, col = (item - row * per_row) * V;
    const int batch = blockIdx.y;
    int tm, tn;
    if (bm == 256)
        grouped_tile32<kGroupWide>(p.whole + at, p.tiles_m, p.tiles_n, tm, tn);
    else
        grouped_tile32<kGroupTile>(p.whole + at, p.tiles_m, p.tiles_n, tm, tn);
    const int64_t m = static_cast<int64_t>(tm) * bm + row, n = static_cast<int64_t>(tn) * cols + col;
    if (row >= bm || m >= p.M || n >= p.N) return;
    const int split_tiles = p.tiles_m * p.tiles_n - p.whole, area = bm * bn;
    const float *in = p.partial +
                      (static_cast<int64_t>(batch) * split_tiles + at) * p.splits * area +
                      row * bn + col;
    float z[V] = {}, u[V] = {};
#pragma unroll 4
    for (int s = 0; s < p.splits; ++s, in += area) {
        float t[V];
        load_row<float, V>(in, t);
#pragma unroll
        for (int e = 0; e < V; ++e) z[e] += t[e];
        if constexpr (GATED) {
            load_row<float, V>(in + cols, t);
#pragma unroll
            for (int e = 0; e < V; ++e) u[e] += t[e];
        }
    }
    with_act(p.epi.act, [&](auto act) __attribute__((always_inline)) {
        finish<T, GATED, decltype(act)::value, V>(p.epi, batch, m, n, z, u);
    });
}

// Binary16 holds 40 binades, and dZ = dY u act' can lie outside them where the
// gradients, its products with X and W, do not.  So it is stored times 2^12, which
// fits where its largest finite |dZ| lies in [2^-12, 16); where that lies
// elsewhere, times the power of two that takes it into [2^14, 2^15).  A rounding of
// dZ is then off by half a step or by 2^-25 of the largest |dZ|, whatever dZ's size.
constexpr float kUsualScale = 4096.0f;

__device__ __forceinline__ float dz_scale(float largest) {
    if (largest == 0.0f || (largest >= 1.0f / kUsualScale && largest * kUsualScale <= 65504.0f))
        return kUsualScale;
    // (of a subnormal: the least exponent; the scale and its inverse stay normal)
    const int e = static_cast<int>(__float_as_uint(largest) >> 23) - 127;
    return ldexpf(1.0f, 14 - e < 126 ? 14 - e : 126);
}

// dZ, times `scale`, of 64 chunks of columns (block `bx` of them) and
// rows_per_chunk rows (block `by`), of which this wave takes every fourth; their
// column sums and largest finite |dZ|, unscaled.
template <typename T, bool GATED>
__device__ __forceinline__ void slope_block(const SlopeArgs &p, int bx, int by, float scale,
                                            float (&sum)[kChunk<T>], float &largest) {
    constexpr int V = kChunk<T>;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t n = (static_cast<int64_t>(bx) * 64 + lane) * V;
    const int64_t first = static_cast<int64_t>(by) * p.rows_per_chunk;
    const int64_t end = first + p.rows_per_chunk < p.M ? first + p.rows_per_chunk : p.M;
    const int64_t valid = p.N - n;
    if (valid > 0) {
        with_act(p.act, [&](auto act) __attribute__((always_inline)) {
            constexpr int ACT = decltype(act)::value;
#pragma unroll 2
            for (int64_t m = first + wave; m < end; m += 4) {
                float dy[V], z[V], u[V], dz[V];
                load_part<T, V>(static_cast<const T *>(p.dY) + m * p.lddy + n, valid, dy);
                if (GATED || ACT != TRA_ACT_NONE)
                    load_part<float, V>(p.Z + m * p.ldz + n, valid, z);
                if constexpr (GATED) load_part<float, V>(p.Z + m * p.ldz + p.N + n, valid, u);
                T *out = static_cast<T *>(p.dZ) + m * p.lddz + n;
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    float y;
                    const float d = GATED || ACT != TRA_ACT_NONE ? activate_slope<ACT>(z[e], y) : 1.0f;
                    dz[e] = GATED ? dy[e] * u[e] * d : dy[e] * d;
                    if constexpr (GATED) u[e] = dy[e] * y;
                    sum[e] += dz[e];
                    if constexpr (kScaled<T>) {
                        const float a = fabsf(dz[e]), b = GATED ? fabsf(u[e]) : 0.0f;
                        if (a < INFINITY) largest = fmaxf(largest, a);
                        if (GATED && b < INFINITY) largest = fmaxf(largest, b);
                        dz[e] *= scale;
                        if constexpr (GATED) u[e] *= scale;
                    }
                }
                if (GATED || p.dZ != nullptr) store_part<T, V>(out, valid, dz);
                if constexpr (GATED) store_part<T, V>(out + p.N, valid, u);
            }
        });
    }
}

// The largest of every lane's value in the workgroup of four waves.
__device__ __forceinline__ float largest_of(float v, float (&part)[4]) {
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) v = fmaxf(v, __shfl_xor(v, d));
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
    __syncthreads();
    return fmaxf(fmaxf(part[0], part[1]), fmaxf(part[2], part[3]));
}

// 64 chunks of columns by rows_per_chunk rows per workgroup; its four waves
// take every fourth row and add their column sums in wave order.  Memory bounds
// it: gated 4096 x 8192 bf16 moves 470 MB in 124 us, 3.8 TB/s.
template <typename T, bool GATED>
__global__ __launch_bounds__(256) void linear_slope(const SlopeArgs p) {
    constexpr int V = kChunk<T>;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    float sum[V] = {}, largest = 0.0f;
    slope_block<T, GATED>(p, blockIdx.x, blockIdx.y, kUsualScale, sum, largest);
    if constexpr (kScaled<T>) {
        if (p.largest != nullptr) {
            __shared__ float most[4];
            lds_poison(most, 4);
            largest = largest_of(largest, most);
            if (threadIdx.x == 0)
                p.largest[static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x] = largest;
        }
    }
    if constexpr (!GATED) {
        if (p.colsum == nullptr) return;
        __shared__ __align__(16) float part[4][64 * V];
        lds_poison(&part[0][0], 4 * 64 * V);
#pragma unroll
        for (int e = 0; e < V; ++e) part[wave][lane * V + e] = sum[e];
        __syncthreads();
        for (int i = threadIdx.x; i < 64 * V; i += 256) {
            const int64_t col = static_cast<int64_t>(blockIdx.x) * 64 * V + i;
            if (col < p.N)
                p.colsum[static_cast<int64_t>(blockIdx.y) * p.N + col] =
                    ((part[0][i] + part[1][i]) + part[2][i]) + part[3][i];
        }
    }
}

// Behind linear_slope, whose grid was blocks_x x blocks_y: notes what undoes dZ's
// scale, and where the usual one does not fit writes dZ again.  4096 x 8192: 5 us, or,
// where it writes, 53 (linear_slope 58); gated 5 or 103 (100).  So the usual scale is
// tried first: the exact one, found by a pass of its own, would cost every call the
// second read of dY and Z.
template <typename T, bool GATED>
__global__ __launch_bounds__(256) void linear_rescale(const SlopeArgs p, int blocks_x,
                                                      int64_t blocks) {
    __shared__ float most[4];
    lds_poison(most, 4);
    float largest = 0.0f;
    for (int64_t i = threadIdx.x; i < blocks; i += 256) largest = fmaxf(largest, p.largest[i]);
    const float scale = dz_scale(largest_of(largest, most));
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.undo = 1.0f / scale;
    if (scale == kUsualScale) return;
    for (int64_t b = blockIdx.x; b < blocks; b += gridDim.x) {
        float sum[kChunk<T>] = {};
        slope_block<T, GATED>(p, static_cast<int>(b % blocks_x), static_cast<int>(b / blocks_x),
                              scale, sum, largest);
    }
}

// Sums the chunks in order: 16 columns per workgroup, whose 16 groups of lanes
// take every 16th chunk and are added in order.
template <typename T>
__global__ __launch_bounds__(256) void linear_colsum_join(const float *colsum, int64_t chunks,
                                                          int64_t N, T *out) {
    __shared__ float part[16][16];
    lds_poison(&part[0][0], 256);
    const int j = threadIdx.x & 15, group = threadIdx.x >> 4;
    const int64_t n = static_cast<int64_t>(blockIdx.x) * 16 + j;
    float sum = 0.0f;
    if (n < N) {
#pragma unroll 4
        for (int64_t c = group; c < chunks; c += 16) sum += colsum[c * N + n];
    }
    part[group][j] = sum;
    __syncthreads();
    if (group == 0 && n < N) {
        for (int i = 1; i < 16; ++i) sum += part[i][j];
        out[n] = static_cast<T>(sum);
    }
}

template <typename T>
hipError_t launch_join(const TilePlan &t, const TileArgs &a, hipStream_t stream) {
    const int64_t rows = a.M < t.bm ? a.M : t.bm;
    const int blocks =
        static_cast<int>(ceil_div(rows * (t.gated ? t.bn / 2 : t.bn) / kChunk<T>, 256));
    const dim3 grid(static_cast<unsigned>((a.tiles_m * a.tiles_n - a.whole) * blocks),
                    static_cast<unsigned>(a.batch));
    if (t.gated)
        linear_join<T, true><<<grid, 256, 0, stream>>>(a, t.bm, t.bn, blocks);
    else
        linear_join<T, false><<<grid, 256, 0, stream>>>(a, t.bm, t.bn, blocks);
    return hipGetLastError();
}

template <typename T>
hipError_t launch_slope(bool gated, const SlopeArgs &a, hipStream_t stream) {
    const dim3 grid(static_cast<unsigned>(ceil_div(a.N, 64 * kChunk<T>)),
                    static_cast<unsigned>(ceil_div(a.M, a.rows_per_chunk)));
    if (gated)
        linear_slope<T, true><<<grid, 256, 0, stream>>>(a);
    else
        linear_slope<T, false><<<grid, 256, 0, stream>>>(a);
    if constexpr (kScaled<T>) {
        if (a.largest != nullptr) {
            const hipError_t err = hipGetLastError();
            if (err != hipSuccess) return err;
            const int64_t blocks = static_cast<int64_t>(grid.x) * grid.y;
            const dim3 again(static_cast<unsigned>(std::min<int64_t>(blocks, 1024)));
            const int blocks_x = static_cast<int>(grid.x);
            if (gated)
                linear_rescale<T, true><<<again, 256, 0, stream>>>(a, blocks_x, blocks);
            else
                linear_rescale<T, false><<<again, 256, 0, stream>>>(a, blocks_x, blocks);
        }
    }
    return hipGetLastError();
}

template <typename T>
hipError_t launch_colsum(const float *colsum, int64_t chunks, int64_t N, void *out,
                         hipStream_t stream) {
    linear_colsum_join<T><<<dim3(static_cast<unsigned>(ceil_div(N, 16))), 256, 0, stream>>>(
        colsum, chunks, N, static_cast<T *>(out));
    return hipGetLastError();
}

}  // namespace
}  // namespace tra

namespace {

using tra::ceil_div;
using tra::TileArgs;
using tra::TileForm;
using tra::TilePlan;

// M, N, K: indices along an axis, rounded up to whole tiles and doubled for a gated
// result, fit 32 bits.
constexpr int64_t kMaxSize = int64_t{1} << 30;
constexpr size_t kAlign = 256;              // of the workspace's parts

size_t align_up(size_t x) { return (x + kAlign - 1) & ~(kAlign - 1); }

int64_t elem_bytes(int dtype) { return dtype == TRA_DTYPE_F32 ? 4 : 2; }

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Rows of a matrix at p start 16-byte aligned.
bool rows16(const void *p, int64_t ld, int64_t bytes) {
    return aligned16(p) && ld * bytes % 16 == 0;
}

// A row-major view: rows x cols elements of `bytes` bytes.
struct View {
    const void *p;
    int64_t rows, cols, ld, bytes;

    bool empty() const { return rows <= 0 || cols <= 0; }
    // A view the kernels may touch: aligned to its elements, rows that do not
    // overlap, extent in the address space.
    bool valid() const {
        if (empty()) return true;
        if (p == nullptr || ld < cols) return false;
        const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
        if (lo % static_cast<uintptr_t>(bytes) != 0) return false;
        const __int128 extent = (static_cast<__int128>(rows - 1) * ld + cols) * bytes;
        return extent <= static_cast<__int128>(INT64_MAX) &&
               static_cast<__int128>(lo) + extent <= static_cast<__int128>(UINTPTR_MAX);
    }
    uintptr_t lo() const { return reinterpret_cast<uintptr_t>(p); }
    uintptr_t hi() const {
        return lo() + static_cast<uintptr_t>(((rows - 1) * ld + cols) * bytes);
    }
};

// True if the two (valid) views share an element, or might: column ranges of
// one row-major buffer (same row pitch) interleave without sharing any.
bool share(const View &a, const View &b) {
    if (a.empty() || b.empty() || a.hi() <= b.lo() || b.hi() <= a.lo()) return false;
    if (a.rows == 1 || b.rows == 1 || a.ld * a.bytes != b.ld * b.bytes) return true;
    const View &x = a.lo() <= b.lo() ? a : b, &y = a.lo() <= b.lo() ? b : a;
    const int64_t pitch = x.ld * x.bytes;
    const int64_t at = static_cast<int64_t>((y.lo() - x.lo()) % static_cast<uintptr_t>(pitch));
    return at < x.cols * x.bytes || at + y.cols * y.bytes > pitch;
}

bool same(const View &a, const View &b) { return a.p == b.p && (a.ld == b.ld || a.rows <= 1); }

bool valid_act(int act) { return act >= TRA_ACT_NONE && act < TRA_ACT_COUNT; }
bool valid_dtype(int d) { return d >= TRA_DTYPE_F32 && d < TRA_DTYPE_COUNT; }

// The weight as stored: N x K when w_trans, else K x N.
View weight(const void *p, int w_trans, int64_t N, int64_t K, int64_t ld, int64_t bytes) {
    return w_trans ? View{p, N, K, ld, bytes} : View{p, K, N, ld, bytes};
}

// Bytes a lane with which an operand can go straight into LDS: 16 where every line
// starts 16-byte aligned and is whole chunks long, 4 for any other binary32, 0 if a
// tile's byte offsets (256 lines) may pass 2^31, and for 16 bits of any alignment.
int direct_bytes(const void *p, int64_t ld, int64_t line, int64_t bytes) {
    if (ld * bytes >= (int64_t{1} << 22)) return 0;
    return rows16(p, ld, bytes) && line * bytes % 16 == 0 ? 16 : bytes == 4 ? 4 : 0;
}

// The same for `line` elements that start `offset` elements into lines that allow `d`.
int at_offset(int d, int64_t offset, int64_t bytes) {
    return d < 16 || offset * bytes % 16 == 0 ? d : bytes == 4 ? 4 : 0;
}

// How a kernel of one tile size goes, in microseconds, as measured on MI355X with
// 1 to 12 workgroups a CU and 16 to 64 K tiles (a K tile is 128 bytes of a row).
struct TileClass {
    int bm, bn;
    int resident;     // workgroups a CU holds
    double alone;     // per K tile, one workgroup on a CU
    double shared;    // per K tile and workgroup, CU full
    double base;      // launch, first loads, epilogue without its stores
};

constexpr int64_t kCUs = 256;
constexpr double kBytesPerUs = 4.8e6;     // memory, as a large copy reaches
// What one workgroup's loads in flight can ask for, as fitted: of 8300 random forward
// products (M to 2048; N, K from 128 to 12288; weights from memory), the 900 whose plan
// it changes between 22 and 32 GB/s took, against the best of those plans, 4.8% longer
// in the geometric mean at 22, 3.8 at 24, 3.3 at 26, 3.3 at 28, 3.6 at 30 and 4.1 at 32;
// 150 more with M to 64, 5.8, 4.7, 4.3, 3.7, 3.3 and 3.6.
constexpr double kBytesPerUsWg = 2.8e4;

// [loads][16-bit, binary32]: direct, 16 bytes a lane; through registers; direct, 4
// bytes a lane.  The 256 x 256 kernel is built for direct 16-bit loads only; 128 x 128
// in binary32 with other than 16-byte loads needs more VGPRs than there are.
// Through registers binary32 goes only with rows of 4 MB or more, in one tile size.
constexpr TileClass kClasses[3][2][4] = {
    {{{256, 256, 1, 1.28, 1.42, 5.7},
      {128, 128, 2, 0.50, 0.47, 5.2},
      {64, 128, 2, 0.30, 0.27, 4.5},
      {64, 64, 3, 0.21, 0.185, 4.0}},
     {{128, 128, 2, 1.77, 1.77, 5.6},
      {64, 128, 2, 0.93, 0.90, 4.5},
      {64, 64, 3, 0.505, 0.46, 4.0},
      {0, 0, 0, 0.0, 0.0, 0.0}}},
    {{{128, 128, 2, 0.97, 0.68, 5.2},
      {64, 128, 3, 0.85, 0.455, 4.5},
      {64, 64, 4, 0.70, 0.32, 4.0},
      {0, 0, 0, 0.0, 0.0, 0.0}},
     {{64, 64, 4, 0.74, 0.545, 4.0}}},
    {{},
     {{64, 128, 2, 1.05, 0.96, 4.5},
      {64, 64, 3, 0.58, 0.52, 4.0},
      {0, 0, 0, 0.0, 0.0, 0.0},
      {0, 0, 0, 0.0, 0.0, 0.0}}}};

// The product's plan: the kernel, tile and split with the least predicted time.
//   Tiles: a CU runs its share of the workgroups (tiles x splits), `resident` at a
//   time; the K loop is bounded by the operands' bytes too; the results' stores
//   add to it.  A split stores binary32 sums and adds a launch that reads them.
//   Split are all tiles, where they are few, or those of the last, partial round
//   over the CUs, whose K loops would leave most CUs idle.
//   Few rows: the weights' bytes at the rate that their strips can ask for (one
//   strip, of 512 lanes, about 25 GB/s; 64-byte pieces of rows K apart reach about
//   half of the memory's rate in 16 bits; unaligned 16-bit rows three quarters).
// Kept pre-activations have no part in it, though their stores add to the time: a
// forward pass that keeps them gives the same bits as one that does not (a
// checkpoint's recomputation).  Of 3000 random forward calls 82 had another plan with
// their stores counted.
TilePlan plan_tile(TileForm form, bool gated, int dtype, int64_t M, int64_t N, int64_t K, int segs,
                   int batch, int direct) {
    const int64_t b = elem_bytes(dtype), slice = 128 / b;
    const bool f32 = dtype == TRA_DTYPE_F32;
    const int64_t k_tiles = std::max<int64_t>(1, segs * ceil_div(K, slice));
    const double columns = static_cast<double>(N) * (gated ? 2 : 1);      // of z and u
    const double in = static_cast<double>(batch) * segs * K * (static_cast<double>(M) + columns) * b;
    TilePlan best{};
    double best_us = 0.0;
    for (const TileClass &c : kClasses[direct == 16 ? 0 : direct == 4 ? 2 : 1][f32 ? 1 : 0]) {
        if (c.bm == 0) break;
        const int64_t tiles = std::max<int64_t>(
            1, ceil_div(M, c.bm) * ceil_div(N, gated ? c.bn / 2 : c.bn));     // of a batch
        // 64-byte lines (16-bit weights, 64 x 64 tiles, not k-contiguous)
        const double most = kBytesPerUs * (form == tra::kFormKN && !f32 && c.bn == 64 ? 0.7 : 1.0);
        const double area = std::min<double>(M, c.bm) * std::min<double>(columns, c.bn);
        const double out = (gated ? 0.5 : 1.0) * b;     // bytes stored per column of z or u
        // K loops of n workgroups of `per` K tiles; a little to begin another round
        auto loops = [&](int64_t n, int64_t per) {
            const int64_t wave = kCUs * c.resident;
            const int64_t full = n / wave, rest = ceil_div(n % wave, kCUs);
            return per * (full * std::max(c.alone, c.resident * c.shared) +
                          (rest > 0 ? std::max(c.alone, rest * c.shared) : 0.0)) +
                   (c.resident == 1 ? 3.0 : 1.5) *
                       std::max<int64_t>(0, full + (rest > 0 ? 1 : 0) - 1);
        };
        auto consider = [&](int64_t whole, int64_t want) {
            const int64_t per = ceil_div(k_tiles, want), splits = ceil_div(k_tiles, per);
            if (splits != want || want > k_tiles) return;
            const int64_t parts = batch * (tiles - whole) * splits, n = batch * whole + parts;
            double loop = (whole > 0 ? loops(batch * whole, k_tiles) : 0.0) +
                          (parts > 0 ? loops(parts, per) : 0.0);
            loop = std::max(loop, in / std::min(most, n * kBytesPerUsWg));
            const double sums = splits > 1 ? parts * area * 4.0 : 0.0;
            const double stored = sums + batch * (splits > 1 ? whole : tiles) * area * out;
            double us = c.base + loop + stored / kBytesPerUs;
            if (splits > 1) us += 2.5 + 0.12 * splits + sums / kBytesPerUs;
            if (best_us == 0.0 || us < best_us) {
                best_us = us;
                best.bm = c.bm;
                best.bn = c.bn;
                best.whole = static_cast<int>(splits > 1 ? whole : tiles);
                best.splits = static_cast<int>(splits);
                best.deep = direct == 16 && n <= kCUs;
                best.partial_bytes =
                    splits > 1 ? static_cast<size_t>(parts) * c.bm * c.bn * sizeof(float) : 0;
            }
        };
        // none split; all split; those past the last whole round over the CUs split
        consider(tiles, 1);
        for (int64_t want = 2; want <= 32 && tiles * batch * want <= 1024; ++want)
            consider(0, want);
        const int64_t rounds = tiles * batch / kCUs * kCUs / batch;
        if (rounds > 0 && rounds < tiles && kCUs % batch == 0)
            for (int64_t want = 2; want <= 16; ++want) consider(rounds, want);
    }
    const int64_t strip = form == tra::kFormKK ? 16 : 64 / b;
    if (form != tra::kFormNN && M <= 16 && K >= 16 / b && N >= 4 / b) {
        const double strips = static_cast<double>(ceil_div(N, strip));
        const double most = form == tra::kFormKK ? (strips < 512 ? 3.9e6 : 4.9e6)
                                                 : (f32 ? 3.8e6 : 2.4e6);
        const double each = form == tra::kFormKK ? 2.6e4 : f32 ? 1.8e4 : 3.0e4;
        const double us = 2.8 + segs * static_cast<double>(K) * columns * b * (1.0 + M / 80.0) /
                                    std::min(most, strips * each) / (direct != 0 || f32 ? 1.0 : 0.75);
        if (us < best_us) {
            best = TilePlan{};
            best.few = true;
            best.whole = static_cast<int>(ceil_div(N, strip));
            best.bm = 16;
            best.bn = static_cast<int>(gated ? 2 * strip : strip);
            best.splits = 1;
        }
    }
    best.form = form;
    best.gated = gated;
    best.direct = direct;
    return best;
}

// Fills in what follows from the plan and checks the launch's size.
tra_status finish_args(const TilePlan &t, int dtype, TileArgs &a, float *partial) {
    const int64_t slice = 128 / elem_bytes(dtype);
    const int64_t tm = ceil_div(a.M, t.bm), tn = ceil_div(a.N, t.gated ? t.bn / 2 : t.bn);
    // kMaxGridLanes work-items (512 a workgroup), and tile indices in 32 bits
    const __int128 tiles = static_cast<__int128>(tm) * tn;
    const __int128 whole = t.splits > 1 ? static_cast<__int128>(t.whole) : tiles;
    if ((whole + (tiles - whole) * t.splits) * 512 > tra::kMaxGridLanes)
        return TRA_ERR_UNSUPPORTED;
    a.tiles_m = static_cast<int>(tm);
    a.tiles_n = static_cast<int>(tn);
    a.seg_tiles = static_cast<int>(ceil_div(a.K, slice));
    a.k_tiles = a.segs * a.seg_tiles;
    a.whole = t.splits > 1 ? t.whole : a.tiles_m * a.tiles_n;
    a.splits = t.splits;
    a.tiles_per_split = static_cast<int>(ceil_div(std::max(a.k_tiles, 1), t.splits));
    a.partial = t.splits > 1 ? partial : nullptr;
    a.epi.M = a.M;
    a.epi.N = a.N;
    return TRA_OK;
}

hipError_t run_tile(int dtype, const TilePlan &t, const TileArgs &a, hipStream_t s) {
    switch (dtype) {
        case TRA_DTYPE_F32: return tra::LinearKernels<float>::tile(t, a, s);
        case TRA_DTYPE_BF16: return tra::LinearKernels<__bf16>::tile(t, a, s);
        default: return tra::LinearKernels<_Float16>::tile(t, a, s);
    }
}

hipError_t run_join(int dtype, const TilePlan &t, const TileArgs &a, hipStream_t s) {
    switch (dtype) {
        case TRA_DTYPE_F32: return tra::launch_join<float>(t, a, s);
        case TRA_DTYPE_BF16: return tra::launch_join<__bf16>(t, a, s);
        default: return tra::launch_join<_Float16>(t, a, s);
    }
}

hipError_t run_product(int dtype, const TilePlan &t, const TileArgs &a, hipStream_t s) {
    const hipError_t err = run_tile(dtype, t, a, s);
    return err == hipSuccess && t.splits > 1 ? run_join(dtype, t, a, s) : err;
}

tra_status status_of(hipError_t err) {
    if (err == hipSuccess) return TRA_OK;
    tra::record_hip_error(err);
    return TRA_ERR_HIP;
}

bool workspace_ok(const void *ws, uint64_t have, size_t need) {
    return need == 0 || (ws != nullptr && have >= need &&
                         (reinterpret_cast<uintptr_t>(ws) & (kAlign - 1)) == 0);
}

// ---- forward ----------------------------------------------------------------------

bool sizes_ok(int64_t M, int64_t N, int64_t K) { return M >= 0 && N >= 0 && K >= 0; }

TilePlan plan_forward(const tra_linear_args &a) {
    const int64_t b = elem_bytes(a.dtype);
    const bool gated = a.gated != 0;
    const int direct = std::min({direct_bytes(a.X, a.ldx, a.K, b),
                                 direct_bytes(a.W, a.ldw, a.w_trans ? a.K : a.N, b),
                                 gated ? direct_bytes(a.W2, a.ldw, a.w_trans ? a.K : a.N, b) : 16});
    return plan_tile(a.w_trans ? tra::kFormKK : tra::kFormKN, gated, a.dtype, a.M, a.N,
                     a.K, 1, 1, direct);
}

// Host-side checks; launches nothing.
tra_status check_forward(const tra_linear_args *p) {
    if (p == nullptr) return TRA_ERR_INVALID_ARG;
    const tra_linear_args &a = *p;
    const bool gated = a.gated != 0;
    if (!valid_dtype(a.dtype) || !valid_act(a.act) || (a.w_trans != 0 && a.w_trans != 1) ||
        (a.gated != 0 && a.gated != 1) || !sizes_ok(a.M, a.N, a.K))
        return TRA_ERR_INVALID_ARG;
    if (gated && (a.bias != nullptr || a.R != nullptr)) return TRA_ERR_INVALID_ARG;
    if (!gated && a.W2 != nullptr) return TRA_ERR_INVALID_ARG;
    if (a.M == 0 || a.N == 0) return TRA_OK;
    if (gated && a.W2 == nullptr && a.K > 0) return TRA_ERR_INVALID_ARG;
    if (a.M > kMaxSize || a.N > kMaxSize || a.K > kMaxSize) return TRA_ERR_UNSUPPORTED;
    const int64_t b = elem_bytes(a.dtype);
    const View X{a.X, a.M, a.K, a.ldx, b};
    const View W = weight(a.W, a.w_trans, a.N, a.K, a.ldw, b);
    const View W2 = gated ? weight(a.W2, a.w_trans, a.N, a.K, a.ldw, b) : View{};
    const View bias{a.bias, a.bias != nullptr, a.N, a.N, b};
    const View R{a.R, a.R != nullptr ? a.M : 0, a.N, a.ldr, b};
    const View Y{a.Y, a.M, a.N, a.ldy, b};
    const View Z{a.Z, a.Z != nullptr ? a.M : 0, gated ? 2 * a.N : a.N, a.ldz, 4};
    const View in[] = {X, W, W2, bias, R};
    for (const View &v : in)
        if (!v.valid()) return TRA_ERR_INVALID_ARG;
    if (!Y.valid() || !Z.valid() || share(Y, Z)) return TRA_ERR_INVALID_ARG;
    // R in place: the lane that reads an element of R writes it, and no other.  That
    // holds for R only, not for another operand that starts where R does.
    for (const View &v : in) {
        const bool in_place = &v == &in[4] && same(R, Y);
        if (share(v, Z) || (share(v, Y) && !in_place)) return TRA_ERR_INVALID_ARG;
    }
    return TRA_OK;
}

tra_status forward(const tra_linear_args *p, void *stream) {
    tra_status st = check_forward(p);
    if (st != TRA_OK || p->M == 0 || p->N == 0) return st;
    const tra_linear_args &a = *p;
    const bool gated = a.gated != 0;
    const TilePlan plan = plan_forward(a);
    if (!workspace_ok(a.workspace, a.workspace_bytes, plan.partial_bytes))
        return TRA_ERR_INVALID_ARG;
    TileArgs t{};
    t.A = a.X;
    t.lda = a.ldx;
    t.B[0] = a.W;
    t.B[1] = gated ? a.W2 : a.W;
    t.ldb = a.ldw;
    t.M = a.M;
    t.N = a.N;
    t.K = a.K;
    t.segs = t.batch = 1;
    t.epi.bias = a.bias;
    t.epi.R = a.R;
    t.epi.ldr = a.ldr;
    t.epi.Y[0] = a.Y;
    t.epi.ldy = a.ldy;
    t.epi.Z = a.Z;
    t.epi.ldz = a.ldz;
    t.epi.act = a.act;
    st = finish_args(plan, a.dtype, t, static_cast<float *>(a.workspace));
    if (st != TRA_OK) return st;
    return status_of(run_product(a.dtype, plan, t, static_cast<hipStream_t>(stream)));
}

// ---- backward ----------------------------------------------------------------------

// The parts of a backward call and where they live in its workspace.
struct GradPlan {
    bool slope;             // dZ differs from dY: an elementwise pass writes it
    size_t scale_bytes;     // binary16: what undoes dZ's scale, then the largest |dZ| by workgroup
    int64_t lddz;           // elements
    size_t dz_bytes;
    int64_t chunks;         // row chunks of the column sums
    int rows_per_chunk;
    size_t colsum_bytes;
    TilePlan dx, dw;
    size_t product_bytes;   // the larger of the two splits' partials
    size_t total;
};

// Rows per workgroup of the elementwise pass: about 1024 workgroups, and no
// more than 64 chunks where their column sums are to be joined.
void plan_slope(const tra_linear_grad_args &a, GradPlan &g) {
    const int64_t cols = std::max<int64_t>(1, ceil_div(a.N, 64 * (16 / elem_bytes(a.dtype))));
    int64_t chunks = std::max<int64_t>(1, 1024 / cols);
    if (a.dbias != nullptr) chunks = std::min<int64_t>(chunks, 64);
    const int64_t rows = std::max<int64_t>(4, ceil_div(a.M, chunks));
    g.rows_per_chunk = static_cast<int>(rows);
    g.chunks = ceil_div(a.M, rows);
}

GradPlan plan_backward(const tra_linear_grad_args &a) {
    GradPlan g{};
    const bool gated = a.gated != 0;
    const int64_t b = elem_bytes(a.dtype);
    const int64_t width = gated ? 2 * a.N : a.N;
    g.slope = gated || a.act != TRA_ACT_NONE;
    g.lddz = (width + 7) / 8 * 8;
    g.dz_bytes = g.slope ? align_up(static_cast<size_t>(a.M) * static_cast<size_t>(g.lddz * b)) : 0;
    plan_slope(a, g);
    g.colsum_bytes =
        a.dbias != nullptr ? align_up(static_cast<size_t>(g.chunks * a.N) * sizeof(float)) : 0;
    if (g.slope && a.dtype == TRA_DTYPE_F16)
        g.scale_bytes = align_up(
            static_cast<size_t>(1 + ceil_div(a.N, 64 * (16 / b)) * g.chunks) * sizeof(float));
    // dZ as an operand: the workspace's copy is aligned
    const int64_t ldz = g.slope ? g.lddz : a.lddy;
    const void *dz = g.slope ? nullptr : a.dY;
    const int dz_direct = at_offset(direct_bytes(dz, ldz, a.N, b), gated ? a.N : 0, b);
    if (a.dX != nullptr) {
        const int64_t line = a.w_trans ? a.K : a.N;
        const int direct = std::min({dz_direct, direct_bytes(a.W, a.ldw, line, b),
                                     gated ? direct_bytes(a.W2, a.ldw, line, b) : 16});
        g.dx = plan_tile(a.w_trans ? tra::kFormKN : tra::kFormKK, false, a.dtype, a.M, a.K, a.N,
                         gated ? 2 : 1, 1, direct);
    }
    if (a.dW != nullptr) {
        const int direct = std::min(dz_direct, direct_bytes(a.X, a.ldx, a.K, b));
        g.dw = plan_tile(tra::kFormNN, false, a.dtype, a.w_trans ? a.N : a.K,
                         a.w_trans ? a.K : a.N, a.M, 1, gated ? 2 : 1, direct);
    }
    g.product_bytes = align_up(std::max(g.dx.partial_bytes, g.dw.partial_bytes));
    g.total = g.dz_bytes + g.scale_bytes + g.colsum_bytes + g.product_bytes;
    return g;
}

tra_status check_backward(const tra_linear_grad_args *p) {
    if (p == nullptr) return TRA_ERR_INVALID_ARG;
    const tra_linear_grad_args &a = *p;
    const bool gated = a.gated != 0;
    if (!valid_dtype(a.dtype) || !valid_act(a.act) || (a.w_trans != 0 && a.w_trans != 1) ||
        (a.gated != 0 && a.gated != 1) || !sizes_ok(a.M, a.N, a.K))
        return TRA_ERR_INVALID_ARG;
    if (gated ? a.dbias != nullptr || (a.dW == nullptr) != (a.dW2 == nullptr)
              : a.W2 != nullptr || a.dW2 != nullptr)
        return TRA_ERR_INVALID_ARG;
    if (a.M > kMaxSize || a.N > kMaxSize || a.K > kMaxSize) return TRA_ERR_UNSUPPORTED;
    // linear_colsum_join: 16 lanes a column
    if (a.dbias != nullptr && a.N * 16 > tra::kMaxGridLanes - 256) return TRA_ERR_UNSUPPORTED;
    const int64_t b = elem_bytes(a.dtype);
    const bool slope = gated || a.act != TRA_ACT_NONE;
    const int64_t wz = gated ? 2 * a.N : a.N;
    const View dY{a.dY, a.M, a.N, a.lddy, b};
    const View Z{a.Z, slope ? a.M : 0, wz, a.ldz, 4};
    const View X{a.X, a.dW != nullptr ? a.M : 0, a.K, a.ldx, b};
    View W = weight(a.W, a.w_trans, a.N, a.K, a.ldw, b);
    View W2 = weight(a.W2, a.w_trans, a.N, a.K, a.ldw, b);
    if (a.dX == nullptr) W.rows = W2.rows = 0;
    if (!gated) W2.rows = 0;
    const View in[] = {dY, Z, X, W, W2};
    for (const View &v : in)
        if (!v.valid()) return TRA_ERR_INVALID_ARG;
    const View dX{a.dX, a.dX != nullptr ? a.M : 0, a.K, a.lddx, b};
    View dW = weight(a.dW, a.w_trans, a.N, a.K, a.lddw, b);
    View dW2 = weight(a.dW2, a.w_trans, a.N, a.K, a.lddw, b);
    if (a.dW == nullptr) dW.rows = 0;
    if (a.dW2 == nullptr) dW2.rows = 0;
    const View db{a.dbias, a.dbias != nullptr, a.N, a.N, b};
    const View out[] = {dX, dW, dW2, db};
    for (int i = 0; i < 4; ++i) {
        if (!out[i].valid()) return TRA_ERR_INVALID_ARG;
        for (const View &v : in)
            if (share(out[i], v)) return TRA_ERR_INVALID_ARG;
        for (int j = 0; j < i; ++j)
            if (share(out[i], out[j])) return TRA_ERR_INVALID_ARG;
    }
    return TRA_OK;
}

hipError_t run_slope(int dtype, bool gated, const tra::SlopeArgs &s, hipStream_t st) {
    switch (dtype) {
        case TRA_DTYPE_F32: return tra::launch_slope<float>(gated, s, st);
        case TRA_DTYPE_BF16: return tra::launch_slope<__bf16>(gated, s, st);
        default: return tra::launch_slope<_Float16>(gated, s, st);
    }
}

hipError_t run_colsum(int dtype, const float *colsum, int64_t chunks, int64_t N, void *out,
                      hipStream_t st) {
    switch (dtype) {
        case TRA_DTYPE_F32:
            return tra::launch_colsum<float>(colsum, chunks, N, out, st);
        case TRA_DTYPE_BF16:
            return tra::launch_colsum<__bf16>(colsum, chunks, N, out, st);
        default: return tra::launch_colsum<_Float16>(colsum, chunks, N, out, st);
    }
}

tra_status backward(const tra_linear_grad_args *p, void *stream_) {
    tra_status st = check_backward(p);
    if (st != TRA_OK) return st;
    const tra_linear_grad_args &a = *p;
    const bool gated = a.gated != 0;
    const hipStream_t stream = static_cast<hipStream_t>(stream_);
    const GradPlan g = plan_backward(a);
    if (!workspace_ok(a.workspace, a.workspace_bytes, g.total)) return TRA_ERR_INVALID_ARG;
    char *ws = static_cast<char *>(a.workspace);
    void *dz_ws = ws;
    float *scale = reinterpret_cast<float *>(ws + g.dz_bytes);
    float *colsum = reinterpret_cast<float *>(ws + g.dz_bytes + g.scale_bytes);
    float *partial =
        reinterpret_cast<float *>(ws + g.dz_bytes + g.scale_bytes + g.colsum_bytes);
    const void *dz = g.slope ? dz_ws : a.dY;
    const int64_t lddz = g.slope ? g.lddz : a.lddy;

    // Both products are set up, and refused if too large, before anything runs.
    const bool want_dx = a.dX != nullptr && a.M > 0 && a.K > 0;
    const bool want_dw = a.dW != nullptr && a.N > 0 && a.K > 0;
    TileArgs tx{}, tw{};
    const bool need_dz = g.slope && ((want_dx && a.N > 0) || (want_dw && a.M > 0));
    // (an empty sum needs nothing undone, and no pass notes it)
    const bool scaled = need_dz && a.M > 0 && a.N > 0 && g.scale_bytes > 0;
    tx.epi.undo = tw.epi.undo = scaled ? scale : nullptr;
    if (want_dx) {
        tx.A = dz;
        tx.lda = lddz;
        tx.a_seg = a.N;
        tx.B[0] = a.W;
        tx.B[1] = gated ? a.W2 : a.W;
        tx.ldb = a.ldw;
        tx.M = a.M;
        tx.N = a.K;
        tx.K = a.N;
        tx.segs = gated ? 2 : 1;
        tx.batch = 1;
        tx.epi.Y[0] = a.dX;
        tx.epi.ldy = a.lddx;
        tx.epi.act = TRA_ACT_NONE;
        if ((st = finish_args(g.dx, a.dtype, tx, partial)) != TRA_OK) return st;
    }
    if (want_dw) {
        // dW = X^T dZ, stored K x N; or its transpose dZ^T X, stored N x K
        tw.A = a.w_trans ? dz : a.X;
        tw.lda = a.w_trans ? lddz : a.ldx;
        tw.B[0] = tw.B[1] = a.w_trans ? a.X : dz;
        tw.ldb = a.w_trans ? a.ldx : lddz;
        tw.a_batch = a.w_trans ? a.N : 0;
        tw.b_batch = a.w_trans ? 0 : a.N;
        tw.M = a.w_trans ? a.N : a.K;
        tw.N = a.w_trans ? a.K : a.N;
        tw.K = a.M;
        tw.segs = 1;
        tw.batch = gated ? 2 : 1;
        tw.epi.Y[0] = a.dW;
        tw.epi.Y[1] = a.dW2;
        tw.epi.ldy = a.lddw;
        tw.epi.act = TRA_ACT_NONE;
        if ((st = finish_args(g.dw, a.dtype, tw, partial)) != TRA_OK) return st;
    }

    hipError_t err = hipSuccess;
    if (a.M > 0 && a.N > 0 && (need_dz || a.dbias != nullptr)) {
        tra::SlopeArgs s{};
        s.dY = a.dY;
        s.lddy = a.lddy;
        s.Z = g.slope ? a.Z : nullptr;
        s.ldz = a.ldz;
        s.dZ = need_dz ? dz_ws : nullptr;
        s.lddz = lddz;
        s.colsum = a.dbias != nullptr ? colsum : nullptr;
        s.undo = scaled ? scale : nullptr;
        s.largest = scaled ? scale + 1 : nullptr;
        s.M = a.M;
        s.N = a.N;
        s.rows_per_chunk = g.rows_per_chunk;
        s.act = a.act;
        err = run_slope(a.dtype, gated, s, stream);
    }
    if (err == hipSuccess && a.dbias != nullptr && a.N > 0)
        err = run_colsum(a.dtype, colsum, a.M > 0 ? g.chunks : 0, a.N, a.dbias, stream);
    if (err == hipSuccess && want_dx) err = run_product(a.dtype, g.dx, tx, stream);
    if (err == hipSuccess && want_dw) err = run_product(a.dtype, g.dw, tw, stream);
    return status_of(err);
}

// Appends a plan to the text in buf.
void describe_plan(const TilePlan &t, const char *prefix, char *buf, size_t len) {
    const size_t used = std::strlen(buf);
    const char *p = prefix;
    std::snprintf(buf + used, len - used,
                  "%s%skernel=%s %stile=%dx%d %sloads=%s %sload_bytes=%d %sstages=%d %swhole=%d "
                  "%ssplits=%d",
                  used > 0 ? " " : "", p,
                  t.few ? "linear_few" : "linear_tile", p, t.bm, t.bn, p,
                  t.few || t.direct == 0 ? "registers" : "direct", p, t.few ? 0 : t.direct, p,
                  tra::plan_stages(t), p, t.whole, p, t.splits);
}

}  // namespace

extern "C" {

tra_status tra_linear(const tra_linear_args *args, void *stream) { return forward(args, stream); }

tra_status tra_linear_workspace_size(const tra_linear_args *args, size_t *bytes) {
    const tra_status st = check_forward(args);
    if (st != TRA_OK || bytes == nullptr) return st != TRA_OK ? st : TRA_ERR_INVALID_ARG;
    *bytes = args->M == 0 || args->N == 0 ? 0 : plan_forward(*args).partial_bytes;
    return TRA_OK;
}

tra_status tra_linear_backward(const tra_linear_grad_args *args, void *stream) {
    return backward(args, stream);
}

tra_status tra_linear_backward_workspace_size(const tra_linear_grad_args *args, size_t *bytes) {
    const tra_status st = check_backward(args);
    if (st != TRA_OK || bytes == nullptr) return st != TRA_OK ? st : TRA_ERR_INVALID_ARG;
    *bytes = plan_backward(*args).total;
    return TRA_OK;
}

tra_status tra_linear_describe(const tra_linear_args *args, char *buf, size_t len) {
    const tra_status st = check_forward(args);
    if (st != TRA_OK) return st;
    if (buf == nullptr) return len == 0 ? TRA_OK : TRA_ERR_INVALID_ARG;
    if (len == 0) return TRA_OK;
    buf[0] = '\0';
    if (args->M == 0 || args->N == 0) {
        std::snprintf(buf, len, "kernel=none");
        return TRA_OK;
    }
    const TilePlan t = plan_forward(*args);
    describe_plan(t, "", buf, len);
    const size_t used = std::strlen(buf);
    std::snprintf(buf + used, len - used, " workspace_bytes=%zu", t.partial_bytes);
    return TRA_OK;
}

tra_status tra_linear_backward_describe(const tra_linear_grad_args *args, char *buf, size_t len) {
    const tra_status st = check_backward(args);
    if (st != TRA_OK) return st;
    if (buf == nullptr) return len == 0 ? TRA_OK : TRA_ERR_INVALID_ARG;
    if (len == 0) return TRA_OK;
    const GradPlan g = plan_backward(*args);
    buf[0] = '\0';
    if (args->dX != nullptr && args->M > 0 && args->K > 0) describe_plan(g.dx, "dx_", buf, len);
    if (args->dW != nullptr && args->N > 0 && args->K > 0) describe_plan(g.dw, "dw_", buf, len);
    const size_t used = std::strlen(buf);
    std::snprintf(buf + used, len - used, "%sworkspace_bytes=%zu", used > 0 ? " " : "", g.total);
    return TRA_OK;
}

}  // extern "C"
