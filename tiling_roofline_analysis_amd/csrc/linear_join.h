// linear_join.h -- finishing the tiles of a product that were split along K.
#pragma once

#include "linear_epilogue.h"

namespace tra {
namespace {

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

}  // namespace
}  // namespace tra
