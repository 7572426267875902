// linear_plan.h -- which tile and split a product on tiles takes (host side).
#pragma once

#include <algorithm>

#include "gemm_internal.h"
#include "linear_internal.h"

namespace tra {
namespace host {

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

// A product as the plan sees it.
struct PlanSizes {
    int64_t M, N, K;       // K of one segment
    int segs, batch;
    bool gated;
    int64_t in_bytes;      // of an operand's element
    double out_bytes;      // stored per column of z or u
    bool short_lines;      // 64 x 64 tiles read lines of 64 bytes
    bool direct16;         // direct loads of 16 bytes: the kernels that go one a CU are built
};

// The tile and split with the least predicted time, which goes to best_us.
//   Tiles: a CU runs its share of the workgroups (tiles x splits), `resident` at a
//   time; the K loop is bounded by the operands' bytes too; the results' stores
//   add to it.  A split stores binary32 sums and adds a launch that reads them.
//   Split are all tiles, where they are few, or those of the last, partial round
//   over the CUs, whose K loops would leave most CUs idle.
// Kept pre-activations have no part in it, though their stores add to the time: a
// forward pass that keeps them gives the same bits as one that does not (a
// checkpoint's recomputation).  Of 3000 random forward calls 82 had another plan with
// their stores counted.
inline TilePlan plan_classes(const TileClass *classes, int count, const PlanSizes &z,
                             double &best_us) {
    const int64_t b = z.in_bytes, slice = 128 / b;
    const int64_t M = z.M, N = z.N, K = z.K;
    const int segs = z.segs, batch = z.batch;
    const bool gated = z.gated;
    const int64_t k_tiles = std::max<int64_t>(1, segs * ceil_div(K, slice));
    const double columns = static_cast<double>(N) * (gated ? 2 : 1);      // of z and u
    const double in = static_cast<double>(batch) * segs * K * (static_cast<double>(M) + columns) * b;
    TilePlan best{};
    best_us = 0.0;
    for (int i = 0; i < count; ++i) {
        const TileClass &c = classes[i];
        if (c.bm == 0) break;
        const int64_t tiles = std::max<int64_t>(
            1, ceil_div(M, c.bm) * ceil_div(N, gated ? c.bn / 2 : c.bn));     // of a batch
        const double most = kBytesPerUs * (z.short_lines && c.bn == 64 ? 0.7 : 1.0);
        const double area = std::min<double>(M, c.bm) * std::min<double>(columns, c.bn);
        const double out = z.out_bytes;
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
                best.deep = z.direct16 && n <= kCUs;
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
    return best;
}

// Fills in what follows from the plan and checks the launch's size.  `slice`: elements of
// K in a K tile.
inline tra_status finish_tile_args(const TilePlan &t, int64_t slice, TileArgs &a, float *partial) {
    const int64_t tm = ceil_div(a.M, t.bm), tn = ceil_div(a.N, t.gated ? t.bn / 2 : t.bn);
    // kMaxGridLanes work-items (512 a workgroup), and tile indices in 32 bits
    const __int128 tiles = static_cast<__int128>(tm) * tn;
    const __int128 whole = t.splits > 1 ? static_cast<__int128>(t.whole) : tiles;
    if ((whole + (tiles - whole) * t.splits) * 512 > kMaxGridLanes) return TRA_ERR_UNSUPPORTED;
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

}  // namespace host
}  // namespace tra
