// zero1_gemm_plan.h - how the products of a gated feed-forward block are cut up,
// in plain C++ (library-internal; the tests compile it for the host alone).
#pragma once

#include <stdint.h>

namespace z1mm {

constexpr int kTileM = 256;   // rows of a pair of CTAs' tile, 128 each
constexpr int kDeep = 64;     // of the contraction, per stage
constexpr int kRunF32 = 8, kRunBf16 = 2048;  // stages that the accumulator sums at one time, for fp32 and bf16 results

// M x N results in tiles of kTileM x tn, over `kblocks` stages.  Tiles from
// `whole` on are split into `splits` parts of per_split stages, whose fp32 sums
// go through the workspace.
struct Plan {
    int tn, tiles_m, tiles_n, kblocks, clusters, whole, splits, per_split;
    int64_t bytes;  // of the parts
};

// Time of a stage of a 128-column tile against that of a 256-column one: its MMAs
// take half, but they wait for A's loads (8192 x 4096 x 14336 in narrow and wide tiles:
// forward 1253 and 978 us, a weight gradient 643 and 521).  Narrow tiles pay where
// wide ones leave pairs idle: 64 rows forward 46 and 53 us, 12981 x 320 x 4096 62 and 65,
// a weight gradient of 1376 x 1000 over 776 rows 6.8 and 8.7.
constexpr double kNarrow = 0.62;
constexpr int kEnds = 8;     // an item's start and end, in stages
constexpr int kLaunch = 10;  // the joining launch, in stages
// (Split and not: 64 rows x 4096 x 14336, input gradient 48 and 90 us; 12981 x 320 x 4096 71
// and 80.  With the ends, the parts and the launch taken for nothing: 2048 x 1024 x 4096
// weight gradient 58 us for 14.)

// The estimated time, in stages of a 256-column tile (0.28 us), of the best way
// to cut tiles of tn columns; fills the plan.  The pairs of CTAs take the tiles in
// rounds; what a last, partial round would leave idle is used by splitting its
// tiles along the contraction, into at most 16 parts of at least 4 stages.
inline double plan_tiles(Plan *p, int64_t M, int64_t N, int tn, int kblocks, int clusters)
{
    const int64_t tm = (M + kTileM - 1) / kTileM, tnn = (N + tn - 1) / tn, tiles = tm * tnn;
    const double stage = tn == 256 ? 1.0 : kNarrow, part = 0.3 * tn / 256;
    p->tn = tn;
    p->tiles_m = (int)tm;
    p->tiles_n = (int)tnn;
    p->kblocks = kblocks;
    p->clusters = clusters;
    p->whole = (int)(tiles / clusters * clusters);
    p->splits = 1;
    p->per_split = kblocks;
    const int rest = (int)(tiles - p->whole);
    const double rounds = p->whole / clusters * (stage * kblocks + kEnds);
    if (rest == 0 || kblocks == 0) {
        p->whole = (int)tiles;
        return rounds;
    }
    double best = stage * kblocks + kEnds;
    for (int s = 2; s <= 16 && s * 4 <= kblocks; ++s) {
        const int per = (kblocks + s - 1) / s, parts = (kblocks + per - 1) / per;
        const int64_t turns = ((int64_t)rest * parts + clusters - 1) / clusters;
        const double cost = turns * (stage * per + kEnds) + part * rest * parts + kLaunch;
        if (cost < best) {
            best = cost;
            p->splits = parts;
            p->per_split = per;
        }
    }
    if (p->splits == 1) p->whole = (int)tiles;
    return rounds + best;
}

// The plan of M x N results over `kblocks` stages.
inline Plan plan_of(int64_t M, int64_t N, int kblocks, int clusters)
{
    Plan wide, narrow;
    const double a = plan_tiles(&wide, M, N, 256, kblocks, clusters), b = plan_tiles(&narrow, M, N, 128, kblocks, clusters);
    Plan p = b < a ? narrow : wide;
    const int64_t tiles = (int64_t)p.tiles_m * p.tiles_n;
    p.bytes = p.splits > 1 ? (tiles - p.whole) * p.splits * kTileM * p.tn * 4 : 0;
    return p;
}

}  // namespace z1mm
