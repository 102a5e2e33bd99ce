// zero1_weight_grad_plan.h - how a weight gradient is cut up, in plain C++
// (library-internal; the tests compile it for the host alone).
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define Z1_HOST_DEVICE __host__ __device__
#else
#define Z1_HOST_DEVICE
#endif

namespace z1wg {

constexpr int kTileK = 256, kTileN = 256;     // of a pair of CTAs
constexpr int kDeep = 64;                     // rows of the contraction per stage
constexpr int kRunF32 = 32, kRunBf16 = 2048;  // stages that the accumulator sums at one time

// A call's tiles and which of them are split along the rows.  The workspace
// holds the split tiles' parts, the sums that whole tiles hold between runs (one
// tile per pair of CTAs), and the aligned copy of dy.
struct Plan {
    int tiles_k, tiles_n, kblocks, clusters, whole, splits, per_split;
    int64_t ld_copy, held_at, copy_at, bytes;
};

// The pairs of CTAs take the tiles in rounds; what a last, partial round would
// leave idle is used by splitting its tiles along the rows.  Of the splits
// into 1 to 16 parts the one with the least estimated time is taken, in
// stages of the contraction (0.28 us): the rounds, about 8 stages for each
// item's start and end, and for a split the writing and joining of its parts
// (0.5 MB each, about 0.3 stages) and one more launch (10 stages).
inline void split_rest(Plan *p)
{
    const int tiles = p->tiles_k * p->tiles_n;
    // (a bf16 tile done whole is stored once, so its rows fit one run)
    const bool all = p->kblocks > kRunBf16;
    p->whole = all ? 0 : tiles / p->clusters * p->clusters;
    const int rest = tiles - p->whole;
    p->splits = 1;
    p->per_split = p->kblocks;
    if (rest == 0 || p->kblocks == 0) return;
    double best = all ? 1e30 : p->kblocks + 8;
    for (int s = 2; s <= 16 && s * 4 <= p->kblocks; ++s) {
        const int per = (p->kblocks + s - 1) / s, parts = (p->kblocks + per - 1) / per;
        const int rounds = (rest * parts + p->clusters - 1) / p->clusters;
        const double cost = (double)rounds * (per + 8) + 0.3 * rest * parts + 10;
        if (cost < best) {
            best = cost;
            p->splits = parts;
            p->per_split = per;
        }
    }
    if (p->splits == 1) p->whole = tiles;
}

// Whether a whole tile may take more than one run of the accumulator.
inline bool holds_sums(const Plan &p) { return p.whole > 0 && p.kblocks > kRunF32; }

// The tiles whose parts one launch of the joining kernel adds: from `tile` on,
// their sums `part` values into the partial sums.  A grid holds at most
// `limit` of them.
struct JoinRun {
    int tile, tiles;
    int64_t part;
};

inline JoinRun join_run(int whole, int tiles, int splits, int tile, int limit)
{
    return JoinRun{tile, tiles - tile < limit ? tiles - tile : limit, (int64_t)(tile - whole) * splits * kTileN * kTileK};
}

// What the barrier of one use of a place for B still lacks once a pair of CTAs
// has given up.  A use is complete after one arrival that announces both CTAs'
// halves (the leading CTA's, with its own load), the converting warps' eight,
// and the bytes of both halves.  q: the use; mine, other: how many uses the
// leading CTA and the other one have loaded; late: converting warps that have
// not arrived.  With these arrivals made and these halves announced or written
// off, the use completes when the loads under way have landed, and not before.
struct Drain {
    uint32_t arrivals, announce, write_off;
};

Z1_HOST_DEVICE inline Drain drain_of(uint32_t q, uint32_t mine, uint32_t other, uint32_t late)
{
    return Drain{late + (q < mine ? 0u : 1u), q >= mine && q < other ? 1u : 0u, q < mine && q >= other ? 1u : 0u};
}

}  // namespace z1wg
