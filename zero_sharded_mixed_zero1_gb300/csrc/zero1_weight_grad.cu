// zero1_weight_grad.cu - the weight gradient of a projection, taken straight
// from the 8-bit checkpoint of its input, on the tensor cores.

#include <cuda.h>

#include "zero1_async.cuh"
#include "zero1_block.cuh"
#include "zero1_weight_grad_plan.h"

namespace {

using namespace z1wg;

// dw[n, k] = c[k] * sum_t dy[t, n] * x8[t, k].
//
// The contraction runs over the rows t of both operands, so both are "M/N
// major": TMA brings dy as it lies in memory into swizzled shared memory,
// which is the layout the MMA reads for its B operand.  x8 becomes the A
// operand: a code is 8 bits of a bf16 (sign, exponent, mantissa) 120 binades
// too low, so shifting it into place and multiplying by 2^(e + 120) gives the
// exact value; sixteen warps do that for 16-bit pairs of rows and write A into
// tensor memory, where it needs no second pass through shared memory.  A
// checkpoint block is 128 columns, which is one CTA's share of the tile, so
// each row has one scale per CTA.
//
// Two CTAs share a 256 (k) x 256 (n) tile: each holds 128 rows of A and of
// the accumulator in its tensor memory and loads half of B, 24 KB per 64 rows
// of the contraction where a CTA alone would load 40.  Products are exact in
// fp32; sums are fp32 in the accumulator.
//
// Measured on GB300: 14336 x 4096 outputs over 8192 rows 509 us in a burst (1890
// TFLOP/s, 0.96 of the measured cuBLAS rate for a plain bf16 product; 550 in a
// long loop), 4096 x 4096 148 to 150 us (1840).  A stage takes about 575 cycles where its MMAs need 512,
// the converting warps 260 on the integer pipe; what is left is the start and
// end of each tile and, over seconds, the power limit.  Steps on the way: one
// ring for codes and dy, releases at cluster scope and the timer read in every
// wait 1.5 ms on the larger size; two barriers per stage for the issuing warp
// instead of one 550 us.
//
// The tensor cores truncate where fp32 would round, an error that grows with
// the number of additions: 2e-7 of a gradient's norm over 777 rows, 1.5e-6 over
// 4096, 9e-6 over 16384.  For bf16 results that is nothing; for fp32 ones the
// accumulator is emptied every 2048 rows and the runs are added in fp32 (6e-7
// over 16384 rows; 4096 x 4096 over 8192 rows 191 to 200 us where bf16 takes 150:
// the MMAs stop for some 5000 cycles each time).
//
// Roles (28 warps): warp 0 loads dy and warp 3 the codes, warp 1 of the
// leading CTA issues the MMAs, warps 4-19 convert (four sets of four take
// stages in turn), warps 20-27 store the result (each 32 lanes and half of the
// columns of the accumulator).  bf16 results leave tensor memory at once, half
// into registers and half into shared memory, so that the next tile's MMAs do
// not wait for the stores to memory.

constexpr int kStages = 8;                 // of B in shared and A in tensor memory
constexpr int kCodeStages = 8;             // of codes and scales in shared memory
constexpr int kBBytes = kDeep * kTileN / 2 * 2, kXBytes = kDeep * kQBlock;  // of a CTA, per stage
constexpr int kSets = 4;                   // of four converting warps
// A set must meet every use of the places it takes: one that came to a place for
// the first time in its second use would take the parity of the phase before
// the first for the one it waits for.
static_assert(kStages % kSets == 0 && kCodeStages % kSets == 0, "a place belongs to one set");
constexpr int kWgThreads = 32 * (4 + 4 * kSets + 8);
constexpr uint32_t kTmemCols = 512, kTmemA = 256, kTmemAStage = kDeep / 2;

struct WgBars {
    uint64_t full[kStages], empty[kStages], cfull[kCodeStages], cempty[kCodeStages], dfull, dempty;
    uint32_t tmem;
    uint32_t failed;                  // a wait of either CTA ran out
    uint32_t loads, mmas, fills;      // uses of B's places loaded, stages and accumulator fills issued
    uint32_t converted[4 * kSets];    // the first use that a converting warp has not arrived at
};
constexpr int kStash = 32;  // packed pairs of bf16 results, or fp32 ones, that a storing thread keeps in shared memory
constexpr int kBoxRows = 16, kPlaces = kStash / kBoxRows;  // of the boxes that a part's sums leave in
constexpr int kStashBytes = 8 * 32 * kStash * 4;
constexpr int kWgSmem = 1024 + kStages * kBBytes + kCodeStages * (kXBytes + kDeep) + kStashBytes + (int)sizeof(WgBars);
static_assert(kWgSmem <= 227 * 1024, "shared memory of a block");
static_assert(kTmemA + kStages * kTmemAStage <= kTmemCols, "tensor memory");

struct Wg {
    int64_t T, N, K;
    int tiles_k, tiles_n, kblocks;      // kblocks: stages of the whole contraction
    int whole, splits, per_split;       // tiles done whole; the others in this many parts of per_split stages
    int run;                            // stages summed in the accumulator at one time
    const uint8_t *exps;
    int64_t ld_exps;
    const void *scale;
    int scale_f32;
    void *dw;
    int64_t ld_dw;
    int out_f32, accumulate, pairs;  // pairs: two outputs of a row per store
    int boxes;                       // fp32 results may go to dw in boxes
    float *part;                     // [split tile][part][kTileN][kTileK]
    float *held;                     // [CTA][storing warp][kTileN / 2][32 lanes]
};

// ------------------------------------------------------------- tcgen05 -----

__device__ __forceinline__ void tc_alloc(uint32_t *slot)
{
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(slot)), "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
}
__device__ __forceinline__ void tc_free(uint32_t base)
{
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(base), "r"(kTmemCols));
}
__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// D (both CTAs' tensor memory) (+)= A (tensor memory) * B (shared memory).
__device__ __forceinline__ void tc_mma(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t add)
{
    asm volatile(
        "{ .reg .pred p; setp.ne.u32 p, %4, 0; tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p; }" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(add)
        : "memory");
}

// Arrive on this barrier of both CTAs when the MMAs issued so far are done.
__device__ __forceinline__ void tc_commit(uint64_t *bar)
{
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_u32(bar)),
        "h"((uint16_t)3)
        : "memory");
}

// 16 lanes x 128 bits, four times: r[2j], r[2j + 1] are lanes l / 4 and 8 + l / 4,
// column 4 j + l % 4.
__device__ __forceinline__ void tc_store(uint32_t addr, const uint32_t r[8])
{
    asm volatile("tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(addr), "r"(r[0]),
                 "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}
__device__ __forceinline__ void tc_store_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 32 accumulator columns of this thread's lane.
__device__ __forceinline__ void tc_load32(uint32_t addr, uint32_t r[32])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void tc_load16(uint32_t addr, uint32_t r[16])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
        "[%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(addr));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

// Descriptor of a B tile: 128-byte swizzle, 64 columns x kDeep rows per TMA
// box (kDeep * 128 bytes from one 64-column group to the next), 8 rows per
// 1024-byte group.
__device__ __forceinline__ uint64_t b_desc(uint32_t addr)
{
    return (uint64_t)((addr & 0x3ffff) >> 4) | (uint64_t)((kDeep * 128) >> 4) << 16 | (uint64_t)(1024 >> 4) << 32 |
           (uint64_t)1 << 46 | (uint64_t)2 << 61;
}

// Instruction descriptor: fp32 accumulator, bf16 operands, B along N in
// memory, M = 256 (both CTAs), N = 256.
constexpr uint32_t kIdesc = (1u << 4) | (1u << 7) | (1u << 10) | (1u << 16) | ((uint32_t)(kTileN / 8) << 17) |
                            ((uint32_t)(kTileK / 16) << 24);

// ------------------------------------------------------------- clusters ----

__device__ __forceinline__ uint32_t cta_rank()
{
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Arrive on the leading CTA's copy of a barrier.
__device__ __forceinline__ void arrive_leader(uint64_t *bar)
{
    asm volatile(
        "{ .reg .b32 a; mapa.shared::cluster.u32 a, %0, 0; mbarrier.arrive.shared::cluster.b64 _, [a]; }" ::"r"(
            smem_u32(bar))
        : "memory");
}

// The same place in the shared memory of the pair's CTA `rank`.
__device__ __forceinline__ uint32_t at_rank(const void *p, uint32_t rank)
{
    uint32_t a;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
    return a;
}
__device__ __forceinline__ uint32_t read_rank(const uint32_t *p, uint32_t rank)
{
    uint32_t x;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(x) : "r"(at_rank(p, rank)) : "memory");
    return x;
}

// A bounded wait of a whole warp; one that runs out is noted in both CTAs.
__device__ __forceinline__ bool warp_wait(WgBars &b, uint64_t *bar, uint32_t parity)
{
    if (__all_sync(0xffffffffu, mbar_wait_long(bar, parity))) return true;
    if ((threadIdx.x & 31) < 2)
        asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(at_rank(&b.failed, threadIdx.x & 31)), "r"(1u) : "memory");
    __syncwarp();
    return false;
}

// The leading CTA's copy of a barrier, as a cluster address.
__device__ __forceinline__ uint32_t leader_addr(uint64_t *bar)
{
    uint32_t a;
    asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(a) : "r"(smem_u32(bar)));
    return a;
}

// A box into this CTA's shared memory, counted on the leading CTA's barrier.
__device__ __forceinline__ void tma_2d_pair(void *dst, const CUtensorMap *map, int x, int y, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], "
        "[%4];" ::"r"(smem_u32(dst)),
        "l"(map), "r"(x), "r"(y), "r"(bar)
        : "memory");
}

__device__ __forceinline__ void tma_2d(void *dst, const CUtensorMap *map, int x, int y, uint64_t *bar)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
            smem_u32(dst)),
        "l"(map), "r"(x), "r"(y), "r"(smem_u32(bar))
        : "memory");
}

// ----------------------------------------------------------- conversion ----

__device__ __forceinline__ void ldmatrix_t(uint32_t addr, uint32_t r[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// bf16 factors of one row's scale E = e + 127: 2^(e + 120) up to e = 7, the
// rest of the binades in a second factor; rows past the end are 0.
__device__ __forceinline__ uint32_t factor1(int E, bool in)
{
    return !in ? 0u : E == kNanE ? 0x7fc0u : (uint32_t)(min(E, 134) + 120) << 7;
}
__device__ __forceinline__ uint32_t factor2(int E) { return (uint32_t)(127 + (E == kNanE ? 0 : max(E - 134, 0))) << 7; }

// ----------------------------------------------------------------- kernel --

struct Item {
    int n0, k0, kb0, kb1, part;  // part: its place among the partial sums, -1 for a whole tile
};

// Tiles run in bands of eight along k, so that the pairs of CTAs at work at
// one time share few columns of both operands (they meet in L2).
__device__ __forceinline__ void tile_of(const Wg &a, int t, int &n0, int &k0)
{
    constexpr int kBand = 8;
    const int per = kBand * a.tiles_n, band = t / per, in = t % per;
    const int width = min(kBand, a.tiles_k - band * kBand);
    k0 = (band * kBand + in % width) * kTileK;
    n0 = in / width * kTileN;
}

// The whole tiles come first, then the parts of the others: all first parts,
// all second ones and so on, so that neighbours in time share operands.
__device__ __forceinline__ Item item_of(const Wg &a, int i)
{
    Item o;
    if (i < a.whole) {
        tile_of(a, i, o.n0, o.k0);
        o.kb0 = 0;
        o.kb1 = a.kblocks;
        o.part = -1;
    } else {
        const int rest = a.tiles_k * a.tiles_n - a.whole, t = (i - a.whole) % rest, p = (i - a.whole) / rest;
        tile_of(a, a.whole + t, o.n0, o.k0);
        o.kb0 = p * a.per_split;
        o.kb1 = min(o.kb0 + a.per_split, a.kblocks);
        o.part = t * a.splits + p;
    }
    return o;
}

__device__ __forceinline__ int items_of(const Wg &a)
{
    return a.whole + (a.tiles_k * a.tiles_n - a.whole) * a.splits;
}

// ------------------------------------------------------------- epilogue ----
//
// A warp stores 32 lanes (columns k) x 128 accumulator columns (rows n).  Lane
// l of a group of 16 holds column 2 l (l < 8) or 2 (l - 8) + 1; lanes l and
// l + 8 trade so that each has both columns of every other row, and a store
// instruction writes 64 consecutive bytes (bf16) of two rows.

__device__ __forceinline__ int own_column(int lane) { return (lane & 16) + 2 * (lane & 7) + ((lane >> 3) & 1); }

// The accumulator has been read: the next tile may overwrite it.
__device__ __forceinline__ void release_acc(uint64_t *dempty)
{
    tc_before();
    __syncwarp();
    if ((threadIdx.x & 31) == 0) arrive_leader(dempty);
}

__device__ __forceinline__ void store_bf16(const Wg &a, uint32_t acc, int64_t k0, int64_t n0, uint32_t *stash, uint64_t *dempty)
{
    const int lane = threadIdx.x & 31;
    float scale = 1.f;
    if (a.scale && k0 + own_column(lane) < a.K) scale = ld_param(a.scale, a.scale_f32, k0 + own_column(lane));
    const bool up = lane & 8;
    const int64_t k = k0 + (lane & 16) + 2 * (lane & 7);
    if (a.accumulate) {  // rounded once, after the addition
        for (int c = 0; c < kTileN / 2; c += 32) {
            uint32_t v[32];
            tc_load32(acc + c, v);
            if (c + 32 == kTileN / 2) release_acc(dempty);
#pragma unroll
            for (int j = 0; j < 32; ++j) {
                const int64_t n = n0 + c + j, kk = k0 + own_column(lane);
                if (n >= a.N || kk >= a.K) continue;
                uint16_t *o = static_cast<uint16_t *>(a.dw) + n * a.ld_dw + kk;
                *o = to_bf16(fmaf(__uint_as_float(v[j]), scale, bf_one(*o)));
            }
        }
        return;
    }
    uint32_t p[kTileN / 4 - kStash];
#pragma unroll
    for (int c = 0; c < kTileN / 2; c += 16) {
        uint32_t v[16];
        tc_load16(acc + c, v);
#pragma unroll
        for (int j = 0; j < 16; j += 2) {
            const uint32_t x = pack_bf16x2(__uint_as_float(v[j]) * scale, __uint_as_float(v[j + 1]) * scale);
            if ((c + j) / 2 < kStash) stash[(c + j) / 2 * 32] = x;
            else p[(c + j) / 2 - kStash] = x;
        }
    }
    release_acc(dempty);
    uint16_t *o = static_cast<uint16_t *>(a.dw) + (n0 + (up ? 1 : 0)) * a.ld_dw + k;
    const bool two = k + 1 < a.K;
    if (a.pairs && n0 + kTileN / 2 <= a.N && k0 + 32 <= a.K) {  // no bounds to check
#pragma unroll
        for (int j = 0; j < kTileN / 2; j += 2, o += 2 * a.ld_dw) {
            const uint32_t mine = j / 2 < kStash ? stash[j / 2 * 32] : p[j / 2 - kStash];
            const uint32_t other = __shfl_xor_sync(0xffffffffu, mine, 8);
            *reinterpret_cast<uint32_t *>(o) = up ? __byte_perm(mine, other, 0x3276) : __byte_perm(mine, other, 0x5410);
        }
        return;
    }
#pragma unroll
    for (int j = 0; j < kTileN / 2; j += 2, o += 2 * a.ld_dw) {
        const uint32_t mine = j / 2 < kStash ? stash[j / 2 * 32] : p[j / 2 - kStash], other = __shfl_xor_sync(0xffffffffu, mine, 8);
        const uint32_t x = up ? __byte_perm(mine, other, 0x3276) : __byte_perm(mine, other, 0x5410);
        if (n0 + j + (up ? 1 : 0) >= a.N || k >= a.K) continue;
        if (a.pairs && two) {
            *reinterpret_cast<uint32_t *>(o) = x;
        } else {
            o[0] = (uint16_t)x;
            if (two) o[1] = (uint16_t)(x >> 16);
        }
    }
}

// Adds to what this thread stored before.  Only this thread ever adds there, one
// addition after the other, so the order of the sum is fixed; a reduction leaves
// no value to wait for.  It takes subnormal values for 0 (measured; copies to
// the same place in boxes, which do not, took 211 us for 188 at 4096 x 4096 over
// 8192 rows), so it serves this call's own sums only, never the caller's.
__device__ __forceinline__ void add_to(float *p, float x) { asm volatile("red.global.add.f32 [%0], %1;" ::"l"(p), "f"(x) : "memory"); }
__device__ __forceinline__ void add_to(float *p, float2 x)
{
    asm volatile("red.global.add.v2.f32 [%0], {%1, %2};" ::"l"(p), "f"(x.x), "f"(x.y) : "memory");
}

// fp32 results, 32 lanes x 128 rows, two columns of a row per lane as above
// (one column per lane, in the lanes' order, took twice the instructions and
// more time).  rows: how many of the 128 are stored; cols: of this lane's two.
template <bool ADD>
__device__ __forceinline__ void store_f32(float *o, int64_t ld, int rows, int cols, bool pairs, float scale, uint32_t acc,
                                          uint64_t *dempty)
{
    const bool up = threadIdx.x & 8;
    const bool easy = pairs && cols == 2 && rows == kTileN / 2;
    o += up ? ld : 0;
#pragma unroll 1
    for (int c = 0; c < kTileN / 2; c += 32) {
        uint32_t v[32];
        tc_load32(acc + c, v);
        if (c + 32 == kTileN / 2) release_acc(dempty);
#pragma unroll
        for (int j = 0; j < 32; j += 2, o += 2 * ld) {
            const float v0 = __uint_as_float(v[j]) * scale, v1 = __uint_as_float(v[j + 1]) * scale;
            const float got = __shfl_xor_sync(0xffffffffu, up ? v0 : v1, 8);
            const float2 x = up ? make_float2(got, v1) : make_float2(v0, got);
            if (easy) {
                if (ADD) add_to(o, x);
                else *reinterpret_cast<float2 *>(o) = x;
            } else if (c + j + up < rows) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    if (e >= cols) continue;
                    if (ADD) add_to(o + e, e ? x.y : x.x);
                    else o[e] = e ? x.y : x.x;
                }
            }
        }
    }
}

// What is added to the caller's gradient is the whole sum, rounded once: the
// sums of the runs before an item's last one are held in the workspace, 128
// values per thread of its own, 32 lanes side by side.
constexpr int kHeld = 16;  // values that are on their way at one time

__device__ __forceinline__ void hold_run(float *held, bool begin, uint32_t acc, uint64_t *dempty)
{
#pragma unroll 1
    for (int c = 0; c < kTileN / 2; c += 32) {
        uint32_t v[32];
        tc_load32(acc + c, v);
        if (c + 32 == kTileN / 2) release_acc(dempty);
#pragma unroll
        for (int j = 0; j < 32; ++j, held += 32) {
            if (begin) *held = __uint_as_float(v[j]);
            else add_to(held, __uint_as_float(v[j]));
        }
    }
}

struct Held {
    const float *p;  // NULL: nothing is held
    // Adds rows c .. c + 15.  (Loading them earlier took registers that the rest
    // of the kernel then spilled.)
    __device__ __forceinline__ void join(int c, uint32_t v[kHeld]) const
    {
        float h[kHeld];
#pragma unroll
        for (int j = 0; j < kHeld; ++j) h[j] = __ldcg(p + (c + j) * 32);
#pragma unroll
        for (int j = 0; j < kHeld; ++j) v[j] = __float_as_uint(h[j] + __uint_as_float(v[j]));
    }
};

// fp32 results added to the caller's where boxes cannot take them (dw off 16-byte
// boundaries), an element at a time.
__device__ __forceinline__ void add_f32_any(float *o, int64_t ld, int rows, bool in, float scale, const Held &held, uint32_t acc,
                                            uint64_t *dempty)
{
#pragma unroll 1
    for (int c = 0; c < kTileN / 2; c += kHeld) {
        uint32_t v[kHeld];
        tc_load16(acc + c, v);
        if (c + kHeld == kTileN / 2) release_acc(dempty);
        if (held.p) held.join(c, v);
        float old[kHeld];
#pragma unroll
        for (int j = 0; j < kHeld; ++j) old[j] = in && c + j < rows ? o[j * ld] : 0.f;
#pragma unroll
        for (int j = 0; j < kHeld; ++j)
            if (in && c + j < rows) o[j * ld] = fmaf(__uint_as_float(v[j]), scale, old[j]);
        o += kHeld * ld;
    }
}

// A box from shared memory, added to what is there or written, and a group of
// its own.  (These reductions keep subnormal values, measured.)
__device__ __forceinline__ void box_out(const CUtensorMap *map, int x, int y, bool add, const uint32_t *place)
{
    if (add)
        asm volatile("cp.reduce.async.bulk.tensor.2d.global.shared::cta.add.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(map),
                     "r"(x), "r"(y), "r"(smem_u32(place))
                     : "memory");
    else
        asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(map), "r"(x),
                     "r"(y), "r"(smem_u32(place))
                     : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}

// 32 lanes x 128 rows as boxes of 32 columns x kBoxRows rows, copied or added
// from the warp's two places in shared memory: no trade between lanes, a
// quarter of the instructions, and nothing to wait for.  rows: how many of the
// 128 are wanted (a box may hang over dw's edge and is clipped there).
__device__ __forceinline__ void store_boxes(const CUtensorMap *map, int x, int y, int rows, bool add, float scale,
                                            const Held &held, uint32_t acc, uint32_t *places, uint64_t *dempty)
{
    static_assert(kBoxRows == kHeld, "a box takes what is on its way");
    const int lane = threadIdx.x & 31;
    int at = 0;
#pragma unroll 1
    for (int c = 0; c < kTileN / 2; c += kBoxRows) {
        uint32_t v[kBoxRows];
        tc_load16(acc + c, v);
        if (c + kBoxRows == kTileN / 2) release_acc(dempty);
        if (held.p) held.join(c, v);
        if (elect_one()) asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(kPlaces - 1) : "memory");  // the place is free
        __syncwarp();
        uint32_t *place = places + at * 32 * kBoxRows;
#pragma unroll
        for (int j = 0; j < kBoxRows; ++j) place[32 * j + own_column(lane)] = __float_as_uint(__uint_as_float(v[j]) * scale);
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (c < rows && elect_one()) box_out(map, x, y + c, add, place);
        __syncwarp();
        at = at + 1 == kPlaces ? 0 : at + 1;
    }
}

// All boxes that this warp has sent are written.
__device__ __forceinline__ void boxes_written()
{
    if (elect_one()) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    __syncwarp();
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kWgThreads, 1)
k_weight_grad(const __grid_constant__ CUtensorMap map_dy, const __grid_constant__ CUtensorMap map_x,
              const __grid_constant__ CUtensorMap map_part, const __grid_constant__ CUtensorMap map_dw, const Wg a)
{
    extern __shared__ unsigned char raw[];
    unsigned char *smem = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
    unsigned char *s_codes = smem + kStages * kBBytes;
    uint8_t *s_exps = s_codes + kCodeStages * kXBytes;
    uint32_t *s_stash = reinterpret_cast<uint32_t *>(s_exps + kCodeStages * kDeep);
    WgBars &bar = *reinterpret_cast<WgBars *>(s_stash + kStashBytes / 4);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cta_rank();
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&bar.full[s], 9);    // the loads of B, four converting warps of each CTA
            mbar_init(&bar.empty[s], 1);
        }
        for (int s = 0; s < kCodeStages; ++s) {
            mbar_init(&bar.cfull[s], 1);
            mbar_init(&bar.cempty[s], 4);  // four converting warps
        }
        mbar_init(&bar.dfull, 1);
        mbar_init(&bar.dempty, 16);  // eight storing warps of each CTA
        bar.failed = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 2) tc_alloc(&bar.tmem);
    tc_before();
    __syncthreads();
    cluster_sync();
    tc_after();
    wait_prior_grid();  // up to here this kernel may run beside the one before it
    const uint32_t tmem = bar.tmem;
    const int items = items_of(a);
    const int first = blockIdx.x / 2, step = gridDim.x / 2;

    // The loading and issuing warps run whole, so that addresses and descriptors
    // stay in uniform registers, and elect one lane for each instruction.
    if (warp == 0) {
        uint32_t it = 0;
        bool ok = true;
        for (int i = first; i < items && ok; i += step) {
            const Item w = item_of(a, i);
            const int n = w.n0 + (int)rank * (kTileN / 2);
            for (int kb = w.kb0; kb < w.kb1; ++kb, ++it) {
                const int s = it % kStages;
                if (it >= kStages && !(ok = warp_wait(bar, &bar.empty[s], (it / kStages - 1) & 1))) break;
                unsigned char *b = smem + s * kBBytes;
                if (elect_one()) {
                    // both CTAs' halves count on the leading CTA's barrier
                    const uint32_t full = leader_addr(&bar.full[s]);
                    if (rank == 0) mbar_expect_tx(&bar.full[s], 2 * kBBytes);
                    tma_2d_pair(b, &map_dy, n, kb * kDeep, full);
                    tma_2d_pair(b + kBBytes / 2, &map_dy, n + 64, kb * kDeep, full);
                }
                __syncwarp();
            }
        }
        // the last copies must land before the pair may exit (both CTAs have as many)
        if (rank == 0)
            for (uint32_t q = it > kStages ? it - kStages : 0; q < it && ok; ++q)
                ok = warp_wait(bar, &bar.full[q % kStages], (q / kStages) & 1);
        if (lane == 0) bar.loads = it;
    } else if (warp == 3) {
        uint32_t it = 0;
        bool ok = true;
        for (int i = first; i < items && ok; i += step) {
            const Item w = item_of(a, i);
            const int64_t block = min((int64_t)(w.k0 / kQBlock) + rank, (a.K - 1) / kQBlock);
            const uint8_t *exps = a.exps + block * a.ld_exps;
            const int k = w.k0 + (int)rank * kQBlock;
            for (int kb = w.kb0; kb < w.kb1; ++kb, ++it) {
                const int s = it % kCodeStages;
                if (it >= kCodeStages && !(ok = warp_wait(bar, &bar.cempty[s], (it / kCodeStages - 1) & 1))) break;
                if (elect_one()) {
                    mbar_expect_tx(&bar.cfull[s], kXBytes + kDeep);
                    tma_2d(s_codes + s * kXBytes, &map_x, k, kb * kDeep, &bar.cfull[s]);
                    bulk_load(s_exps + s * kDeep, exps + (int64_t)kb * kDeep, kDeep, &bar.cfull[s]);
                }
                __syncwarp();
            }
        }
        // (only the copies themselves are waited for here)
        for (uint32_t q = it > kCodeStages ? it - kCodeStages : 0; q < it; ++q)
            warp_wait(bar, &bar.cfull[q % kCodeStages], (q / kCodeStages) & 1);
    } else if (warp == 1) {
        if (rank == 0) {
            uint32_t it = 0, tile = 0, fills = 0;  // stages, accumulator fills begun and done so far
            bool ok = true;
            const uint64_t b0 = b_desc(smem_u32(smem));
            for (int i = first; i < items && ok; i += step) {
                const Item w = item_of(a, i);
                for (int kb = w.kb0; kb < w.kb1 && ok; ++tile) {
                    if (tile > 0 && !(ok = warp_wait(bar, &bar.dempty, (tile - 1) & 1))) break;
                    const int start = kb, end = min(kb + a.run, w.kb1);
                    for (; kb < end; ++kb, ++it) {
                        const int s = it % kStages;
                        // what the instructions take is ready before the branch, in uniform registers
                        const uint64_t b = b0 + (uint64_t)(s * (kBBytes >> 4));
                        const uint32_t ta = tmem + kTmemA + s * kTmemAStage, more = kb > start;
                        if (!(ok = warp_wait(bar, &bar.full[s], (it / kStages) & 1))) break;
                        tc_after();
                        if (elect_one()) {
#pragma unroll
                            for (int j = 0; j < kDeep / 16; ++j)
                                tc_mma(tmem, ta + 8 * j, b + j * (2048 >> 4), kIdesc, j ? 1u : more);
                            tc_commit(&bar.empty[s]);
                            if (kb + 1 == end) tc_commit(&bar.dfull);
                        }
                        __syncwarp();
                    }
                    fills += ok;
                }
            }
            // the MMAs must have finished with both CTAs' memory before the exit
            if (it > 0) warp_wait(bar, &bar.empty[(it - 1) % kStages], ((it - 1) / kStages) & 1);
            if (lane == 0) {
                bar.mmas = it;
                bar.fills = fills;
            }
        }
    } else if (warp >= 4 && warp < 4 + 4 * kSets) {
        const uint32_t set = (warp - 4) / 4, q = warp % 4;
        uint32_t it0 = 0, stopped = 0;  // stages before this item; where a wait ran out
        bool ok = true;
        // this thread's share of a stage: ldmatrix rows `lane` and 32 + lane, columns 32 q .. 32 q + 31
        const uint32_t x_row = smem_u32(s_codes) + lane * 128, x_swz = lane & 7;
        const uint32_t a_addr = tmem + ((32 * q) << 16) + kTmemA;
        for (int i = first; i < items && ok; i += step) {
            const Item w = item_of(a, i);
            const uint32_t n = w.kb1 - w.kb0;
            for (uint32_t j = (set - it0) % kSets; j < n; j += kSets) {
                const uint32_t it = it0 + j, s = it % kStages, c = it % kCodeStages;
                stopped = it;
                if (!(ok = warp_wait(bar, &bar.cfull[c], (it / kCodeStages) & 1))) break;
                // Scales of rows 2 lane and 2 lane + 1 as a bf16 pair, passed to
                // the lanes that convert those rows.  Almost always every scale
                // of the stage is at most 2^7 and every row is there: then one
                // factor 2^(e + 120) does.
                const uint32_t e = reinterpret_cast<const uint16_t *>(s_exps + c * kDeep)[lane];
                const int left = (int)(a.T - (int64_t)(w.kb0 + j) * kDeep) - 2 * lane;  // rows from this lane's on
                uint32_t mine = (__byte_perm(e, 0, 0x4140) + 0x00780078u) << 7, more = 0x3f803f80u;
                const bool plain = __all_sync(0xffffffffu, (e & 255) <= 134 && (e >> 8) <= 134 && left >= 2);
                if (!plain) {
                    mine = factor1(e & 255, left >= 1) | factor1(e >> 8, left >= 2) << 16;
                    more = factor2(e & 255) | factor2(e >> 8) << 16;
                }
                if (it >= kStages && !(ok = warp_wait(bar, &bar.empty[s], (it / kStages - 1) & 1))) break;
                tc_after();
                const uint32_t x = x_row + c * kXBytes, at = a_addr + s * kTmemAStage;
#pragma unroll
                for (int h = 0; h < 2; ++h) {  // 32 rows
                    uint32_t f[4];
#pragma unroll
                    for (int p = 0; p < 4; ++p) f[p] = __shfl_sync(0xffffffffu, mine, 16 * h + 4 * p + (lane & 3));
#pragma unroll
                    for (int g = 0; g < 2; ++g) {  // 16 columns
                        uint32_t m[4], r[8];
                        ldmatrix_t(x + h * 4096 + (((2 * q + g) ^ x_swz) << 4), m);
#pragma unroll
                        for (int p = 0; p < 4; ++p) {
                            // even and odd columns of the pair, sign and magnitude put in place
                            const uint32_t lo = (m[p] & 0x007f007fu) * 16u, hi = (m[p] >> 4) & 0x07f007f0u;
                            r[2 * p] = mul_bf16x2((m[p] & 0x00800080u) * 256u + lo, f[p]);
                            r[2 * p + 1] = mul_bf16x2(hi | (m[p] & 0x80008000u), f[p]);
                        }
                        if (!plain) {
#pragma unroll
                            for (int p = 0; p < 4; ++p) {
                                const uint32_t f2 = __shfl_sync(0xffffffffu, more, 16 * h + 4 * p + (lane & 3));
                                r[2 * p] = mul_bf16x2(r[2 * p], f2);
                                r[2 * p + 1] = mul_bf16x2(r[2 * p + 1], f2);
                            }
                        }
                        tc_store(at + ((16 * g) << 16) + 16 * h, r);
                    }
                }
                tc_store_wait();
                tc_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&bar.cempty[c]);
                    arrive_leader(&bar.full[s]);
                }
            }
            it0 += n;
        }
        if (lane == 0) bar.converted[warp - 4] = ok ? it0 : stopped;
    } else if (warp >= 4 + 4 * kSets) {
        const int q = warp % 4, half = (warp - 4 - 4 * kSets) / 4;
        uint32_t *const places = s_stash + (4 * half + q) * 32 * kStash, *const stash = places + lane;
        float *const sums = a.held + ((int64_t)blockIdx.x * 8 + 4 * half + q) * (kTileN / 2) * 32 + lane;
        uint32_t tile = 0;
        bool ok = true;
        for (int i = first; i < items && ok; i += step) {
            const Item w = item_of(a, i);
            const uint32_t acc = tmem + ((uint32_t)(32 * q) << 16) + half * (kTileN / 2);
            const int64_t k0 = w.k0 + (int64_t)rank * kQBlock + 32 * q, n0 = w.n0 + half * (kTileN / 2);
            for (int kb = w.kb0; kb < w.kb1; kb += a.run, ++tile) {
                if (!(ok = warp_wait(bar, &bar.dfull, tile & 1))) break;
                tc_after();
                const bool begin = kb == w.kb0, end = kb + a.run >= w.kb1;
                if (w.part < 0 && !a.out_f32) {  // (takes one run)
                    store_bf16(a, acc, k0, n0, stash, &bar.dempty);
                    continue;
                }
                const int64_t k = k0 + own_column(lane), two = k0 + (lane & 16) + 2 * (lane & 7);
                const int rows = (int)max((int64_t)0, min((int64_t)(kTileN / 2), a.N - n0));
                const float scale = w.part < 0 && a.scale && k < a.K ? ld_param(a.scale, a.scale_f32, k) : 1.f;
                float *const o = static_cast<float *>(a.dw) + n0 * a.ld_dw;
                if (w.part < 0 && !a.accumulate && !(a.boxes && begin && end)) {
                    const int cols = (int)max((int64_t)0, min((int64_t)2, a.K - two));
                    if (begin) store_f32<false>(o + two, a.ld_dw, rows, cols, a.pairs, scale, acc, &bar.dempty);
                    else store_f32<true>(o + two, a.ld_dw, rows, cols, a.pairs, scale, acc, &bar.dempty);
                    continue;
                }
                if (w.part < 0 && !end) {
                    hold_run(sums, begin, acc, &bar.dempty);
                    continue;
                }
                const Held held{w.part < 0 && !begin ? sums : nullptr};
                if (w.part < 0 && !a.boxes) {
                    add_f32_any(o + k, a.ld_dw, rows, k < a.K, scale, held, acc, &bar.dempty);
                    continue;
                }
                const bool part = w.part >= 0;
                if (part && !begin) boxes_written();  // the run before
                store_boxes(part ? &map_part : &map_dw, (int)(part ? k0 - w.k0 : k0),
                            part ? w.part * kTileN + half * (kTileN / 2) : (int)n0, part ? kTileN / 2 : k0 < a.K ? rows : 0,
                            part ? !begin : a.accumulate, scale, held, acc, places, &bar.dempty);
            }
        }
        boxes_written();  // before the grid counts as done
    }
    __syncwarp();
    __syncthreads();
    cluster_sync();
    // From here on neither CTA starts anything.  If no wait ran out, all that was
    // started has finished (the waits above).  If one did, what is under way to
    // either CTA's shared memory, or reads it, is waited for before the pair's
    // memory is given back: the loads of B, by making up what their barriers
    // lack, and the MMAs with the arrivals that follow them.
    if (bar.failed) {
        if (warp == 0 && rank == 0) {
            const uint32_t mine = bar.loads, other = read_rank(&bar.loads, 1), n = max(mine, other);
            for (uint32_t q = n > kStages ? n - kStages : 0; q < n; ++q) {
                const uint32_t *c = &bar.converted[q % kSets * 4 + lane % 4];  // lanes 0-3 here, 4-7 there
                const uint32_t late = __popc(__ballot_sync(0xffffffffu, lane < 8 && read_rank(c, lane / 4 & 1) <= q));
                const Drain d = drain_of(q, mine, other, late);
                if (lane == 0) mbar_make_up(&bar.full[q % kStages], d.arrivals, d.announce * kBBytes, d.write_off * kBBytes);
                __syncwarp();
                warp_wait(bar, &bar.full[q % kStages], (q / kStages) & 1);
            }
        } else if (warp == 1) {
            const uint32_t m = read_rank(&bar.mmas, 0), f = read_rank(&bar.fills, 0);
            if (m > 0) warp_wait(bar, &bar.empty[(m - 1) % kStages], ((m - 1) / kStages) & 1);
            if (f > 0) warp_wait(bar, &bar.dfull, (f - 1) & 1);
        }
        __syncthreads();
        cluster_sync();
    }
    if (warp == 2) {
        tc_after();
        tc_free(tmem);
    }
}

// Adds a split tile's parts in order and finishes the gradient there; with no
// parts at all (no rows) the gradient of every tile is 0.  A block takes 8 rows
// of a tile, a thread 8 columns.  a.whole: the launch's first tile, a.part: its
// first part.
__global__ void __launch_bounds__(256) k_weight_grad_join(const Wg a)
{
    wait_prior_grid();
    int n0, k0;
    tile_of(a, a.whole + blockIdx.y, n0, k0);
    const int n = blockIdx.x * 8 + threadIdx.x / 32, k = threadIdx.x % 32 * 8;
    if (n0 + n >= a.N || k0 + k >= a.K) return;
    float x[8] = {};
    const float *p = a.part + (int64_t)blockIdx.y * a.splits * kTileN * kTileK + n * kTileK + k;
#pragma unroll 4
    for (int s = 0; s < a.splits; ++s, p += kTileN * kTileK) {
        Raw8<float> q;
        float v[8];
        q.load(p);
        q.get(v);
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] += v[j];
    }
    const int64_t kk = (int64_t)k0 + k;
    const int width = kk + 8 <= a.K ? 8 : (int)(a.K - kk);
    float scale[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) scale[j] = a.scale && j < width ? ld_param(a.scale, a.scale_f32, kk + j) : 1.f;
    const int64_t at = (int64_t)(n0 + n) * a.ld_dw + kk;
    if (a.out_f32) {
        float *o = static_cast<float *>(a.dw) + at;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < width) o[j] = a.accumulate ? fmaf(x[j], scale[j], o[j]) : x[j] * scale[j];
    } else {
        uint16_t *o = static_cast<uint16_t *>(a.dw) + at;
        if (!a.accumulate && width == 8 && ((uintptr_t)o & 15) == 0) {
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] *= scale[j];
            store8(o, x);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (j < width) o[j] = to_bf16(a.accumulate ? fmaf(x[j], scale[j], bf_one(o[j])) : x[j] * scale[j]);
        }
    }
}

// Copies dy to rows that start on 16-byte boundaries, eight elements per thread.
__global__ void __launch_bounds__(256)
k_align_rows(const uint16_t *__restrict__ src, int64_t ld, int64_t T, int64_t N, uint16_t *__restrict__ dst, int64_t ld_dst)
{
    for (int64_t c = ((int64_t)blockIdx.y * 32 + threadIdx.x % 32) * 8; c < N; c += (int64_t)gridDim.y * 256)
        for (int64_t t = (int64_t)blockIdx.x * 8 + threadIdx.x / 32; t < T; t += (int64_t)gridDim.x * 8)
            *reinterpret_cast<uint4 *>(dst + t * ld_dst + c) = load8_any(src + t * ld, c, N, t * ld == 0);
}

// --------------------------------------------------------------- launch ----

using EncodeTiled = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                 const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_tiled()
{
    static const EncodeTiled fn = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess) {
            cudaGetLastError();
            p = nullptr;
        }
        return reinterpret_cast<EncodeTiled>(p);
    }();
    return fn;
}

// A [rows, cols] matrix in boxes of box_x columns and box_y rows.
int make_map(CUtensorMap *m, CUtensorMapDataType type, int es, const void *p, int64_t rows, int64_t cols, int64_t ld,
             int box_x, const char *what, int box_y = kDeep, CUtensorMapSwizzle swizzle = CU_TENSOR_MAP_SWIZZLE_128B)
{
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)(ld * es)};
    const cuuint32_t box[2] = {(cuuint32_t)box_x, (cuuint32_t)box_y}, one[2] = {1, 1};
    const EncodeTiled fn = encode_tiled();
    if (!fn) return z1_fail(ZERO1_ECUDA, "weight gradient: the driver has no tensor maps");
    const CUresult r = fn(m, type, 2, const_cast<void *>(p), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                          swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return z1_fail(ZERO1_ECUDA, "weight gradient: tensor map of %s: error %d", what, (int)r);
    return ZERO1_OK;
}

bool rows_aligned(const void *dy, int64_t ld, int64_t rows)
{
    return (((uintptr_t)dy) & 15) == 0 && (rows <= 1 || (ld % 8 == 0 && ld > 0));
}

int plan_of(int64_t T, int64_t N, int64_t K, const void *dy, int64_t ld, Plan *p)
{
    const char *call = "weight gradient";
    const int64_t tk = (K + kTileK - 1) / kTileK, tn = (N + kTileN - 1) / kTileN, kb = (T + kDeep - 1) / kDeep;
    if (T > INT32_MAX - kDeep || N > INT32_MAX - kTileN || K > INT32_MAX - kTileK || tk * tn > (1 << 24))
        return z1_fail(ZERO1_ERANGE, "%s: %lld rows, %lld x %lld outputs: size not supported", call, (long long)T,
                       (long long)N, (long long)K);
    const int sms = sm_count();
    if (sms == 0) return z1_fail(ZERO1_ECUDA, "%s: no CUDA device", call);
    p->clusters = sms / 2;
    p->tiles_k = (int)tk;
    p->tiles_n = (int)tn;
    p->kblocks = (int)kb;
    split_rest(p);
    p->held_at = p->splits > 1 ? (tk * tn - p->whole) * p->splits * kTileN * kTileK * 4 : 0;
    p->copy_at = p->held_at + (holds_sums(*p) ? (int64_t)p->clusters * kTileN * kTileK * 4 : 0);
    p->ld_copy = round_up(N, 8);
    p->bytes = p->copy_at + (rows_aligned(dy, ld, T) ? 0 : round_up(T * p->ld_copy * 2, 128));
    return ZERO1_OK;
}

}  // namespace

int z1_weight_grad_status(uint32_t *status, int32_t clear) { return (int)async_status(status, clear); }

extern "C" int zero1_weight_grad_workspace(int64_t rows, int64_t n, int64_t k, const void *dy, int64_t ld_dy,
                                           int64_t *bytes)
{
    if (!bytes) return z1_fail(ZERO1_EINVAL, "weight gradient workspace: bytes is NULL");
    if (rows < 0 || n < 1 || k < 1)
        return z1_fail(ZERO1_EINVAL, "weight gradient workspace: %lld rows, %lld x %lld outputs", (long long)rows,
                       (long long)n, (long long)k);
    Plan p;
    const int rc = plan_of(rows, n, k, dy, ld_dy, &p);
    if (rc == ZERO1_OK) *bytes = p.bytes;
    return rc;
}

extern "C" int zero1_weight_grad(const void *dy, int64_t ld_dy, int64_t n, const zero1_checkpoint8_t *x8,
                                 const void *col_scale, int32_t scale_dtype, void *dw, int64_t ld_dw, int32_t out_dtype,
                                 int32_t accumulate, void *workspace, int64_t workspace_bytes, zero1_stream_t stream)
{
    Z1Trace trace("zero1_weight_grad");
    const char *call = "weight gradient";
    int rc = check_ckpt(x8, call, "x8");
    if (rc != ZERO1_OK) return rc;
    if (n < 1) return z1_fail(ZERO1_EINVAL, "%s: n = %lld < 1", call, (long long)n);
    if ((rc = check_dtype(out_dtype, call, "out_dtype")) || (col_scale && (rc = check_dtype(scale_dtype, call, "scale_dtype"))))
        return rc;
    const int64_t T = x8->rows, K = x8->cols;
    const int eo = esize(out_dtype), es = esize(scale_dtype);
    const Mat my = mat(dy, T, n, ld_dy, 2, "dy"), mo = mat(dw, n, K, ld_dw, eo, "dw");
    if ((rc = check_mat(my, 2, false, call)) || (rc = check_mat(mo, eo, true, call)) ||
        (col_scale && (rc = check_natural(col_scale, es, "col_scale"))))
        return rc;
    const Mat in[] = {my, codes_mat(x8, "the codes of x8"), exps_mat(x8, "the exps of x8"),
                      mat(col_scale, 1, K, 0, es, "col_scale")};
    for (const Mat &m : in)
        if (mats_overlap(mo, m)) return z1_fail(ZERO1_EINVAL, "%s: dw and %s overlap", call, m.what);
    Plan p;
    if ((rc = plan_of(T, n, K, dy, ld_dy, &p)) != ZERO1_OK) return rc;
    if (p.bytes > 0) {
        if (!workspace || workspace_bytes < p.bytes)
            return z1_fail(ZERO1_EINVAL, "%s: workspace of %lld bytes, needs %lld", call,
                           (long long)(workspace ? workspace_bytes : 0), (long long)p.bytes);
        if ((uintptr_t)workspace & 127) return z1_fail(ZERO1_EALIGN, "%s: the workspace is not 128-byte aligned", call);
        const Mat w{workspace, 1, p.bytes, p.bytes, "the workspace"};
        for (const Mat &m : {mo, in[0], in[1], in[2], in[3]})
            if (mats_overlap(w, m)) return z1_fail(ZERO1_EINVAL, "%s: the workspace and %s overlap", call, m.what);
    }
    if (T > 0 && (in_host_memory(dy) || in_host_memory(x8->codes) || in_host_memory(x8->exps)))
        return z1_fail(ZERO1_EINVAL, "%s: dy and x8 must be device memory", call);
    if (in_host_memory(dw) || (col_scale && in_host_memory(col_scale)) || (p.bytes > 0 && in_host_memory(workspace)))
        return z1_fail(ZERO1_EINVAL, "%s: dw, col_scale and the workspace must be device memory", call);

    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    Wg a{};
    a.T = T; a.N = n; a.K = K;
    a.tiles_k = p.tiles_k; a.tiles_n = p.tiles_n; a.kblocks = p.kblocks;
    a.whole = p.whole; a.splits = p.splits; a.per_split = p.per_split;
    a.run = out_dtype == ZERO1_DTYPE_F32 ? kRunF32 : kRunBf16;
    a.scale = col_scale;
    a.scale_f32 = scale_dtype == ZERO1_DTYPE_F32;
    a.dw = dw; a.ld_dw = n > 1 ? ld_dw : K;
    a.out_f32 = out_dtype == ZERO1_DTYPE_F32;
    a.accumulate = accumulate != 0;
    a.pairs = ((uintptr_t)dw & (2 * eo - 1)) == 0 && a.ld_dw % 2 == 0;
    a.part = static_cast<float *>(workspace);
    a.held = workspace ? reinterpret_cast<float *>(static_cast<char *>(workspace) + p.held_at) : nullptr;
    if (T > 0) {
        a.exps = x8->exps;
        a.ld_exps = x8->ld_exps;
        const void *src = dy;
        int64_t ld = T > 1 ? ld_dy : round_up(n, 8);
        if (!rows_aligned(dy, ld_dy, T)) {
            uint16_t *copy = reinterpret_cast<uint16_t *>(static_cast<char *>(workspace) + p.copy_at);
            const dim3 grid((unsigned)(T < 32768 ? (T + 7) / 8 : 4096), (unsigned)(p.ld_copy < 256 * 65535 ? (p.ld_copy + 255) / 256 : 65535));
            k_align_rows<<<grid, 256, 0, st>>>(static_cast<const uint16_t *>(dy), T > 1 ? ld_dy : 0, T, n, copy, p.ld_copy);
            if ((rc = launch_status("weight gradient: aligned copy")) != ZERO1_OK) return rc;
            src = copy;
            ld = p.ld_copy;
        }
        // (a box is clipped at dw's edge by 16 bytes)
        a.boxes = a.out_f32 && ((uintptr_t)dw & 15) == 0 && a.ld_dw % 4 == 0 && K % 4 == 0 &&
                  a.ld_dw < (INT64_C(1) << 37);  // (a tensor map's strides are below 2^40 bytes)
        CUtensorMap mdy, mx, mpart{}, mdw{};
        if ((rc = make_map(&mdy, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, src, T, n, ld, 64, "dy")) ||
            (rc = make_map(&mx, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, x8->codes, T, round_up(K, kQBlock), x8->ld_codes, kQBlock,
                           "the codes")) ||
            (p.splits > 1 && (rc = make_map(&mpart, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, workspace, p.held_at / (kTileK * 4), kTileK,
                                            kTileK, 32, "the parts", kBoxRows, CU_TENSOR_MAP_SWIZZLE_NONE))) ||
            (a.boxes && (rc = make_map(&mdw, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, dw, n, K, a.ld_dw, 32, "dw", kBoxRows,
                                       CU_TENSOR_MAP_SWIZZLE_NONE))))
            return rc;
        static std::atomic<uint64_t> done{0};
        const cudaError_t e = allow_smem(k_weight_grad, kWgSmem, done);
        if (e != cudaSuccess) return z1_fail(ZERO1_ECUDA, "%s: %s", call, cudaGetErrorString(e));
        const int64_t items = p.whole + (int64_t)(p.tiles_k * p.tiles_n - p.whole) * p.splits;
        const int grid = 2 * (int)(items < p.clusters ? items : p.clusters);
        const cudaError_t le = launch_after(k_weight_grad, dim3(grid), kWgThreads, kWgSmem, st, mdy, mx, mpart, mdw, a);
        if (le != cudaSuccess) return pdl_fail(le, "weight gradient launch");
        z1_note_launch(reinterpret_cast<const void *>(k_weight_grad), grid, 1, kWgThreads, 0);
        if (p.splits == 1) return ZERO1_OK;
    } else {
        a.whole = a.splits = 0;
    }
    // (no rows: every tile is finished here, without parts)
    for (int t = a.whole, tiles = p.tiles_k * p.tiles_n; t < tiles;) {
        const JoinRun run = join_run(a.whole, tiles, a.splits, t, 65535);
        Wg j = a;
        j.whole = run.tile;
        j.part = a.part + run.part;
        const cudaError_t e = launch_after(k_weight_grad_join, dim3(kTileN / 8, (unsigned)run.tiles), 256, 0, st, j);
        if (e != cudaSuccess) return pdl_fail(e, "weight gradient: joining the parts");
        t += run.tiles;
    }
    return ZERO1_OK;
}
