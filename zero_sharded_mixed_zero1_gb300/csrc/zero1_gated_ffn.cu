// zero1_gated_ffn.cu - the gated feed-forward block on the tensor cores: both
// projections with the activation and the product in one kernel, its backward
// pass with the pre-activations computed again, the gradient of its input, and
// weight gradients from bf16 activations.

#include "zero1_gemm_plan.h"
#include "zero1_tensor.cuh"

namespace {

using namespace z1mm;

// Four products share one kernel (T rows, D the block's width, F its inner one):
//   kForward    g = h Wg^T, u = h Wu^T;  a = act(g) u
//   kBackward   the same g and u;  dg = da u act'(g), du = da act(g), a if wanted
//   kInputGrad  dh = dg Wg + du Wu, one contraction over 2 F
//   kWeightGrad dw (+)= dy^T x, contracted over T
// Two CTAs share a tile of 256 rows x 256 columns (or 128, where that fills the
// pairs better): each loads 128 rows of A and half of B's columns by TMA into a
// ring of swizzled shared memory, one thread issues the MMAs of the pair, and the
// accumulator is kept twice in tensor memory, so that a tile is stored while the
// next one is summed.  For the first two products B's two halves are rows of Wg
// and of Wu: a thread that stores finds the g and the u of an element in its own
// lane of tensor memory.  Operands lie in shared memory as they do in device
// memory, along the contraction (h, Wg, Wu, dg) or across it (the weights of
// kInputGrad, both operands of kWeightGrad); the MMA reads either.
//
// What bounds them at large sizes is the rate of the MMAs, under the power limit over
// seconds: a stage of 64 takes 512 cycles, and as many to bring its 32 KB to each SM
// from L2.  8192 rows, D 4096, F 14336, in a burst (fraction of the measured cuBLAS bf16
// rate) and in a long loop, over four GPUs: forward 930 to 1050 us (0.95 to 1.07) and 1090
// to 1140; backward 1010 to 1220 (0.82 to 0.99) and 1155 to 1200; input gradient 970 to
// 1160 (0.86 to 1.03) and 1160; a bf16 weight gradient 475 to 600 (0.84 to 1.05) and 570,
// fp32 533 to 600 and 600.  With few rows it is HBM: 64 rows 46 us (5.1 TB/s of the
// weights), and below that launch, set-up and one round trip of each: 16 rows of 768 x 2048
// 5.8 us.  At small widths the storing warps hold the backward call up: 12981 x 320 x 4096
// 112 to 122 us (gelu 121 to 128) where forward takes 56 to 60 and the bytes 66.  They issue
// in 46 % of the cycles (gelu 50 %), the tensor pipe works in 24 %: two of them per
// scheduler, each waiting for the last instruction, for da, for tensor memory and for a
// place in turn, do not hide one another's waits.
//
// Roles (12 warps): warp 0 loads, warp 1 of the leading CTA issues the MMAs,
// warp 2 keeps the tensor memory, warps 4-11 store, each 32 rows and half of the
// tile's columns.

constexpr int kForward = 0, kBackward = 1, kInputGrad = 2, kWeightGrad = 3;

constexpr int kThreads = 32 * 12, kStoring = 8;  // storing warps
constexpr int kABytes = 128 * kDeep * 2;
template <int TN>
constexpr int kStageBytes = kABytes + TN / 2 * kDeep * 2;

constexpr int kRingBytes = 6 * kStageBytes<256>;
template <int TN>
constexpr int kStages = kRingBytes / kStageBytes<TN>;

// Results on their way out: 32 rows of 64 bytes, swizzled, in two places of each
// storing warp.  (Four, for a stage less, were no faster where kBackward stores three
// results for each pair of sums, and cost 5% at 8192 x 4096 x 14336.)
constexpr int kPlaceBytes = 32 * 64, kPlaces = 2;

struct Bars {
    uint64_t full[8], empty[8], dfull[2], dempty[2];
    uint32_t tmem;
    uint32_t failed;       // a wait of either CTA ran out
    uint32_t loads, mmas;  // stages loaded and issued
    uint32_t fills;        // accumulator fills issued
};
constexpr int kSmem = 1024 + kRingBytes + kStoring * kPlaces * kPlaceBytes + (int)sizeof(Bars);
static_assert(kSmem <= 227 * 1024, "shared memory of a block");
static_assert(kStages<256> == 6 && kStages<128> == 8, "stages");

struct Out {
    void *p;
    int64_t ld;
    int boxes;  // stored in boxes by TMA
};

struct Mm {
    int64_t M, N;                     // results: rows, columns (of a, or of the gradient)
    int tiles_m, tiles_n, kblocks;    // kblocks: stages of the whole contraction
    int second;                       // the stage from which kInputGrad reads du and Wu
    int a_bytes[2];                   // of A, per stage, that each CTA of a pair loads
    int whole, splits, per_split, run;
    int gelu;
    const uint16_t *da;
    int64_t ld_da;
    int da_vec;                       // da in 128-bit loads
    Out out[3];                       // kForward: a; kBackward: dg, du, a; the others: their gradient
    int out_f32, accumulate;
    float *part;                      // [split tile][part][slot][column][32 lanes]
};

__host__ __device__ constexpr bool dual(int kind) { return kind <= kBackward; }

// ------------------------------------------------------------- operands ----

// Shared-memory descriptor of an operand, 128-byte swizzle, 8 rows per
// 1024-byte group.  Along the contraction: rows of 64 elements.  Across it: TMA
// boxes of 64 elements x kDeep rows of the contraction, one behind the other.
__device__ __forceinline__ uint64_t operand_desc(uint32_t addr, bool across)
{
    return (uint64_t)((addr & 0x3ffff) >> 4) | (uint64_t)(across ? (kDeep * 128) >> 4 : 1) << 16 |
           (uint64_t)(1024 >> 4) << 32 | (uint64_t)1 << 46 | (uint64_t)2 << 61;
}
// From 16 elements of the contraction to the next.
template <bool ACROSS>
constexpr int kDescStep = (ACROSS ? 16 * 128 : 32) >> 4;

__device__ __forceinline__ void mma_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t add)
{
    asm volatile("{ .reg .pred p; setp.ne.u32 p, %4, 0; tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p; }" ::"r"(d),
                 "l"(a), "l"(b), "r"(idesc), "r"(add)
                 : "memory");
}

// fp32 accumulator, bf16 operands, M = 256 (both CTAs).
template <int TN, bool A_ACROSS, bool B_ACROSS>
constexpr uint32_t kInstr = (1u << 4) | (1u << 7) | (1u << 10) | ((A_ACROSS ? 1u : 0u) << 15) | ((B_ACROSS ? 1u : 0u) << 16) |
                            ((uint32_t)(TN / 8) << 17) | ((uint32_t)(kTileM / 16) << 24);

// ---------------------------------------------------------------- items ----

struct Item {
    int m, n, kb0, kb1, part;  // tile's row and column number; part: its place among the parts, -1 for a whole tile
};

// Tiles run in bands of eight along the rows, so that the pairs of CTAs at work
// at one time share few rows of both operands (they meet in L2).
__device__ __forceinline__ void tile_of(const Mm &a, int t, int &m, int &n)
{
    constexpr int kBand = 8;
    const int per = kBand * a.tiles_n, band = t / per, in = t % per;
    const int height = min(kBand, a.tiles_m - band * kBand);
    m = band * kBand + in % height;
    n = in / height;
}

// The whole tiles come first, then all first parts of the others, all second
// ones and so on, so that neighbours in time share operands.
__device__ __forceinline__ Item item_of(const Mm &a, int i)
{
    Item o;
    o.part = -1;
    o.kb0 = 0;
    o.kb1 = a.kblocks;
    int t = i;
    if (i >= a.whole) {
        const int rest = a.tiles_m * a.tiles_n - a.whole, p = (i - a.whole) / rest;
        t = a.whole + (i - a.whole) % rest;
        o.kb0 = p * a.per_split;
        o.kb1 = min(o.kb0 + a.per_split, a.kblocks);
        o.part = (t - a.whole) * a.splits + p;
    }
    tile_of(a, t, o.m, o.n);
    return o;
}

__device__ __forceinline__ int items_of(const Mm &a) { return a.whole + (a.tiles_m * a.tiles_n - a.whole) * a.splits; }

// ----------------------------------------------------------- activation ----

// f = act(g) = g s(k(g)) and df = act'(g) = s + g s (1 - s) k'(g), s the logistic
// function: silu has k(g) = g, the tanh form of gelu 2 sqrt(2 / pi) (g + 0.044715 g^3).
// With e = 2^t, t = k log2(e) cut at 64: s = e / (1 + e), right from the subnormal e of
// very negative k on, and 1 itself from t = 64 on (2^64 and its inverse are exact), in six
// instructions; its error is that of the product t, |k| half steps, which is nothing to
// a bf16 result (the logistic function of the gates, good to 2.5 ulps, takes eleven, and
// the storing warps hold the backward call up at small widths).  s (1 - s) is s
// - s^2 from the rounded s: where s is near but not 1, g k' is at most 140 and a half
// step of s counts for nothing beside the s that it is added to.
// From |g| = 1.17e13 on gelu's g k' leaves fp32, where s is 0 or 1 and s - s^2 is 0 to the
// last bit (both are so from |g| = 16 on): it is cut to a finite value, which 0 makes 0, in
// one instruction that lets NaN through (12981 x 320 x 4096 120.5 us, without it 119.2; a
// comparison and a selection took 3% more).
struct Activated {
    float f, df;
    __device__ __forceinline__ Activated(float g, int gelu)
    {
        constexpr float kA = 1.5957691216f, kB = 0.0713548163f;  // 2 sqrt(2 / pi), 0.044715 of it
        float k = g, dk = g;                                     // dk: g k'(g)
        if (gelu) {
            const float q = __fmul_rn(g, g);
            k = __fmul_rn(g, __fmaf_rn(kB, q, kA));
            asm("min.NaN.xorsign.abs.f32 %0, %1, %2;" : "=f"(dk) : "f"(__fmul_rn(g, __fmaf_rn(3.f * kB, q, kA))), "f"(3e38f));
        }
        float e, r;
        asm("ex2.approx.f32 %0, %1;" : "=f"(e) : "f"(fminf(__fmul_rn(k, 1.44269504f), 64.f)));
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(__fadd_rn(1.f, e)));
        const float s = __fmul_rn(e, r);
        f = __fmul_rn(g, s);
        df = __fmaf_rn(dk, __fmaf_rn(-s, s, s), s);
    }
};

// ------------------------------------------------------------- results -----

// 16 bytes of a place: 64-byte rows, 16-byte pieces exchanged as TMA's 64-byte
// swizzle does, which also keeps these stores off each other's banks.
__device__ __forceinline__ unsigned char *piece(unsigned char *place, int row, int k)
{
    return place + row * 64 + ((k ^ ((row >> 1) & 3)) << 4);
}

// 32 rows x 64 bytes of results from a place: a box, or, off 16-byte boundaries
// or to be added to, an element at a time.  rows, cols: how many of them lie
// inside the matrix.
struct Leaving {
    unsigned char *places;  // of this warp
    int at;

    // Waits until the next place may be written.
    __device__ __forceinline__ unsigned char *next()
    {
        if (elect_one()) asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(kPlaces - 1) : "memory");
        __syncwarp();
        unsigned char *p = places + at * kPlaceBytes;
        at = at + 1 == kPlaces ? 0 : at + 1;
        return p;
    }
    // The place that next() gave is given again.
    __device__ __forceinline__ void again() { at = at == 0 ? kPlaces - 1 : at - 1; }
    // Every use of a place is a group, an empty one where nothing of it lies inside
    // the matrix: next() counts them.
    __device__ __forceinline__ void empty_group()
    {
        __syncwarp();
        if (elect_one()) asm volatile("cp.async.bulk.commit_group;" ::: "memory");
        __syncwarp();
    }
    __device__ __forceinline__ void box(const CUtensorMap *map, int64_t row, int64_t col, bool inside, const unsigned char *place)
    {
        if (!inside) return empty_group();
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (elect_one()) box_out(map, (int)col, (int)row, false, reinterpret_cast<const uint32_t *>(place));
        __syncwarp();
    }
    template <class T>
    __device__ __forceinline__ void elements(T *o, int64_t ld, int rows, int cols, bool add, unsigned char *place)
    {
        constexpr int kCols = 64 / (int)sizeof(T);  // one lane to an element of a row
        const int lane = threadIdx.x & 31, c = lane % kCols;
        __syncwarp();
        if (c < cols) {
#pragma unroll 4
            for (int r = lane / kCols; r < rows; r += 32 / kCols) {
                const T x = *reinterpret_cast<const T *>(piece(place, r, c * (int)sizeof(T) / 16) + c * sizeof(T) % 16);
                T *q = o + r * ld + c;
                if constexpr (sizeof(T) == 4) *q = add ? *q + x : x;
                else *q = x;
            }
        }
        empty_group();
    }
    // fp32 sums stored as bf16, or added to bf16 results, rounded once.
    __device__ __forceinline__ void round_to(uint16_t *o, int64_t ld, int rows, int cols, bool add, unsigned char *place)
    {
        const int lane = threadIdx.x & 31, c = lane % 16;
        __syncwarp();
        if (c < cols) {
#pragma unroll 4
            for (int r = lane / 16; r < rows; r += 2) {
                uint16_t *q = o + r * ld + c;
                const float x = *reinterpret_cast<const float *>(piece(place, r, c / 4) + c % 4 * 4);
                *q = to_bf16(add ? bf_one(*q) + x : x);
            }
        }
        empty_group();
    }
};

// 32 bf16 results of this thread's row, packed in pairs, from column `col` on.
__device__ __forceinline__ void leave_bf16(Leaving &l, const Out &o, const CUtensorMap *map, int64_t row0, int64_t col, int rows,
                                           int64_t N, const uint32_t x[16])
{
    unsigned char *place = l.next();
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int k = 0; k < 4; ++k)
        *reinterpret_cast<uint4 *>(piece(place, lane, k)) = make_uint4(x[4 * k], x[4 * k + 1], x[4 * k + 2], x[4 * k + 3]);
    const int cols = (int)max((int64_t)0, min((int64_t)32, N - col));
    if (o.boxes) {
        l.box(map, row0, col, rows > 0 && cols > 0, place);
    } else {
        l.elements(static_cast<uint16_t *>(o.p) + row0 * o.ld + col, o.ld, rows, cols, false, place);
    }
}

// 16 fp32 sums of this thread's row: stored, or added to what is there, as fp32
// or rounded to bf16.
__device__ __forceinline__ void leave_f32(Leaving &l, const Mm &a, const CUtensorMap *map, int64_t row0, int64_t col, int rows,
                                          const float x[16])
{
    const Out &o = a.out[0];
    unsigned char *place = l.next();
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int k = 0; k < 4; ++k)
        *reinterpret_cast<float4 *>(piece(place, lane, k)) = make_float4(x[4 * k], x[4 * k + 1], x[4 * k + 2], x[4 * k + 3]);
    const int cols = (int)max((int64_t)0, min((int64_t)16, a.N - col));
    if (!a.out_f32)
        l.round_to(static_cast<uint16_t *>(o.p) + row0 * o.ld + col, o.ld, rows, cols, a.accumulate != 0, place);
    else if (a.accumulate || !o.boxes)
        l.elements(static_cast<float *>(o.p) + row0 * o.ld + col, o.ld, rows, cols, a.accumulate != 0, place);
    else l.box(map, row0, col, rows > 0 && cols > 0, place);
}

// The accumulator has been read: it may be filled again.
__device__ __forceinline__ void release(uint64_t *dempty)
{
    tc_before();
    __syncwarp();
    if ((threadIdx.x & 31) == 0) arrive_leader(dempty);
}

// Eight accumulator columns of this thread's lane.
__device__ __forceinline__ void load8_acc(uint32_t addr, uint32_t r[8])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n\ttcgen05.wait::ld.sync.aligned;"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(addr)
                 : "memory");
}

// The sum of a run, put in place of or added to those before it, in registers.
template <int N>
__device__ __forceinline__ void take_run(float (&sum)[N], bool begin, uint32_t acc, uint64_t *dempty)
{
#pragma unroll
    for (int c = 0; c < N; c += 8) {
        uint32_t v[8];
        load8_acc(acc + c, v);
        if (c + 8 == N) release(dempty);
#pragma unroll
        for (int j = 0; j < 8; ++j) sum[c + j] = (begin ? 0.f : sum[c + j]) + __uint_as_float(v[j]);
    }
}

// 16 accumulator columns of g and of u, under way together.
__device__ __forceinline__ void load_pair(uint32_t at_g, uint32_t at_u, uint32_t g[16], uint32_t u[16])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
        "[%32];\n\t"
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, "
        "%31}, [%33];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(g[0]), "=r"(g[1]), "=r"(g[2]), "=r"(g[3]), "=r"(g[4]), "=r"(g[5]), "=r"(g[6]), "=r"(g[7]), "=r"(g[8]),
          "=r"(g[9]), "=r"(g[10]), "=r"(g[11]), "=r"(g[12]), "=r"(g[13]), "=r"(g[14]), "=r"(g[15]), "=r"(u[0]), "=r"(u[1]),
          "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7]), "=r"(u[8]), "=r"(u[9]), "=r"(u[10]),
          "=r"(u[11]), "=r"(u[12]), "=r"(u[13]), "=r"(u[14]), "=r"(u[15])
        : "r"(at_g), "r"(at_u)
        : "memory");
}

// da of a warp's 32 rows x 32 columns from row0, col on: four lanes to a row of 64
// bytes, eight rows at a time, zeros outside.  (A row to each thread asked for 32 lines
// at once: 132 us at 12981 x 320 x 4096 where this takes 113.)  take_da turns that into
// the thread's own row, by way of a place.
__device__ __forceinline__ void load_da(const Mm &a, int64_t row0, int64_t col, uint4 (&d)[4])
{
    const int lane = threadIdx.x & 31;
    col += lane % 4 * 8;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int64_t row = row0 + lane / 4 + 8 * k;
        d[k] = make_uint4(0, 0, 0, 0);
        if (row >= a.M || col >= a.N) continue;
        const uint16_t *p = a.da + row * a.ld_da + col;
        if (a.da_vec && col + 8 <= a.N) {
            d[k] = *reinterpret_cast<const uint4 *>(p);
            continue;
        }
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t lo = col + 2 * j < a.N ? p[2 * j] : 0, hi = col + 2 * j + 1 < a.N ? p[2 * j + 1] : 0;
            w[j] = lo | hi << 16;
        }
        d[k] = make_uint4(w[0], w[1], w[2], w[3]);
    }
}
__device__ __forceinline__ void take_da(const uint4 (&from)[4], uint4 (&d)[4], unsigned char *place)
{
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int k = 0; k < 4; ++k) *reinterpret_cast<uint4 *>(piece(place, lane / 4 + 8 * k, lane % 4)) = from[k];
    __syncwarp();
#pragma unroll
    for (int k = 0; k < 4; ++k) d[k] = *reinterpret_cast<const uint4 *>(piece(place, lane, k));
    __syncwarp();
}

// ----------------------------------------------------------------- kernel --

struct Maps {
    CUtensorMap a0, a1, b0, b1, out0, out1, out2;
};

// RUNS: a contraction of more stages than the accumulator sums at one time; the
// storing threads add the runs up in registers (128 of them each, tensor memory read eight
// columns at a time; of 168 registers two words are spilled).  The tensor cores' truncation is
// one-sided and grows with the terms of a run: an fp32 weight gradient of normal draws is
// off by 2.1e-6 of its norm with runs of 2048 rows, 1.0e-6 with 1024, 4.8e-7 with 512,
// 2.4e-7 with 256 (an fp32 library product 3.9e-7 over 2048 rows, 9.6e-7 over 8192).  512
// rows it is: on one GPU 8192 x 4096 x 14336 took 560 us where sums of 2048 rows held in
// the workspace took 605; 8192 x 1024 x 4096 46 for 53.
template <int KIND, int TN, bool RUNS>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
k_gated_ffn(const __grid_constant__ Maps maps, const Mm a)
{
    constexpr bool kDual = dual(KIND), kAAcross = KIND == kWeightGrad, kBAcross = KIND >= kInputGrad;
    constexpr int S = kStages<TN>, kBytes = kStageBytes<TN>, kBBytes = kBytes - kABytes;
    extern __shared__ unsigned char raw[];
    unsigned char *smem = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
    unsigned char *s_places = smem + kRingBytes;
    Bars &bar = *reinterpret_cast<Bars *>(s_places + kStoring * kPlaces * kPlaceBytes);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cta_rank();
    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(&bar.full[s], 1);
            mbar_init(&bar.empty[s], 1);
        }
        for (int k = 0; k < 2; ++k) {
            mbar_init(&bar.dfull[k], 1);
            mbar_init(&bar.dempty[k], 2 * kStoring);
        }
        bar.failed = bar.loads = bar.mmas = bar.fills = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 2) tc_alloc(&bar.tmem);
    if (warp == 3 && lane == 0) {  // (every product has these two)
        asm volatile("prefetch.tensormap [%0];" ::"l"(&maps.a0) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(&maps.b0) : "memory");
    }
    tc_before();
    __syncthreads();
    cluster_sync();
    tc_after();
    wait_prior_grid();  // up to here this kernel may run beside the one before it
    let_next_grid_start();
    const uint32_t tmem = bar.tmem;
    const int items = items_of(a);
    const int first = blockIdx.x / 2, step = gridDim.x / 2;

    if (warp == 0) {
        uint32_t it = 0;
        bool ok = true;
        for (int i = first; i < items && ok; i += step) {
            const Item w = item_of(a, i);
            const int m = w.m * kTileM + (int)rank * 128;
            const int n = kDual ? w.n * (TN / 2) : w.n * TN + (int)rank * (TN / 2);
            for (int kb = w.kb0; kb < w.kb1; ++kb, ++it) {
                const uint32_t s = it % S;
                if (it >= S && !(ok = warp_wait(bar, &bar.empty[s], (it / S - 1) & 1))) break;
                unsigned char *pa = smem + s * kBytes, *pb = pa + kABytes;
                const bool late = KIND == kInputGrad && kb >= a.second;
                const int k = (late ? kb - a.second : kb) * kDeep;
                const CUtensorMap *ma = late ? &maps.a1 : &maps.a0;
                const CUtensorMap *mb = late || (kDual && rank) ? &maps.b1 : &maps.b0;
                if (elect_one()) {
                    // both CTAs' loads count on the leading CTA's barrier
                    const uint32_t full = leader_addr(&bar.full[s]);
                    if (rank == 0) mbar_expect_tx(&bar.full[s], 2 * kBBytes + a.a_bytes[0] + a.a_bytes[1]);
                    if (a.a_bytes[rank] == 0) {
                    } else if (kAAcross) {
                        tma_2d_pair(pa, ma, m, k, full);
                        tma_2d_pair(pa + kABytes / 2, ma, m + 64, k, full);
                    } else {
                        tma_2d_pair(pa, ma, k, m, full);
                    }
                    if (kBAcross) {
                        tma_2d_pair(pb, mb, n, k, full);
                        if (TN == 256) tma_2d_pair(pb + 64 * kDeep * 2, mb, n + 64, k, full);
                    } else {
                        tma_2d_pair(pb, mb, k, n, full);
                    }
                }
                __syncwarp();
            }
        }
        // the last copies must land before the pair may exit (both CTAs have as many)
        if (rank == 0)
            for (uint32_t q = it > S ? it - S : 0; q < it && ok; ++q)
                ok = warp_wait(bar, &bar.full[q % S], (q / S) & 1);
        if (lane == 0) bar.loads = it;
    } else if (warp == 1) {
        if (rank == 0) {
            uint32_t it = 0, fill = 0, fills = 0;
            bool ok = true;
            const uint64_t a0 = operand_desc(smem_u32(smem), kAAcross), b0 = operand_desc(smem_u32(smem) + kABytes, kBAcross);
            for (int i = first; i < items && ok; i += step) {
                const Item w = item_of(a, i);
                for (int kb = w.kb0; kb < w.kb1 && ok; ++fill) {
                    const uint32_t buf = fill & 1;
                    if (fill >= 2 && !(ok = warp_wait(bar, &bar.dempty[buf], ((fill >> 1) - 1) & 1))) break;
                    const int start = kb, end = min(kb + a.run, w.kb1);
                    for (; kb < end; ++kb, ++it) {
                        const uint32_t s = it % S;
                        const uint64_t da = a0 + (uint64_t)(s * (kBytes >> 4)), db = b0 + (uint64_t)(s * (kBytes >> 4));
                        const uint32_t more = kb > start, acc = tmem + buf * TN;
                        if (!(ok = warp_wait(bar, &bar.full[s], (it / S) & 1))) break;
                        tc_after();
                        if (elect_one()) {
#pragma unroll
                            for (int j = 0; j < kDeep / 16; ++j)
                                mma_pair(acc, da + j * kDescStep<kAAcross>, db + j * kDescStep<kBAcross>,
                                         kInstr<TN, kAAcross, kBAcross>, j ? 1u : more);
                            tc_commit(&bar.empty[s]);
                            if (kb + 1 == end) tc_commit(&bar.dfull[buf]);
                        }
                        __syncwarp();
                    }
                    fills += ok;
                }
            }
            // the MMAs must have finished with both CTAs' memory before the exit
            if (it > 0) warp_wait(bar, &bar.empty[(it - 1) % S], ((it - 1) / S) & 1);
            if (lane == 0) {
                bar.mmas = it;
                bar.fills = fills;
            }
        }
    } else if (warp >= 4) {
        const int q = warp % 4, half = (warp - 4) / 4, slot = (int)rank * 8 + half * 4 + q;
        constexpr int kCols = TN / 2, W = TN / 4;  // accumulator columns of a warp; results' columns where it has g and u
        Leaving leaving{s_places + (warp - 4) * kPlaces * kPlaceBytes, 0};
        uint32_t fill = 0;
        bool ok = true;
        uint4 ahead[4];  // kBackward: da of the next 32 columns, on its way while these are computed
        auto load_ahead = [&](int i, int c) {  // of an item's columns from c on
            if (i >= items) return;
            const Item w = item_of(a, i);
            load_da(a, (int64_t)w.m * kTileM + (int)rank * 128 + 32 * q, (int64_t)w.n * (TN / 2) + half * W + c, ahead);
        };
        if (KIND == kBackward) load_ahead(first, 0);
        for (int i = first; i < items && ok; i += step) {
            const Item w = item_of(a, i);
            const int64_t row0 = (int64_t)w.m * kTileM + (int)rank * 128 + 32 * q;
            const int rows = (int)max((int64_t)0, min((int64_t)32, a.M - row0));
            float *const part = a.part + ((int64_t)w.part * 16 + slot) * kCols * 32 + lane;
            if (kDual) {
                const int64_t col0 = (int64_t)w.n * (TN / 2) + half * W;
                if (!(ok = warp_wait(bar, &bar.dfull[fill & 1], (fill >> 1) & 1))) break;
                tc_after();
                uint64_t *dempty = &bar.dempty[fill & 1];
                const uint32_t acc = tmem + ((uint32_t)(32 * q) << 16) + (fill & 1) * TN + half * W;
                ++fill;
                if (w.part >= 0) {
                    // (of a part, g's columns come first, then u's; the last call releases the accumulator)
                    uint32_t v[16];
#pragma unroll 1
                    for (int c = 0; c < kCols; c += 16) {
                        tc_load16(acc + (c < W ? c : c - W + TN / 2), v);
                        if (c + 16 == kCols) release(dempty);
#pragma unroll
                        for (int j = 0; j < 16; ++j) __stcg(part + (c + j) * 32, __uint_as_float(v[j]));
                    }
                    continue;  // (all items behind it are parts as well: da is not needed again)
                }
#pragma unroll 1
                for (int c = 0; c < W; c += 32) {
                    uint32_t x[3][16];
                    uint4 da[4];
                    if (KIND == kBackward) {
                        take_da(ahead, da, leaving.next());
                        leaving.again();
                        // of the 32 columns after these, of the next tile's after the last ones
                        load_ahead(c + 32 < W ? i : i + step, c + 32 < W ? c + 32 : 0);
                    }
#pragma unroll
                    for (int e = 0; e < 32; e += 16) {
                        uint32_t g[16], u[16];
                        load_pair(acc + c + e, acc + TN / 2 + c + e, g, u);
                        if (c + e + 16 == W) release(dempty);
#pragma unroll
                        for (int j = 0; j < 16; j += 2) {
                            const Activated f0(__uint_as_float(g[j]), a.gelu), f1(__uint_as_float(g[j + 1]), a.gelu);
                            const float u0 = __uint_as_float(u[j]), u1 = __uint_as_float(u[j + 1]);
                            const int at = (e + j) / 2;
                            if (KIND == kForward) {
                                x[0][at] = pack_bf16x2(__fmul_rn(f0.f, u0), __fmul_rn(f1.f, u1));
                            } else {
                                const uint4 d4 = da[(e + j) / 8];
                                const uint32_t d = (j / 2) % 4 == 0 ? d4.x : (j / 2) % 4 == 1 ? d4.y : (j / 2) % 4 == 2 ? d4.z : d4.w;
                                const float d0 = bf_lo(d), d1 = bf_hi(d);
                                x[0][at] = pack_bf16x2(__fmul_rn(__fmul_rn(d0, u0), f0.df), __fmul_rn(__fmul_rn(d1, u1), f1.df));
                                x[1][at] = pack_bf16x2(__fmul_rn(d0, f0.f), __fmul_rn(d1, f1.f));
                                x[2][at] = pack_bf16x2(__fmul_rn(f0.f, u0), __fmul_rn(f1.f, u1));
                            }
                        }
                    }
                    leave_bf16(leaving, a.out[0], &maps.out0, row0, col0 + c, rows, a.N, x[0]);
                    if (KIND == kBackward) {
                        leave_bf16(leaving, a.out[1], &maps.out1, row0, col0 + c, rows, a.N, x[1]);
                        if (a.out[2].p) leave_bf16(leaving, a.out[2], &maps.out2, row0, col0 + c, rows, a.N, x[2]);
                    }
                }
                continue;
            }
            const int64_t col0 = (int64_t)w.n * TN + half * kCols;
            float sum[RUNS ? kCols : 1];
            uint32_t acc = 0;
            uint64_t *dempty = nullptr;
            for (int kb = w.kb0; kb < w.kb1; kb += a.run) {  // (without RUNS once)
                if (!(ok = warp_wait(bar, &bar.dfull[fill & 1], (fill >> 1) & 1))) break;
                tc_after();
                dempty = &bar.dempty[fill & 1];
                acc = tmem + ((uint32_t)(32 * q) << 16) + (fill & 1) * TN + half * kCols;
                ++fill;
                if constexpr (RUNS) take_run(sum, kb == w.kb0, acc, dempty);
            }
            if (!ok) break;
            if constexpr (RUNS) {
                // (registers are not indexed at run time)
                if (w.part >= 0) {
#pragma unroll
                    for (int j = 0; j < kCols; ++j) __stcg(part + j * 32, sum[j]);
                } else {
#pragma unroll
                    for (int c = 0; c < kCols; c += 16) leave_f32(leaving, a, &maps.out0, row0, col0 + c, rows, sum + c);
                }
            } else if (w.part < 0 && !a.out_f32 && !a.accumulate) {
#pragma unroll 1
                for (int c = 0; c < kCols; c += 32) {
                    uint32_t v[32], x[16];
                    tc_load32(acc + c, v);
                    if (c + 32 == kCols) release(dempty);
#pragma unroll
                    for (int j = 0; j < 16; ++j) x[j] = pack_bf16x2(__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1]));
                    leave_bf16(leaving, a.out[0], &maps.out0, row0, col0 + c, rows, a.N, x);
                }
            } else {
#pragma unroll 1
                for (int c = 0; c < kCols; c += 16) {
                    uint32_t v[16];
                    float x[16];
                    tc_load16(acc + c, v);
                    if (c + 16 == kCols) release(dempty);
#pragma unroll
                    for (int j = 0; j < 16; ++j) x[j] = __uint_as_float(v[j]);
                    if (w.part >= 0) {
#pragma unroll
                        for (int j = 0; j < 16; ++j) __stcg(part + (c + j) * 32, x[j]);
                    } else {
                        leave_f32(leaving, a, &maps.out0, row0, col0 + c, rows, x);
                    }
                }
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
    // memory is given back: the loads, by making up what their barriers lack, and
    // the MMAs with the arrivals that follow them.
    if (bar.failed) {
        if (warp == 0 && rank == 0) {
            const uint32_t mine = bar.loads, other = read_rank(&bar.loads, 1), n = max(mine, other);
            for (uint32_t q = n > S ? n - S : 0; q < n; ++q) {
                // a use is complete after the leading CTA's arrival and both CTAs' bytes
                const bool announced = q < mine, there = q < other;
                if (lane == 0)
                    mbar_make_up(&bar.full[q % S], announced ? 0u : 1u, !announced && there ? kBBytes + a.a_bytes[1] : 0u,
                                 announced && !there ? kBBytes + a.a_bytes[1] : 0u);
                __syncwarp();
                warp_wait(bar, &bar.full[q % S], (q / S) & 1);
            }
        } else if (warp == 1) {
            const uint32_t m = read_rank(&bar.mmas, 0), f = read_rank(&bar.fills, 0);
            if (m > 0) warp_wait(bar, &bar.empty[(m - 1) % S], ((m - 1) / S) & 1);
            if (f > 0) warp_wait(bar, &bar.dfull[(f - 1) & 1], ((f - 1) >> 1) & 1);
        }
        __syncthreads();
        cluster_sync();
    }
    if (warp == 2) {
        tc_after();
        tc_free(tmem);
    }
}

// Adds a split tile's parts in order and finishes its results; with no parts at
// all (nothing to contract) the sums are 0.  A block takes 32 rows x 32 columns of
// a tile: sums with lanes along the rows, as they were written, results with lanes
// along the columns.
template <int KIND, int TN>
__global__ void __launch_bounds__(256) k_gated_ffn_join(const Mm a)
{
    constexpr bool kDual = dual(KIND);
    constexpr int kCols = TN / 2, W = kDual ? TN / 4 : TN / 2, kGroups = W / 32;  // results' columns of a warp
    wait_prior_grid();
    let_next_grid_start();
    __shared__ float sum[kDual ? 2 : 1][32][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int slot = blockIdx.x / kGroups, c0 = blockIdx.x % kGroups * 32;
    const int rest = a.tiles_m * a.tiles_n - a.whole;
    for (int t = blockIdx.y; t < rest; t += gridDim.y) {
        int m, n;
        tile_of(a, a.whole + t, m, n);
        const int64_t row0 = (int64_t)m * kTileM + slot / 8 * 128 + slot % 4 * 32;
        const int64_t col0 = (int64_t)n * (kDual ? TN / 2 : TN) + slot / 4 % 2 * W + c0;
        __syncthreads();  // what the tile before left has been read
        if (row0 >= a.M || col0 >= a.N) continue;
        constexpr int kEach = kDual ? 8 : 4;  // columns of a thread, all under way together
        const float *p = a.part + (((int64_t)t * a.splits * 16 + slot) * kCols + c0 + warp * 4) * 32 + lane;
        constexpr int kAtOnce = 16 / kEach;   // of as many parts
        constexpr int64_t kPart = 16 * kCols * 32;
        float x[kEach] = {};
        for (int s = 0; s < a.splits; s += kAtOnce, p += kAtOnce * kPart) {
            float v[kAtOnce][kEach];
#pragma unroll
            for (int j = 0; j < kAtOnce; ++j)
#pragma unroll
                for (int k = 0; k < kEach; ++k) v[j][k] = s + j < a.splits ? __ldcg(p + j * kPart + (k / 4 * W + k % 4) * 32) : 0.f;
#pragma unroll
            for (int j = 0; j < kAtOnce; ++j)
#pragma unroll
                for (int k = 0; k < kEach; ++k) x[k] += v[j][k];
        }
#pragma unroll
        for (int k = 0; k < kEach; ++k) sum[k / 4][warp * 4 + k % 4][lane] = x[k];
        __syncthreads();
        const int64_t col = col0 + lane;
        if (col >= a.N) continue;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int r = warp * 4 + k;
            const int64_t row = row0 + r;
            if (row >= a.M) continue;
            if (kDual) {
                const Activated f(sum[0][lane][r], a.gelu);
                const float u = sum[kDual ? 1 : 0][lane][r];
                const uint16_t y = to_bf16(__fmul_rn(f.f, u));
                if (KIND == kForward) {
                    static_cast<uint16_t *>(a.out[0].p)[row * a.out[0].ld + col] = y;
                } else {
                    const float d = bf_one(a.da[row * a.ld_da + col]);
                    static_cast<uint16_t *>(a.out[0].p)[row * a.out[0].ld + col] = to_bf16(__fmul_rn(__fmul_rn(d, u), f.df));
                    static_cast<uint16_t *>(a.out[1].p)[row * a.out[1].ld + col] = to_bf16(__fmul_rn(d, f.f));
                    if (a.out[2].p) static_cast<uint16_t *>(a.out[2].p)[row * a.out[2].ld + col] = y;
                }
            } else {
                const float x = sum[0][lane][r];
                const int64_t at = row * a.out[0].ld + col;
                if (a.out_f32) {
                    float *o = static_cast<float *>(a.out[0].p) + at;
                    *o = a.accumulate ? *o + x : x;
                } else {
                    uint16_t *o = static_cast<uint16_t *>(a.out[0].p) + at;
                    *o = to_bf16(a.accumulate ? bf_one(*o) + x : x);
                }
            }
        }
    }
}

// ------------------------------------------------------- aligned copies ----
//
// Operands whose rows do not start on 16-byte boundaries (or, along the
// contraction, do not end on one) are copied to rows that do, all of a call's in
// one launch: a warp takes 1024 columns of a row, by the 16-byte pieces that hold
// them, shifted into place; columns past the last one become 0.

constexpr int kCopyCols = 1024;

struct AlignCopy {
    const uint16_t *src;
    uint16_t *dst;
    int64_t ld, rows, cols, wide, segments, end;  // segments of a row; end: of its items among all
};
struct AlignCopies {
    AlignCopy m[4];
    int count;
    int64_t items;
};

// 16 bytes of a matrix that lies in [begin, end); what is outside is not read.
__device__ __forceinline__ uint4 piece_of(const unsigned char *p, const unsigned char *begin, const unsigned char *end)
{
    if (p >= begin && p + 16 <= end) return __ldg(reinterpret_cast<const uint4 *>(p));
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        w[k] = 0;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const unsigned char *q = p + 4 * k + 2 * h;
            if (q >= begin && q < end) w[k] |= (uint32_t) * reinterpret_cast<const uint16_t *>(q) << (16 * h);
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

__global__ void __launch_bounds__(256) k_align_operands(const AlignCopies all)
{
    wait_prior_grid();
    let_next_grid_start();
    const int lane = threadIdx.x & 31;
    for (int64_t i = (int64_t)blockIdx.x * 8 + threadIdx.x / 32; i < all.items; i += (int64_t)gridDim.x * 8) {
        int k = 0;
        while (i >= all.m[k].end) ++k;
        const AlignCopy &m = all.m[k];
        const int64_t in = i - (k ? all.m[k - 1].end : 0), row = in / m.segments, c0 = in % m.segments * kCopyCols + lane * 8;
        const unsigned char *begin = reinterpret_cast<const unsigned char *>(m.src), *end = begin + ((m.rows - 1) * m.ld + m.cols) * 2;
        const unsigned char *p = begin + (row * m.ld + c0) * 2;
        const int odd = (int)((uintptr_t)p & 15) / 2;  // the same for every lane
        p -= 2 * odd;
        uint4 lo[4], hi[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            lo[u] = hi[u] = make_uint4(0, 0, 0, 0);
            if (c0 + 256 * u >= m.cols) continue;
            lo[u] = piece_of(p + 512 * u, begin, end);
            if (odd) hi[u] = piece_of(p + 512 * u + 16, begin, end);
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int64_t c = c0 + 256 * u;
            if (c >= m.wide) continue;
            const uint32_t x[9] = {lo[u].x, lo[u].y, lo[u].z, lo[u].w, hi[u].x, hi[u].y, hi[u].z, hi[u].w, 0};
            uint32_t w[5], o[4];
            if (odd & 4) {
#pragma unroll
                for (int j = 0; j < 5; ++j) w[j] = odd & 2 ? x[min(j + 3, 8)] : x[j + 2];
            } else {
#pragma unroll
                for (int j = 0; j < 5; ++j) w[j] = odd & 2 ? x[j + 1] : x[j];
            }
            const int left = (int)min((int64_t)8, m.cols - c);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                o[j] = odd & 1 ? __funnelshift_r(w[j], w[j + 1], 16) : w[j];
                if (2 * j >= left) o[j] = 0;
                else if (2 * j + 1 >= left) o[j] &= 0xffffu;
            }
            *reinterpret_cast<uint4 *>(m.dst + row * m.wide + c) = make_uint4(o[0], o[1], o[2], o[3]);
        }
    }
}

// --------------------------------------------------------------- launch ----

// An operand as a product takes it.
struct Operand {
    const void *p;
    int64_t rows, cols, ld;
    bool across;  // the contraction runs over the rows
    const char *what;
};

// Rows that TMA can address as they are.  Along the contraction their width is a
// multiple of eight elements too: what a box takes beyond the last column has to
// be zero.
bool usable(const Operand &o)
{
    return rows_aligned(o.p, o.ld, o.rows) && (o.across || o.cols % 8 == 0) && (o.rows <= 1 || o.ld < (INT64_C(1) << 38));
}

int64_t copy_bytes(const Operand &o) { return usable(o) ? 0 : round_up(o.rows * round_up(o.cols, 8) * 2, 128); }

// One product: its plan, and the workspace's bytes with the operands' copies.
struct Call {
    const char *name;
    int kind;
    int64_t M, N, K;  // K: the contraction, of one of kInputGrad's two halves
    Operand a[2], b[2];
    int na, nb;
    int run;
    Plan plan;
    int64_t bytes;
};

int plan_call(Call *c)
{
    if (c->M > INT32_MAX - 256 || c->N > INT32_MAX / 2 - 256 || c->K > INT32_MAX / 2 - 256)
        return z1_fail(ZERO1_ERANGE, "%s: %lld x %lld x %lld: size not supported", c->name, (long long)c->M, (long long)c->N,
                       (long long)c->K);
    const int sms = sm_count();
    if (sms == 0) return z1_fail(ZERO1_ECUDA, "%s: no CUDA device", c->name);
    if (dual(c->kind) && c->K > (int64_t)kRunBf16 * kDeep)
        return z1_fail(ZERO1_ERANGE, "%s: a width of %lld (at most %d)", c->name, (long long)c->K, kRunBf16 * kDeep);
    const int64_t stages = (c->K + kDeep - 1) / kDeep * (c->kind == kInputGrad ? 2 : 1);
    const int64_t N = dual(c->kind) ? 2 * c->N : c->N;
    if ((c->M + 255) / 256 * ((N + 127) / 128) > (1 << 24))
        return z1_fail(ZERO1_ERANGE, "%s: %lld x %lld results: size not supported", c->name, (long long)c->M, (long long)c->N);
    c->plan = plan_of(c->M, N, (int)stages, sms / 2);
    c->bytes = c->plan.bytes;
    for (int k = 0; k < c->na; ++k) c->bytes += copy_bytes(c->a[k]);
    for (int k = 0; k < c->nb; ++k) c->bytes += copy_bytes(c->b[k]);
    return ZERO1_OK;
}

int check_workspace(const Call &c, const void *workspace, int64_t bytes, const Mat *mats, int n)
{
    if (c.bytes == 0) return ZERO1_OK;
    if (!workspace || bytes < c.bytes)
        return z1_fail(ZERO1_EINVAL, "%s: workspace of %lld bytes, needs %lld", c.name, (long long)(workspace ? bytes : 0),
                       (long long)c.bytes);
    if ((uintptr_t)workspace & 127) return z1_fail(ZERO1_EALIGN, "%s: the workspace is not 128-byte aligned", c.name);
    const Mat w{workspace, 1, c.bytes, c.bytes, "the workspace"};
    for (int k = 0; k < n; ++k)
        if (mats_overlap(w, mats[k])) return z1_fail(ZERO1_EINVAL, "%s: the workspace and %s overlap", c.name, mats[k].what);
    if (in_host_memory(workspace)) return z1_fail(ZERO1_EINVAL, "%s: the workspace must be device memory", c.name);
    return ZERO1_OK;
}

int check_device(const char *call, const Mat *mats, int n)
{
    for (int k = 0; k < n; ++k)
        if (mats[k].p && mats[k].rows > 0 && in_host_memory(mats[k].p))
            return z1_fail(ZERO1_EINVAL, "%s: %s must be device memory", call, mats[k].what);
    return ZERO1_OK;
}

// Rows of A's boxes along the contraction.  Where one tile holds all rows, no more of
// them are loaded than there are; what lies in shared memory beyond is summed into
// rows that are not stored.  (One row of 4096 x 14336 forward takes 45 us, with boxes of
// 128 rows 81.)
int a_rows(const Call &c) { return c.M < 128 ? (int)round_up(c.M, 8) : 128; }

// The map of an operand, or of its copy in the workspace.
int operand_map(const Call &c, const Operand &o, int box_rows, const AlignCopy *copy, CUtensorMap *map)
{
    const int64_t cols = copy ? copy->wide : o.cols, ld = copy ? copy->wide : o.rows > 1 ? o.ld : round_up(o.cols, 8);
    return make_map(c.name, map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, copy ? copy->dst : o.p, o.rows, cols, ld, 64, o.what, box_rows);
}

// The maps of a product's operands, after one launch that copies those that TMA
// cannot address.
int operand_maps(const Call &c, int b_rows, char *scratch, Maps *maps, int sms, cudaStream_t st)
{
    const Operand *ops[4] = {c.a, c.b, c.na > 1 ? c.a + 1 : nullptr, c.nb > 1 ? c.b + 1 : nullptr};
    CUtensorMap *to[4] = {&maps->a0, &maps->b0, &maps->a1, &maps->b1};
    AlignCopies all{};
    const AlignCopy *copy[4] = {};
    for (int k = 0; k < 4; ++k) {
        if (!ops[k] || usable(*ops[k])) continue;
        const Operand &o = *ops[k];
        AlignCopy &q = all.m[all.count++];
        q = AlignCopy{static_cast<const uint16_t *>(o.p), reinterpret_cast<uint16_t *>(scratch), o.rows > 1 ? o.ld : 0, o.rows, o.cols,
                      round_up(o.cols, 8), (o.cols + kCopyCols - 1) / kCopyCols, 0};
        scratch += copy_bytes(o);
        all.items += o.rows * q.segments;
        q.end = all.items;
        copy[k] = &q;
    }
    if (all.count) {
        const int64_t need = (all.items + 7) / 8, wave = (int64_t)sms * 8;
        const cudaError_t e = launch_after(k_align_operands, dim3((unsigned)(need < wave ? need : wave)), 256, 0, st, all);
        if (e != cudaSuccess) return pdl_fail(e, "gated feed-forward: aligned copies");
    }
    for (int k = 0; k < 4; ++k) {
        if (!ops[k]) continue;
        const int rc = operand_map(c, *ops[k], ops[k]->across ? kDeep : k % 2 ? b_rows : a_rows(c), copy[k], to[k]);
        if (rc != ZERO1_OK) return rc;
    }
    return ZERO1_OK;
}

int out_map(const Call &c, const Out &o, int64_t M, int64_t N, bool f32, CUtensorMap *map, const char *what)
{
    if (!o.p || !o.boxes) return ZERO1_OK;
    return make_map(c.name, map, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, f32 ? 4 : 2, o.p, M, N,
                    o.ld, f32 ? 16 : 32, what, 32, CU_TENSOR_MAP_SWIZZLE_64B);
}

// A result matrix; boxes where its rows start on 16-byte boundaries and end on one
// (a box is clipped by 16 bytes).
Out out_of(const Mat &m, int es)
{
    Out o{const_cast<void *>(m.p), m.pitch / es, 0};
    o.boxes = m.p && (((uintptr_t)m.p | (uintptr_t)m.pitch | (uintptr_t)m.width) & 15) == 0 && m.pitch < (INT64_C(1) << 39);
    return o;
}

template <int KIND, int TN, bool RUNS>
int launch(const Call &c, Mm &a, void *workspace, cudaStream_t st)
{
    auto kernel = k_gated_ffn<KIND, TN, RUNS>;
    const Plan &p = c.plan;
    a.M = c.M; a.N = c.N;
    a.tiles_m = p.tiles_m; a.tiles_n = p.tiles_n; a.kblocks = p.kblocks;
    a.second = p.kblocks / 2;
    a.whole = p.whole; a.splits = p.splits; a.per_split = p.per_split;
    a.run = c.run;
    a.a_bytes[0] = KIND == kWeightGrad ? kABytes : a_rows(c) * kDeep * 2;
    a.a_bytes[1] = KIND == kWeightGrad || c.M > 128 ? kABytes : 0;
    a.part = static_cast<float *>(workspace);
    int rc;
    if (p.kblocks > 0) {
        Maps maps{};
        if ((rc = operand_maps(c, TN / 2, static_cast<char *>(workspace) + p.bytes, &maps, 2 * p.clusters, st))) return rc;
        if ((rc = out_map(c, a.out[0], c.M, c.N, a.out_f32, &maps.out0, "the results")) ||
            (rc = out_map(c, a.out[1], c.M, c.N, false, &maps.out1, "du")) ||
            (rc = out_map(c, a.out[2], c.M, c.N, false, &maps.out2, "a")))
            return rc;
        static std::atomic<uint64_t> done{0};
        const cudaError_t e = allow_smem(kernel, kSmem, done);
        if (e != cudaSuccess) return z1_fail(ZERO1_ECUDA, "%s: %s", c.name, cudaGetErrorString(e));
        const int64_t items = p.whole + ((int64_t)p.tiles_m * p.tiles_n - p.whole) * p.splits;
        const int grid = 2 * (int)(items < p.clusters ? items : p.clusters);
        const cudaError_t le = launch_after(kernel, dim3(grid), kThreads, kSmem, st, maps, a);
        if (le != cudaSuccess) return pdl_fail(le, c.name);
        z1_note_launch(reinterpret_cast<const void *>(kernel), grid, 1, kThreads, 0);
        if (p.splits == 1) return ZERO1_OK;
    } else {
        a.whole = a.splits = 0;  // every tile is finished here, without parts
    }
    constexpr int kGroups = (dual(KIND) ? TN / 4 : TN / 2) / 32;
    const int64_t rest = (int64_t)p.tiles_m * p.tiles_n - a.whole;
    const cudaError_t e = launch_after(k_gated_ffn_join<KIND, TN>, dim3(16 * kGroups, (unsigned)(rest < 65535 ? rest : 65535)), 256, 0,
                                       st, a);
    if (e != cudaSuccess) return pdl_fail(e, c.name);
    return ZERO1_OK;
}

template <int KIND>
int launch_tile(const Call &c, Mm &a, void *workspace, zero1_stream_t stream)
{
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if constexpr (!dual(KIND)) {  // (the widths of the others fit one run)
        if (c.plan.kblocks > c.run)
            return c.plan.tn == 256 ? launch<KIND, 256, true>(c, a, workspace, st) : launch<KIND, 128, true>(c, a, workspace, st);
    }
    return c.plan.tn == 256 ? launch<KIND, 256, false>(c, a, workspace, st) : launch<KIND, 128, false>(c, a, workspace, st);
}

// ------------------------------------------------- gated feed-forward ------

// The matrices of a call; those that it does not use are absent.
struct Ffn {
    Mat h, w_gate, w_up, da, a, dg, du, dh;
};

Ffn mats_of(const zero1_gated_ffn_t *f)
{
    const int64_t T = f->rows, D = f->d_model, F = f->d_ff;
    return Ffn{mat(f->h, T, D, f->ld_h, 2, "h"), mat(f->w_gate, F, D, f->ld_w_gate, 2, "w_gate"),
               mat(f->w_up, F, D, f->ld_w_up, 2, "w_up"), mat(f->da, T, F, f->ld_da, 2, "da"), mat(f->a, T, F, f->ld_a, 2, "a"),
               mat(f->dg, T, F, f->ld_dg, 2, "dg"), mat(f->du, T, F, f->ld_du, 2, "du"), mat(f->dh, T, D, f->ld_dh, 2, "dh")};
}

Operand operand(const Mat &m, int64_t cols, bool across) { return Operand{m.p, m.rows, cols, m.rows > 1 ? m.pitch / 2 : cols, across, m.what}; }

int check_sizes(const zero1_gated_ffn_t *f, const char *call)
{
    if (!f) return z1_fail(ZERO1_EINVAL, "%s: the arguments are NULL", call);
    if (f->rows < 0 || f->d_model < 1 || f->d_ff < 1)
        return z1_fail(ZERO1_EINVAL, "%s: %lld rows, widths %lld and %lld", call, (long long)f->rows, (long long)f->d_model,
                       (long long)f->d_ff);
    if (f->act != ZERO1_FFN_SILU && f->act != ZERO1_FFN_GELU) return z1_fail(ZERO1_EINVAL, "%s: unknown activation %d", call, f->act);
    if (f->rows > INT32_MAX / 2 || f->d_model > INT32_MAX / 4 || f->d_ff > INT32_MAX / 4)
        return z1_fail(ZERO1_ERANGE, "%s: size not supported", call);
    return ZERO1_OK;
}

const char *const kNames[] = {"gated feed-forward", "gated feed-forward backward", "gated feed-forward input gradient"};

void fill_call(Call *c, const zero1_gated_ffn_t *f, int kind)
{
    const Ffn x = mats_of(f);
    const int64_t D = f->d_model, F = f->d_ff;
    *c = Call{};
    c->name = kNames[kind];
    c->kind = kind;
    c->run = kRunBf16;
    c->M = f->rows;
    if (kind == kInputGrad) {
        c->N = D; c->K = F;
        c->a[0] = operand(x.dg, F, false); c->a[1] = operand(x.du, F, false);
        c->b[0] = operand(x.w_gate, D, true); c->b[1] = operand(x.w_up, D, true);
        c->na = c->nb = 2;
    } else {
        c->N = F; c->K = D;
        c->a[0] = operand(x.h, D, false);
        c->b[0] = operand(x.w_gate, D, false); c->b[1] = operand(x.w_up, D, false);
        c->na = 1; c->nb = 2;
    }
}

// EINVAL if an output shares memory with an input or another output; dg may be
// da (the same pointer and stride).
int check_ffn(const Call &c, const zero1_gated_ffn_t *f, Mat all[7], int *count)
{
    const Ffn x = mats_of(f);
    Mat in[4], out[3];
    int ni = 0, no = 0, rc;
    in[ni++] = x.w_gate;
    in[ni++] = x.w_up;
    if (c.kind == kInputGrad) {
        in[ni++] = x.dg;
        in[ni++] = x.du;
        out[no++] = x.dh;
    } else {
        in[ni++] = x.h;
        if (c.kind == kBackward) {
            in[ni++] = x.da;
            out[no++] = x.dg;
            out[no++] = x.du;
        }
        if (c.kind == kForward || x.a.p) out[no++] = x.a;
    }
    for (int k = 0; k < ni; ++k)
        if ((rc = check_mat(in[k], 2, false, c.name)) != ZERO1_OK) return rc;
    for (int k = 0; k < no; ++k)
        if ((rc = check_mat(out[k], 2, true, c.name)) != ZERO1_OK) return rc;
    for (int o = 0; o < no; ++o) {
        for (int k = o + 1; k < no; ++k)
            if (mats_overlap(out[o], out[k])) return z1_fail(ZERO1_EINVAL, "%s: %s and %s overlap", c.name, out[o].what, out[k].what);
        for (int k = 0; k < ni; ++k) {
            if (!mats_overlap(out[o], in[k])) continue;
            if (c.kind == kBackward && o == 0 && k == 3 && out[o].p == in[k].p && out[o].pitch == in[k].pitch) continue;
            return z1_fail(ZERO1_EINVAL, "%s: %s and %s overlap", c.name, out[o].what, in[k].what);
        }
    }
    *count = 0;
    for (int k = 0; k < ni; ++k) all[(*count)++] = in[k];
    for (int k = 0; k < no; ++k) all[(*count)++] = out[k];
    return ZERO1_OK;
}

// Checks and plans a call; nothing is left to do without rows (*idle).
int begin_call(Call *c, const zero1_gated_ffn_t *f, int kind, void *workspace, int64_t bytes, bool *idle)
{
    int rc = check_sizes(f, kNames[kind]), n;
    if (rc != ZERO1_OK) return rc;
    *idle = f->rows == 0;
    if (*idle) return ZERO1_OK;
    Mat all[7];
    fill_call(c, f, kind);
    if ((rc = check_ffn(*c, f, all, &n)) || (rc = plan_call(c)) || (rc = check_workspace(*c, workspace, bytes, all, n))) return rc;
    return check_device(c->name, all, n);
}

}  // namespace

int z1_gated_ffn_status(uint32_t *status, int32_t clear) { return (int)async_status(status, clear); }

extern "C" int zero1_gated_ffn_workspace(const zero1_gated_ffn_t *ffn, int32_t call, int64_t *bytes)
{
    const char *name = "gated feed-forward workspace";
    if (!bytes) return z1_fail(ZERO1_EINVAL, "%s: bytes is NULL", name);
    if (call < ZERO1_FFN_FORWARD || call > ZERO1_FFN_INPUT_GRAD) return z1_fail(ZERO1_EINVAL, "%s: unknown call %d", name, call);
    int rc = check_sizes(ffn, name);
    if (rc != ZERO1_OK) return rc;
    *bytes = 0;
    if (ffn->rows == 0) return ZERO1_OK;
    Call c;
    fill_call(&c, ffn, call);
    if ((rc = plan_call(&c)) == ZERO1_OK) *bytes = c.bytes;
    return rc;
}

extern "C" int zero1_gated_ffn_forward(const zero1_gated_ffn_t *ffn, void *workspace, int64_t workspace_bytes, zero1_stream_t stream)
{
    Z1Trace trace("zero1_gated_ffn_forward");
    Call c;
    bool idle;
    const int rc = begin_call(&c, ffn, kForward, workspace, workspace_bytes, &idle);
    if (rc != ZERO1_OK || idle) return rc;
    Mm a{};
    a.gelu = ffn->act == ZERO1_FFN_GELU;
    a.out[0] = out_of(mats_of(ffn).a, 2);
    return launch_tile<kForward>(c, a, workspace, stream);
}

extern "C" int zero1_gated_ffn_backward(const zero1_gated_ffn_t *ffn, void *workspace, int64_t workspace_bytes, zero1_stream_t stream)
{
    Z1Trace trace("zero1_gated_ffn_backward");
    Call c;
    bool idle;
    const int rc = begin_call(&c, ffn, kBackward, workspace, workspace_bytes, &idle);
    if (rc != ZERO1_OK || idle) return rc;
    const Ffn x = mats_of(ffn);
    Mm a{};
    a.gelu = ffn->act == ZERO1_FFN_GELU;
    a.da = static_cast<const uint16_t *>(ffn->da);
    a.ld_da = x.da.rows > 1 ? ffn->ld_da : 0;
    a.da_vec = vec_ok(x.da);
    a.out[0] = out_of(x.dg, 2);
    a.out[1] = out_of(x.du, 2);
    a.out[2] = out_of(x.a, 2);
    return launch_tile<kBackward>(c, a, workspace, stream);
}

extern "C" int zero1_gated_ffn_input_grad(const zero1_gated_ffn_t *ffn, void *workspace, int64_t workspace_bytes, zero1_stream_t stream)
{
    Z1Trace trace("zero1_gated_ffn_input_grad");
    Call c;
    bool idle;
    const int rc = begin_call(&c, ffn, kInputGrad, workspace, workspace_bytes, &idle);
    if (rc != ZERO1_OK || idle) return rc;
    Mm a{};
    a.out[0] = out_of(mats_of(ffn).dh, 2);
    return launch_tile<kInputGrad>(c, a, workspace, stream);
}

// ------------------------------------------------------ weight gradient ----

namespace {

int weight_call(Call *c, int64_t rows, int64_t n, int64_t k, const void *dy, int64_t ld_dy, const void *x, int64_t ld_x,
                int32_t out_dtype, const char *call)
{
    if (rows < 0 || n < 1 || k < 1)
        return z1_fail(ZERO1_EINVAL, "%s: %lld rows, %lld x %lld outputs", call, (long long)rows, (long long)n, (long long)k);
    const int rc = check_dtype(out_dtype, call, "out_dtype");
    if (rc != ZERO1_OK) return rc;
    *c = Call{};
    c->name = call;
    c->kind = kWeightGrad;
    c->M = n; c->N = k; c->K = rows;
    c->a[0] = Operand{dy, rows, n, ld_dy, true, "dy"};
    c->b[0] = Operand{x, rows, k, ld_x, true, "x"};
    c->na = c->nb = rows > 0 ? 1 : 0;
    c->run = out_dtype == ZERO1_DTYPE_F32 ? kRunF32 : kRunBf16;
    return ZERO1_OK;
}

}  // namespace

extern "C" int zero1_weight_grad_bf16_workspace(int64_t rows, int64_t n, int64_t k, const void *dy, int64_t ld_dy, const void *x,
                                                int64_t ld_x, int32_t out_dtype, int64_t *bytes)
{
    const char *call = "bf16 weight gradient workspace";
    if (!bytes) return z1_fail(ZERO1_EINVAL, "%s: bytes is NULL", call);
    Call c;
    int rc = weight_call(&c, rows, n, k, dy, ld_dy, x, ld_x, out_dtype, call);
    if (rc == ZERO1_OK && (rc = plan_call(&c)) == ZERO1_OK) *bytes = c.bytes;
    return rc;
}

extern "C" int zero1_weight_grad_bf16(const void *dy, int64_t ld_dy, int64_t n, const void *x, int64_t ld_x, int64_t k, int64_t rows,
                                      void *dw, int64_t ld_dw, int32_t out_dtype, int32_t accumulate, void *workspace,
                                      int64_t workspace_bytes, zero1_stream_t stream)
{
    Z1Trace trace("zero1_weight_grad_bf16");
    const char *call = "bf16 weight gradient";
    Call c;
    int rc = weight_call(&c, rows, n, k, dy, ld_dy, x, ld_x, out_dtype, call);
    if (rc != ZERO1_OK) return rc;
    const int eo = esize(out_dtype);
    const Mat all[] = {mat(dw, n, k, ld_dw, eo, "dw"), mat(dy, rows, n, ld_dy, 2, "dy"), mat(x, rows, k, ld_x, 2, "x")};
    if ((rc = check_mat(all[0], eo, true, call)) || (rc = check_mat(all[1], 2, false, call)) || (rc = check_mat(all[2], 2, false, call)))
        return rc;
    for (int q = 1; q < 3; ++q)
        if (mats_overlap(all[0], all[q])) return z1_fail(ZERO1_EINVAL, "%s: dw and %s overlap", call, all[q].what);
    if ((rc = plan_call(&c)) || (rc = check_workspace(c, workspace, workspace_bytes, all, 3)) ||
        (rc = check_device(call, all, 3)))
        return rc;
    if (rows == 0 && accumulate) return ZERO1_OK;  // (adding 0 would make -0 of dw +0 and change a NaN's bits)
    Mm a{};
    a.out[0] = out_of(all[0], eo);
    a.out_f32 = out_dtype == ZERO1_DTYPE_F32;
    a.accumulate = accumulate != 0;
    return launch_tile<kWeightGrad>(c, a, workspace, stream);
}
