// zero1_layer_norm.cuh - the kernels of layer norm with its residual, forward and
// backward (library-internal; each source that includes this compiles one pair of
// types: activations, residual stream).
#pragma once

#include "zero1_block_norm.cuh"

namespace z1ln {

struct Fwd {
    int64_t rows;
    int D;
    float eps, alpha, inv_d, inv_d_low;  // 1 / D, and what its rounding leaves
    int pf32;                // fp32 weight and bias
    const void *x, *y, *w, *b;  // y, w, b may be NULL
    void *r, *h;             // r NULL without y
    float *mean, *rstd;
    z1bn::Ckpt r8;           // codes NULL: not wanted
    int64_t ld_x, ld_y, ld_r, ld_h;
};

struct Bwd {
    int64_t rows;
    int D;
    float alpha, inv_d;
    int pf32;
    const void *dh, *dr, *r, *w;  // dr, w may be NULL; r NULL with a checkpoint
    const float *mean, *rstd;
    z1bn::Ckpt r8;
    void *dx, *dy;           // dy may be NULL
    int64_t ld_dh, ld_dr, ld_r, ld_dx, ld_dy;
    int need_w, need_b;
    float *part;             // [2][blocks][ld_part]: partial column sums (dw, db)
    int ld_part;             // D rounded up to 8, so that eight columns are two 16-byte stores
};

// Launch for one pair of types; vec: every row can be read and written in
// 128-bit accesses.
template <class TA, class TR>
int run_forward(const Fwd &a, bool vec, int sms, cudaStream_t st);
template <class TA, class TR>
int run_backward(const Bwd &a, bool vec, int64_t grid, cudaStream_t st);

}  // namespace z1ln

namespace {

// Sum of eight values.
__device__ __forceinline__ float sum8(const V8 &v)
{
    const float2 s = split(add2(add2(v.p[0], v.p[1]), add2(v.p[2], v.p[3])));
    return s.x + s.y;
}
__device__ __forceinline__ V8 plus8(const V8 &v, float x)
{
    const uint64_t p = pair(x, x);
    return V8{{add2(v.p[0], p), add2(v.p[1], p), add2(v.p[2], p), add2(v.p[3], p)}};
}

// Two sums over the block at one barrier, the same in every thread.
template <int T>
__device__ __forceinline__ float2 block_sum2(float x, float y, float2 *red)
{
    const int lane = threadIdx.x & 31;
    x = warp_sum(x);
    y = warp_sum(y);
    if (lane == 0) red[threadIdx.x >> 5] = make_float2(x, y);
    __syncthreads();
    float2 s = red[lane & (T / 32 - 1)];
#pragma unroll
    for (int o = T / 64; o > 0; o >>= 1) {
        s.x += __shfl_xor_sync(0xffffffffu, s.x, o);
        s.y += __shfl_xor_sync(0xffffffffu, s.y, o);
    }
    return s;
}

// The mean of a row from its sum: by 1 / D in two parts, as the rounded inverse alone
// moves the mean of equal values off their value, which 1 / sqrt(eps) then multiplies
// (100, 1000 times: 2e-3 in h).  (An infinite sum stays one.  A division instead took
// 7.9 us for 6.9 at 2003 x 1021 fp32.)
__device__ __forceinline__ float mean_of(float sum, const z1ln::Fwd &a)
{
    constexpr float kMost = 3e38f;
    return __fmaf_rn(sum, a.inv_d, fminf(fmaxf(__fmul_rn(sum, a.inv_d_low), -kMost), kMost));
}

// How a row's columns are shared out over a block, in chunks of eight per thread.
// kAligned: eight consecutive ones, in 128-bit accesses; kAnywhere: the same at any
// element offset, by the words that hold them; kLanes: fp32 rows at any offset
// without a checkpoint, a thread's columns 16 apart, so that 16 lanes copy and
// store 64 consecutive bytes (2003 x 1021, backward: 12 us, where words of eight
// consecutive columns per thread took 20).
enum class Lay { kAnywhere, kAligned, kLanes };  // (no number: it must not pass for a count or a flag)
constexpr Lay kAnywhere = Lay::kAnywhere, kAligned = Lay::kAligned, kLanes = Lay::kLanes;

template <int T, Lay LAY>
struct Cols {
    using Ld = Row<T, LAY == kAligned>;
    static __device__ __forceinline__ int col(int i)
    {
        return LAY == kLanes ? chunk_col<false>(i, threadIdx.x, T) : threadIdx.x * 8 + i * T * 8;
    }
    template <int E>
    static __host__ __device__ constexpr int bytes(int n)
    {
        return LAY == kLanes ? n * E : Ld::template bytes<E>(n);
    }
    template <int E>
    static __device__ __forceinline__ void copy(unsigned char *region, int i, const void *row, int D, bool first)
    {
        if constexpr (LAY == kLanes) {
            const float *src = static_cast<const float *>(row);
            const uint32_t d = (uint32_t)__cvta_generic_to_shared(region) + (i * 8 * T + threadIdx.x) * 4;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int c = col(i) + 16 * k, n = c < D ? 4 : 0;
                asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(d + 4 * T * k), "l"(n ? src + c : src), "r"(n) : "memory");
            }
        } else {
            Ld::template copy<E>(region, i, row, col(i), D, first);
        }
    }
    template <class V>
    static __device__ __forceinline__ V8 take(const unsigned char *region, int i, const V *row)
    {
        if constexpr (LAY == kLanes) {
            const float *f = reinterpret_cast<const float *>(region) + i * 8 * T + threadIdx.x;
            return V8{{pair(f[0], f[T]), pair(f[2 * T], f[3 * T]), pair(f[4 * T], f[5 * T]), pair(f[6 * T], f[7 * T])}};
        } else {
            return Ld::template take<V>(region, i, row);
        }
    }
    template <class V>
    static __device__ __forceinline__ void put(V *row, int i, int D, const V8 &v)
    {
        if constexpr (LAY == kLanes) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float2 f = split(v.p[k]);
                const int c = col(i) + 32 * k;
                if (c < D) __stcs(row + c, f.x);
                if (c + 16 < D) __stcs(row + c + 16, f.y);
            }
        } else {
            Ld::put(row, col(i), D, v);
        }
    }
    // The values below column D, zeros beyond.
    static __device__ __forceinline__ V8 inside(const V8 &v, int i, int D)
    {
        if constexpr (LAY == kAligned) return v;
        if constexpr (LAY == kAnywhere) return below(v, col(i), D);
        V8 r;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float2 f = split(v.p[k]);
            const int c = col(i) + 32 * k;
            r.p[k] = pair(c < D ? f.x : 0.f, c + 16 < D ? f.y : 0.f);
        }
        return r;
    }
};

// Keeps a [D] vector in shared memory as fp32 values, as keep_vector does and in
// the columns' layout; `without` where there is none.
template <int T, int C, Lay LAY>
__device__ __forceinline__ void keep_or(unsigned char *kept, const void *src, int f32, int D, float without)
{
    if (src && LAY != kLanes) return keep_vector<T, C>(kept, src, f32, D, 0);
#pragma unroll
    for (int i = 0; i < C; ++i) {
        float f[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) f[k] = without;
        if (src) param8<false>(src, f32, 0, 0, Cols<T, LAY>::col(i), D, f);
        float4 *q = reinterpret_cast<float4 *>(kept) + i * T + threadIdx.x;
        q[0] = make_float4(f[0], f[1], f[2], f[3]);
        q[C * T] = make_float4(f[4], f[5], f[6], f[7]);
    }
}

// ------------------------------------------------------------- forward -----
//
//   r = x + a y;  mean = sum r / D;  rstd = 1 / sqrt(sum (r - mean)^2 / D + eps)
//   rh = (r - mean) rstd;  h = w rh + b
//
// One pass over memory: x and y are read once, through the block norms' ring of
// shared-memory stages (a thread copies and reads its own columns, so the ring
// needs no barrier); the row stays in registers for both sums, the second one of
// squares of differences, so that the variance does not cancel.  A large mean costs what
// its fp32 sum is rounded by, a few 2^-24 of it in every r - mean: h of fp32 rows of mean
// 1000 and spread 1 is off by 3e-5 of its norm (4096 columns; a plain fp32 form by 3e-5 as
// well), by 6e-8 with mean 0.  (Summing the differences as well and correcting the mean by them
// made bf16 rows worse: sums of bf16 values are nearly exact, those of differences are
// not.)  HBM is the bound: 8192 x 4096 bf16 with residual
// and checkpoint 54 us (5.6 TB/s of 9 bytes per element, 0.84 of the measured copy
// rate), without a checkpoint 47 us (0.87).
//
// The forward kernel keeps no column sums and so fits more threads on an SM than the
// block norms' 512: 1024 where a warp or two hold a row, else 768 (us at 512, 768 and 1024
// threads, bf16: 131072 x 128 53, 42, 34; 32768 x 768 with an fp32 residual stream 62, 51,
// 52; 32768 x 1024 63, 56, 56; 8192 x 4096 without residual 35, 26, 25, with it 48, 47,
// 53), but 512 for rows of 2049 to 4096 columns with residual and checkpoint (53, 54, 62)
// or off 16-byte boundaries (8191 x 4095 fp32 57, 76, 70).  fp32 rows off 16-byte
// boundaries of up to 1024 columns take 768 (16001 x 1021 33 us at 512, 28); those of 1025
// to 2048 take them too, although two chunks per thread spill 61 words there (8191 x 2045
// 30 us at 512, 43): open.
template <int T, int MIX, Lay LAY>
constexpr int kFwdBlocks = T >= 512 ? 1 : T == 256 ? (MIX == 1 || LAY != kAligned ? 2 : 3) : T >= 128 ? 768 / T : 1024 / T;

// MIX: 1 y and a checkpoint, 2 y and no checkpoint, 3 neither, 0 decided at run
// time.  FULL: the row has exactly 8 C T columns.

template <class TA, class TR, int T, int C, int MIX, bool FULL, Lay LAY>
__global__ void __launch_bounds__(T, kFwdBlocks<T, MIX, LAY>)
k_layer_norm_fwd_staged(const z1ln::Fwd a, const int stages, const int stage_bytes)
{
    using Ld = Cols<T, LAY>;
    constexpr int A = sizeof(TA), B = sizeof(TR), N = 8 * C * T, kVector = N * 4;
    constexpr int at_x = 0, at_y = Ld::template bytes<B>(N);
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ float red[2][2][16];  // by the row's parity and sum
    const int tid = threadIdx.x;
    const bool res = MIX ? MIX != 3 : a.y != nullptr, r8 = LAY != kLanes && (MIX ? MIX == 1 : a.r8.codes != nullptr);
    unsigned char *kept = smem;  // w, b
    unsigned char *ring = smem + 2 * kVector;
    auto in = [&](int i) { return FULL || Ld::col(i) < a.D; };
    auto fetch = [&](int64_t row, unsigned char *to) {
        if (row < a.rows) {
            const TR *x = static_cast<const TR *>(a.x) + row * a.ld_x;
            const TA *y = static_cast<const TA *>(a.y) + row * a.ld_y;
#pragma unroll
            for (int i = 0; i < C; ++i) {
                if (!in(i)) continue;
                Ld::template copy<B>(to + at_x, i, x, a.D, row * a.ld_x == 0);
                if (res) Ld::template copy<A>(to + at_y, i, y, a.D, row * a.ld_y == 0);
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    wait_prior_grid();
    let_next_grid_start();
    for (int k = 0; k + 1 < stages; ++k) fetch(blockIdx.x + (int64_t)k * gridDim.x, ring + k * stage_bytes);
    keep_or<T, C, LAY>(kept, a.w, a.pf32, a.D, 1.f);
    keep_or<T, C, LAY>(kept + kVector, a.b, a.pf32, a.D, 0.f);

    int st = 0, flip = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        // what this thread has read a row ago is filled again
        fetch(row + (int64_t)(stages - 1) * gridDim.x, ring + (st == 0 ? stages - 1 : st - 1) * stage_bytes);
        copies_wait(stages - 1);
        const unsigned char *p = ring + st * stage_bytes;
        V8 v[C];
        float s = 0.f;
        TR *r = static_cast<TR *>(a.r) + row * a.ld_r;
#pragma unroll
        for (int i = 0; i < C; ++i) {
            v[i] = splat8(0.f);
            if (!in(i)) continue;
            v[i] = Ld::take(p + at_x, i, static_cast<const TR *>(a.x) + row * a.ld_x);
            if (res) {
                v[i] = fma8(Ld::take(p + at_y, i, static_cast<const TA *>(a.y) + row * a.ld_y), a.alpha, v[i]);
                Ld::put(r, i, a.D, v[i]);
            }
            s += sum8(v[i]);
        }
        const float mean = mean_of(block_sum<T>(s, red[flip][0]), a);
        s = 0.f;
#pragma unroll
        for (int i = 0; i < C; ++i) {
            if (!in(i)) continue;
            v[i] = plus8(v[i], -mean);
            v[i] = Ld::inside(v[i], i, a.D);
            s += dot8(v[i], v[i]);
        }
        const float rstd = rsqrtf(fmaf(block_sum<T>(s, red[flip][1]), a.inv_d, a.eps));
        if (tid == 0) {
            a.mean[row] = mean;
            a.rstd[row] = rstd;
        }
        TA *h = static_cast<TA *>(a.h) + row * a.ld_h;
#pragma unroll
        for (int i = 0; i < C; ++i) {
            v[i] = mul8(v[i], rstd);
            if (r8) {
                const int col = Ld::col(i);
                int E;
                const uint2 q = encode8(v[i], E);
                if (FULL || col / kQBlock * kQBlock < a.D) {
                    __stcs(reinterpret_cast<uint2 *>(a.r8.codes + row * a.r8.ld_codes + col), q);
                    if ((tid & 15) == 0) a.r8.exps[(int64_t)(col / kQBlock) * a.r8.ld_exps + row] = (uint8_t)E;
                }
            }
            if (in(i)) Ld::put(h, i, a.D, fma8(v[i], kept8<T, C>(kept, i), kept8<T, C>(kept + kVector, i)));
        }
        flip ^= 1;
        if (++st == stages) st = 0;
    }
}

// The direct kernel, for rows that do not fit the ring (above 8192 columns): a
// block's threads hold 16 elements of a row each, and nothing of the next row is under way
// while its two sums are taken (bf16 with residual and checkpoint, 2048 x 16384 78 us, its
// bytes 45; 2048 x 12288 65 of 34; fp32 with residual, 2048 x 16384 92 of 80).
template <class TA, class TR, bool VEC>
__global__ void __launch_bounds__(1024) k_layer_norm_fwd(const z1ln::Fwd a)
{
    constexpr int C = 2;
    __shared__ float red[2][2][32];
    const int tid = threadIdx.x, nthr = blockDim.x;
    int flip = 0;
    wait_prior_grid();
    let_next_grid_start();
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, flip ^= 1) {
        Chunk<TR, VEC> xq[C];
        Chunk<TA, VEC> yq[C];
#pragma unroll
        for (int i = 0; i < C; ++i) xq[i].load(static_cast<const TR *>(a.x) + row * a.ld_x, chunk_col<VEC>(i, tid, nthr), a.D);
        if (a.y) {
#pragma unroll
            for (int i = 0; i < C; ++i) yq[i].load(static_cast<const TA *>(a.y) + row * a.ld_y, chunk_col<VEC>(i, tid, nthr), a.D);
        }
        float f[C][8], s = 0.f;
#pragma unroll
        for (int i = 0; i < C; ++i) {
            xq[i].get(f[i]);
            if (a.y) {
                float y[8];
                yq[i].get(y);
#pragma unroll
                for (int k = 0; k < 8; ++k) f[i][k] = fmaf(a.alpha, y[k], f[i][k]);
                store_chunk<TR, VEC>(static_cast<TR *>(a.r) + row * a.ld_r, chunk_col<VEC>(i, tid, nthr), a.D, f[i]);
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) s += f[i][k];
        }
        const float mean = mean_of(row_sum(s, red[flip][0]), a);
        s = 0.f;
#pragma unroll
        for (int i = 0; i < C; ++i)
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                f[i][k] = chunk_col<VEC>(i, tid, nthr) + kStep<VEC> * k < a.D ? f[i][k] - mean : 0.f;
                s = fmaf(f[i][k], f[i][k], s);
            }
        const float rstd = rsqrtf(fmaf(row_sum(s, red[flip][1]), a.inv_d, a.eps));
        if (tid == 0) {
            a.mean[row] = mean;
            a.rstd[row] = rstd;
        }
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const int col = chunk_col<VEC>(i, tid, nthr);
#pragma unroll
            for (int k = 0; k < 8; ++k) f[i][k] *= rstd;
            if (a.r8.codes) pack_chunk<VEC>(a.r8, row, col, a.D, f[i]);
            float w[8], b[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) { w[k] = 1.f; b[k] = 0.f; }
            const int wide = (((uintptr_t)a.w | (uintptr_t)a.b) & 15) == 0;
            if (a.w) param8<VEC>(a.w, a.pf32, wide, 0, col, a.D, w);
            if (a.b) param8<VEC>(a.b, a.pf32, wide, 0, col, a.D, b);
#pragma unroll
            for (int k = 0; k < 8; ++k) f[i][k] = fmaf(f[i][k], w[k], b[k]);
            store_chunk<TA, VEC>(static_cast<TA *>(a.h) + row * a.ld_h, col, a.D, f[i]);
        }
    }
}

// ------------------------------------------------------------ backward -----
//
//   t = w dh;  d = dr + rstd (t - mean(t) - rh mean(t rh));  dx = d;  dy = a d
//   dw = sum over rows of dh rh;  db = sum over rows of dh
//
// One pass: both means of a row come from one barrier, and a thread keeps the
// column sums of its own columns over all rows that its block visits; a second
// kernel adds the blocks' sums in block order.  8192 x 4096 bf16 from the checkpoint 53
// us (5.7 TB/s of 9 bytes per element, 0.85 of the measured copy rate), of which the
// column sums and their joining take 5; with the partial sums stored a word at a time
// 60.
//
// MIX: 1 dr and a checkpoint, 2 dr and the tensor r, 3 no dr and the tensor, 0
// decided at run time.

// A row's statistics and scale bytes travel through the ring as well: each warp
// has 16 words per stage, mean, rstd, and from word 4 on the aligned words around
// the scale bytes of its 128-column blocks, two per chunk.  This lane copies word
// `lane`.
template <int T, int C>
struct LnWords {
    const char *from = nullptr;
    int bytes_per_row = 1;

    __device__ __forceinline__ explicit LnWords(const z1ln::Bwd &a)
    {
        const int lane = threadIdx.x & 31, k = lane - 4;
        if (lane < 2) {
            from = reinterpret_cast<const char *>(lane == 0 ? a.mean : a.rstd);
            bytes_per_row = 4;
        } else if (k >= 0 && k < 2 * C && a.r8.codes) {
            const int col = (threadIdx.x / 32 * 32 + (k % 2) * 16) * 8 + k / 2 * T * 8;
            if (col < a.D) from = reinterpret_cast<const char *>(a.r8.exps + (int64_t)(col / kQBlock) * a.r8.ld_exps);
        }
    }
    __device__ __forceinline__ void copy_ahead(uint32_t *words, int64_t row) const
    {
        if (!from) return;
        const uint32_t d = (uint32_t)__cvta_generic_to_shared(words + (threadIdx.x & 31));
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(d), "l"(from + ((row * bytes_per_row) & ~INT64_C(3)))
                     : "memory");
    }
    static __device__ __forceinline__ float scale(const uint32_t *words, int64_t row, int i)
    {
        const uint32_t w = words[4 + 2 * i + (threadIdx.x >> 4 & 1)];
        return scale_of((w >> (8 * ((int)row & 3))) & 255);
    }
};

template <class TA, class TR, int T, int C, int MIX, Lay LAY>
struct LnStage {
    using Ld = Cols<T, LAY>;
    static constexpr int n = 8 * C * T;
    static constexpr int A = Ld::template bytes<sizeof(TA)>(n), B = Ld::template bytes<sizeof(TR)>(n);
    static constexpr int dh = 0, dr = dh + A, r = dr + (MIX == 3 ? 0 : B), words = r + (MIX == 1 ? n : B);
    static constexpr int words_bytes = 64;  // of a warp
    static constexpr int bytes = words + T / 32 * words_bytes;
};

template <class TA, class TR, int T, int C, int MIX, bool FULL, Lay LAY>
__global__ void __launch_bounds__(T, kOwnRegs / T)
k_layer_norm_bwd_staged(const z1ln::Bwd a, const int stages)
{
    using S = LnStage<TA, TR, T, C, MIX, LAY>;
    using Ld = Cols<T, LAY>;
    constexpr int A = sizeof(TA), B = sizeof(TR), kVector = S::n * 4;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ float2 red[2][16];
    const int tid = threadIdx.x;
    const bool has_dr = MIX ? MIX != 3 : a.dr != nullptr, r8 = LAY != kLanes && (MIX ? MIX == 1 : a.r8.codes != nullptr);
    unsigned char *kept = smem, *ring = smem + kVector;
    auto in = [&](int i) { return FULL || Ld::col(i) < a.D; };
    const LnWords<T, C> row_words(a);
    auto words_of = [&](unsigned char *stage) { return reinterpret_cast<uint32_t *>(stage + S::words + tid / 32 * S::words_bytes); };

    // Starts the copies of a row; past the last row, an empty group that keeps the count.
    auto fetch = [&](int64_t row, unsigned char *to) {
        if (row < a.rows) {
            row_words.copy_ahead(words_of(to), row);
            const TA *dh = static_cast<const TA *>(a.dh) + row * a.ld_dh;
            const TR *dr = static_cast<const TR *>(a.dr) + row * a.ld_dr;
            const void *r = r8 ? (const void *)(a.r8.codes + row * a.r8.ld_codes) : (const void *)(static_cast<const TR *>(a.r) + row * a.ld_r);
#pragma unroll
            for (int i = 0; i < C; ++i) {
                if (!in(i)) continue;
                Ld::template copy<A>(to + S::dh, i, dh, a.D, row * a.ld_dh == 0);
                if (r8) copy8_ahead<1>(to + S::r + chunk_at<T, 1>(i), r, Ld::col(i));
                else Ld::template copy<B>(to + S::r, i, r, a.D, row * a.ld_r == 0);
                if (has_dr) Ld::template copy<B>(to + S::dr, i, dr, a.D, row * a.ld_dr == 0);
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    wait_prior_grid();
    let_next_grid_start();
    for (int k = 0; k + 1 < stages; ++k) fetch(blockIdx.x + (int64_t)k * gridDim.x, ring + k * S::bytes);
    keep_or<T, C, LAY>(kept, a.w, a.pf32, a.D, 1.f);
    V8 acc_w[C], acc_b[C];
#pragma unroll
    for (int i = 0; i < C; ++i) acc_w[i] = acc_b[i] = splat8(0.f);

    int st = 0, flip = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        // the stage that this warp has read a row ago is filled again
        __syncwarp();
        fetch(row + (int64_t)(stages - 1) * gridDim.x, ring + (st == 0 ? stages - 1 : st - 1) * S::bytes);
        copies_wait(stages - 1);
        __syncwarp();
        unsigned char *p = ring + st * S::bytes;
        const uint32_t *words = words_of(p);
        const float mean = __uint_as_float(words[0]), rstd = __uint_as_float(words[1]);
        V8 d[C], h[C];
        float s = 0.f, t = 0.f;
#pragma unroll
        for (int i = 0; i < C; ++i) {
            if (!in(i)) continue;
            d[i] = Ld::take(p + S::dh, i, static_cast<const TA *>(a.dh) + row * a.ld_dh);
            if (r8) h[i] = take_codes(p + S::r + chunk_at<T, 1>(i), row_words.scale(words, row, i));
            else h[i] = mul8(plus8(Ld::take(p + S::r, i, static_cast<const TR *>(a.r) + row * a.ld_r), -mean), rstd);
            h[i] = Ld::inside(h[i], i, a.D);
            acc_w[i] = fma8(d[i], h[i], acc_w[i]);
            acc_b[i] = add8(acc_b[i], d[i]);
            d[i] = mul8(d[i], kept8<T, C>(kept, i));
            s += sum8(d[i]);
            t += dot8(d[i], h[i]);
        }
        const float2 m = block_sum2<T>(s, t, red[flip]);
        s = m.x * -a.inv_d;
        t = m.y * -a.inv_d;
        TR *dx = static_cast<TR *>(a.dx) + row * a.ld_dx;
        TA *dy = static_cast<TA *>(a.dy) + row * a.ld_dy;
#pragma unroll
        for (int i = 0; i < C; ++i) {
            if (!in(i)) continue;
            const V8 x = plus8(fma8(h[i], t, d[i]), s);
            if (has_dr) d[i] = fma8(x, rstd, Ld::take(p + S::dr, i, static_cast<const TR *>(a.dr) + row * a.ld_dr));
            else d[i] = mul8(x, rstd);
            Ld::put(dx, i, a.D, d[i]);
            if (a.dy) Ld::put(dy, i, a.D, mul8(d[i], a.alpha));
        }
        flip ^= 1;
        if (++st == stages) st = 0;
    }
    float *part = a.part + (int64_t)blockIdx.x * a.ld_part;
    const int64_t plane = (int64_t)gridDim.x * a.ld_part;
    auto put = [&](float *p, int i, const V8 &v) {
        if constexpr (LAY == kLanes) {
            Ld::put(p, i, a.D, v);
        } else {
            const float2 x = split(v.p[0]), y = split(v.p[1]), z = split(v.p[2]), w = split(v.p[3]);
            float4 *q = reinterpret_cast<float4 *>(p + Ld::col(i));
            q[0] = make_float4(x.x, x.y, y.x, y.y);
            q[1] = make_float4(z.x, z.y, w.x, w.y);
        }
    };
#pragma unroll
    for (int i = 0; i < C; ++i) {
        if (!in(i)) continue;
        if (a.need_w) put(part, i, acc_w[i]);
        if (a.need_b) put(part + plane, i, acc_b[i]);
    }
}

// The direct kernel, for rows that do not fit the ring: above 8192 columns, and fp32 rows
// of 1025 to 2048 and of 4097 to 8192, whose two stages, with room for dr, miss a block's
// share of shared memory by 1024 and by 256 bytes.  A row of more than 8192 columns takes
// 1024 threads, whose column sums are in shared memory (SACC) and whose 64 registers spill
// (bf16 30 words, fp32 72).  bf16 from the checkpoint, 2048 x 16384 139 us, its bytes 45;
// 2048 x 12288 123 of 34; fp32 from r, 8192 x 2048 70 of 50, 4096 x 8192 160 of 100.
template <class TA, class TR, bool VEC, bool SACC>
__global__ void __launch_bounds__(SACC ? 1024 : 512) k_layer_norm_bwd(const z1ln::Bwd a)
{
    constexpr int C = 2, V = 8 * C;
    __shared__ float red[2][2][32];
    extern __shared__ float sacc[];  // SACC: [2][V][threads]
    const int tid = threadIdx.x, nthr = blockDim.x;
    float acc[SACC ? 1 : 2][C][8];
    if constexpr (SACC) {
        for (int q = 0; q < 2 * V; ++q) sacc[q * nthr + tid] = 0.f;
    } else {
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int i = 0; i < C; ++i)
#pragma unroll
                for (int k = 0; k < 8; ++k) acc[s][i][k] = 0.f;
    }
    auto add = [&](int s, int i, int k, float x) {
        if constexpr (SACC) sacc[(s * V + i * 8 + k) * nthr + tid] += x;
        else acc[s][i][k] += x;
    };
    int flip = 0;
    wait_prior_grid();
    let_next_grid_start();
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, flip ^= 1) {
        Chunk<TA, VEC> hq[C];
        Chunk<TR, VEC> rq[C], dq[SACC ? 1 : C];
        uint2 q8[C];
        int e8[C];
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const int col = chunk_col<VEC>(i, tid, nthr);
            hq[i].load(static_cast<const TA *>(a.dh) + row * a.ld_dh, col, a.D);
            if (a.r8.codes) load_codes<VEC>(a.r8, row, col, a.D, q8[i], e8[i]);
            else rq[i].load(static_cast<const TR *>(a.r) + row * a.ld_r, col, a.D);
            if (!SACC && a.dr) dq[i].load(static_cast<const TR *>(a.dr) + row * a.ld_dr, col, a.D);
        }
        const float mean = a.mean[row], rstd = a.rstd[row];
        float d[C][8], h[C][8], s = 0.f, t = 0.f;
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const int col = chunk_col<VEC>(i, tid, nthr);
            hq[i].get(d[i]);
            if (a.r8.codes) {
                values8(q8[i], scale_of(e8[i]), h[i]);
            } else {
                rq[i].get(h[i]);
#pragma unroll
                for (int k = 0; k < 8; ++k) h[i][k] = (h[i][k] - mean) * rstd;
            }
            float w[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) w[k] = 1.f;
            if (a.w) param8<VEC>(a.w, a.pf32, ((uintptr_t)a.w & 15) == 0, 0, col, a.D, w);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                if (col + kStep<VEC> * k >= a.D) h[i][k] = 0.f;
                if (a.need_w) add(0, i, k, d[i][k] * h[i][k]);
                if (a.need_b) add(1, i, k, d[i][k]);
                d[i][k] *= w[k];
                s += d[i][k];
                t = fmaf(d[i][k], h[i][k], t);
            }
        }
        s = row_sum(s, red[flip][0]) * a.inv_d;
        t = row_sum(t, red[flip][1]) * a.inv_d;
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const int col = chunk_col<VEC>(i, tid, nthr);
            float r0[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) r0[k] = 0.f;
            if (SACC && a.dr) dq[0].load(static_cast<const TR *>(a.dr) + row * a.ld_dr, col, a.D);  // (registers are short)
            if (a.dr) dq[SACC ? 0 : i].get(r0);
#pragma unroll
            for (int k = 0; k < 8; ++k) d[i][k] = fmaf(rstd, fmaf(-h[i][k], t, d[i][k]) - s, r0[k]);
            store_chunk<TR, VEC>(static_cast<TR *>(a.dx) + row * a.ld_dx, col, a.D, d[i]);
            if (a.dy) {
#pragma unroll
                for (int k = 0; k < 8; ++k) d[i][k] *= a.alpha;
                store_chunk<TA, VEC>(static_cast<TA *>(a.dy) + row * a.ld_dy, col, a.D, d[i]);
            }
        }
    }
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        if (!(s == 0 ? a.need_w : a.need_b)) continue;
        float *part = a.part + ((int64_t)s * gridDim.x + blockIdx.x) * a.ld_part;
#pragma unroll
        for (int i = 0; i < C; ++i)
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int c = chunk_col<VEC>(i, tid, nthr) + kStep<VEC> * k;
                if (c < a.D) part[c] = SACC ? sacc[(s * V + i * 8 + k) * nthr + tid] : acc[SACC ? 0 : s][i][k];
            }
    }
}

// -------------------------------------------------------------- launch -----

template <class TA, class TR, int T, int C, int MIX, bool FULL, Lay LAY>
bool ln_fwd_staged(const z1ln::Fwd &a, int sms, cudaStream_t st, int *rc)
{
    auto kernel = k_layer_norm_fwd_staged<TA, TR, T, C, MIX, FULL, LAY>;
    using Ld = Cols<T, LAY>;
    constexpr int N = 8 * C * T, kept = 2 * N * 4;
    const int stage = Ld::template bytes<sizeof(TR)>(N) + (a.y ? Ld::template bytes<sizeof(TA)>(N) : 0);
    int blocks = kFwdBlocks<T, MIX, LAY>, stages = 0;
    for (;; --blocks) {  // fewer where so many rings do not fit
        stages = (kSmemPerSm / blocks - 1280 - kept) / stage;
        if (stages >= 2 || blocks <= kOwnRegs / T) break;
    }
    if (stages < 2) return false;
    stages = stages < 4 ? stages : 4;
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = allow_smem(kernel, kSmemPerSm - 1024, done);
    if (e != cudaSuccess) {
        *rc = z1_fail(ZERO1_ECUDA, "layer norm forward: %s", cudaGetErrorString(e));
        return true;
    }
    const int64_t wave = (int64_t)sms * blocks, grid = a.rows < wave ? a.rows : wave;
    const cudaError_t le = launch_after(kernel, dim3((unsigned)grid), T, kept + stages * stage, st, a, stages, stage);
    z1_note_launch(reinterpret_cast<const void *>(kernel), (int)grid, blocks, T, 0);
    *rc = le == cudaSuccess ? ZERO1_OK : pdl_fail(le, "layer norm forward launch");
    return true;
}

template <class TA, class TR>
bool ln_forward_staged(const z1ln::Fwd &a, bool vec, int sms, cudaStream_t st, int *rc)
{
    if (a.D > 8192) return false;
    const int mix = a.y ? (a.r8.codes ? 1 : 2) : (a.r8.codes ? 0 : 3);
    return pick_threads(a.D, [&](auto t, auto n) {
        constexpr int T = decltype(t)::value, C = decltype(n)::value;
        if constexpr (sizeof(TA) == 4) {
            if (!vec && !a.r8.codes) return ln_fwd_staged<TA, TR, T, C, 0, false, kLanes>(a, sms, st, rc);
        }
        if (!vec) return ln_fwd_staged<TA, TR, T, C, 0, false, kAnywhere>(a, sms, st, rc);
        if constexpr (sizeof(TA) == 2 && !(T == 512 && C == 1)) {
            const int m = a.D == 8 * C * T ? mix : 0;
            if (m == 1) return ln_fwd_staged<TA, TR, T, C, 1, true, kAligned>(a, sms, st, rc);
            if (m == 2) return ln_fwd_staged<TA, TR, T, C, 2, true, kAligned>(a, sms, st, rc);
            if (m == 3) return ln_fwd_staged<TA, TR, T, C, 3, true, kAligned>(a, sms, st, rc);
        }
        return ln_fwd_staged<TA, TR, T, C, 0, false, kAligned>(a, sms, st, rc);
    });
}

template <class TA, class TR, bool VEC>
int ln_fwd_direct(const z1ln::Fwd &a, int sms, cudaStream_t st)
{
    auto kernel = k_layer_norm_fwd<TA, TR, VEC>;
    const int threads = row_threads(a.D), per_sm = blocks_per_sm(reinterpret_cast<const void *>(kernel), threads);
    const int64_t grid = a.rows < (int64_t)sms * per_sm ? a.rows : (int64_t)sms * per_sm;
    const cudaError_t le = launch_after(kernel, dim3((unsigned)grid), threads, 0, st, a);
    z1_note_launch(reinterpret_cast<const void *>(kernel), (int)grid, per_sm, threads, 0);
    return le == cudaSuccess ? ZERO1_OK : pdl_fail(le, "layer norm forward launch");
}

template <class TA, class TR, int T, int C, int MIX, bool FULL, Lay LAY>
bool ln_bwd_staged(const z1ln::Bwd &a, int64_t grid, cudaStream_t st, int *rc)
{
    auto kernel = k_layer_norm_bwd_staged<TA, TR, T, C, MIX, FULL, LAY>;
    using S = LnStage<TA, TR, T, C, MIX, LAY>;
    const int stages = stages_that_fit(T, S::n * 4, S::bytes);
    if (stages == 0) return false;
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = allow_smem(kernel, kSmemPerSm - 1024, done);
    if (e != cudaSuccess) {
        *rc = z1_fail(ZERO1_ECUDA, "layer norm backward: %s", cudaGetErrorString(e));
        return true;
    }
    const cudaError_t le = launch_after(kernel, dim3((unsigned)grid), T, S::n * 4 + stages * S::bytes, st, a, stages);
    z1_note_launch(reinterpret_cast<const void *>(kernel), (int)grid, kOwnRegs / T, T, 0);
    *rc = le == cudaSuccess ? ZERO1_OK : pdl_fail(le, "layer norm backward launch");
    return true;
}

template <class TA, class TR>
bool ln_backward_staged(const z1ln::Bwd &a, bool vec, int64_t grid, cudaStream_t st, int *rc)
{
    if (a.D > 8192) return false;
    const int mix = a.dr ? (a.r8.codes ? 1 : 2) : (a.r8.codes ? 0 : 3);
    return pick_threads(a.D, [&](auto t, auto n) {
        constexpr int T = decltype(t)::value, C = decltype(n)::value;
        if constexpr (sizeof(TA) == 4) {
            if (!vec && !a.r8.codes) return ln_bwd_staged<TA, TR, T, C, 0, false, kLanes>(a, grid, st, rc);
        }
        if (!vec) return ln_bwd_staged<TA, TR, T, C, 0, false, kAnywhere>(a, grid, st, rc);
        if constexpr (sizeof(TA) == 2 && !(T == 512 && C == 1)) {
            const int m = a.D == 8 * C * T ? mix : 0;
            if (m == 1) return ln_bwd_staged<TA, TR, T, C, 1, true, kAligned>(a, grid, st, rc);
            if (m == 2) return ln_bwd_staged<TA, TR, T, C, 2, true, kAligned>(a, grid, st, rc);
            if (m == 3) return ln_bwd_staged<TA, TR, T, C, 3, true, kAligned>(a, grid, st, rc);
        }
        return ln_bwd_staged<TA, TR, T, C, 0, false, kAligned>(a, grid, st, rc);
    });
}

template <class TA, class TR, bool VEC, bool SACC>
int ln_bwd_direct(const z1ln::Bwd &a, int64_t grid, cudaStream_t st)
{
    auto kernel = k_layer_norm_bwd<TA, TR, VEC, SACC>;
    const int threads = row_threads(a.D), smem = SACC ? 2 * 16 * threads * 4 : 0;
    if (SACC) {
        static std::atomic<uint64_t> done{0};
        const cudaError_t e = allow_smem(kernel, 2 * 16 * 1024 * 4, done);
        if (e != cudaSuccess) return z1_fail(ZERO1_ECUDA, "layer norm backward: %s", cudaGetErrorString(e));
    }
    const cudaError_t le = launch_after(kernel, dim3((unsigned)grid), threads, smem, st, a);
    z1_note_launch(reinterpret_cast<const void *>(kernel), (int)grid, 1, threads, 0);
    return le == cudaSuccess ? ZERO1_OK : pdl_fail(le, "layer norm backward launch");
}

}  // namespace

template <class TA, class TR>
int z1ln::run_forward(const Fwd &a, bool vec, int sms, cudaStream_t st)
{
    int rc;
    if (ln_forward_staged<TA, TR>(a, vec, sms, st, &rc)) return rc;
    return vec ? ln_fwd_direct<TA, TR, true>(a, sms, st) : ln_fwd_direct<TA, TR, false>(a, sms, st);
}

template <class TA, class TR>
int z1ln::run_backward(const Bwd &a, bool vec, int64_t grid, cudaStream_t st)
{
    int rc;
    if (ln_backward_staged<TA, TR>(a, vec, grid, st, &rc)) return rc;
    if (a.D <= 8192) return vec ? ln_bwd_direct<TA, TR, true, false>(a, grid, st) : ln_bwd_direct<TA, TR, false, false>(a, grid, st);
    return vec ? ln_bwd_direct<TA, TR, true, true>(a, grid, st) : ln_bwd_direct<TA, TR, false, true>(a, grid, st);
}
