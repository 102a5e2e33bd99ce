// zero1_block_norm.cuh - what the block norms' sources share: their arguments,
// the row geometry, and the ring that feeds a row through shared memory
// (library-internal).
#pragma once

#include "zero1_block.cuh"

// The kernels are compiled per pair of types (activations, residual stream),
// forward and backward apart, so that the sources build in parallel.
namespace z1bn {

// The arguments that both directions share.
struct Common {
    int64_t rows;
    int D;
    float eps, alpha, inv_d;
    int gate_kind, sigmoid;
    int pf32, gf32, wf32;  // fp32 weights, fp32 gate, fp32 weight gradients
    int pvec, gvec;        // weights (and a channel gate); the [rows, D] gate: vector loads
    const void *w_post, *w_pre, *gate;
    int64_t ld_gate;
    Ckpt y8, r8;  // codes NULL: absent
};

struct Fwd {
    const void *y, *x;
    void *r, *h;
    float *rstd_post, *rstd_pre;
    int64_t ld_y, ld_x, ld_r, ld_h;
};

struct Bwd {
    const void *dh, *dr, *y, *r;
    const float *rstd_post, *rstd_pre;
    void *dy, *dx, *dgate;
    int64_t ld_dh, ld_dr, ld_y, ld_r, ld_dy, ld_dx, ld_dgate;
    int need_post, need_pre, need_gate;  // column sums and gate gradients wanted
    int dgvec;
    float *part;  // [3][blocks][D]: partial column sums (dw_post, dw_pre, dgate)
};

// Launch for one pair of types; vec: every row can be read and written in
// 128-bit accesses.  The backward call returns its number of blocks, which is
// that of the partial column sums.
template <class TA, class TR>
int run_forward(const Common &c, const Fwd &a, bool vec, int sms, cudaStream_t st);
template <class TA, class TR>
int run_backward(const Common &c, const Bwd &a, bool vec, int64_t grid, cudaStream_t st);

}  // namespace z1bn

namespace {

using z1bn::Bwd;
using z1bn::Common;
using z1bn::Fwd;

constexpr int kMaxCols = ZERO1_BLOCK_NORM_MAX_COLS;

// Threads of a block of the direct kernels for D columns, 16 each.
int row_threads(int64_t D) { return (int)round_up(D, 512) / 16; }

// Blocks of the backward kernel for `rows` rows: one resident wave of the
// staged kernel at most (the per-element kernels use the same number).
int64_t bwd_blocks(int64_t rows, int64_t D, int sms)
{
    const int64_t per_sm = D <= 256 ? 16 : D <= 512 ? 8 : D <= 2048 ? 4 : D <= 4096 ? 2 : 1;
    return rows < per_sm * sms ? rows : per_sm * sms;
}

// ---------------------------------------------------------- row geometry ---
//
// A row is shared out over a block in chunks of 8 elements per thread.  Here,
// for the direct kernels, a chunk is 8 consecutive columns on the vector path;
// otherwise its elements are 16 columns apart.  Either way 16 neighbouring
// lanes hold one 128-column checkpoint block per chunk.

template <bool VEC>
__device__ __forceinline__ int chunk_col(int i, int tid, int nthr)
{
    const int v = i * nthr + tid;
    return VEC ? v * 8 : v / 16 * kQBlock + v % 16;
}

template <bool VEC>
constexpr int kStep = VEC ? 1 : 16;

// Eight elements of a row: loaded early as they lie in memory, converted when
// they are used.
template <class T, bool VEC>
struct Chunk {
    Raw8<T> q;
    __device__ __forceinline__ void load(const T *row, int col, int D)
    {
        if (col < D) q.load(row + col);
        else q.zero();
    }
    __device__ __forceinline__ void get(float f[8]) const { q.get(f); }
};
template <class T>
struct Chunk<T, false> {
    T e[8];
    __device__ __forceinline__ void load(const T *row, int col, int D)
    {
#pragma unroll
        for (int k = 0; k < 8; ++k) e[k] = col + 16 * k < D ? row[col + 16 * k] : (T)0;
    }
    __device__ __forceinline__ void get(float f[8]) const
    {
#pragma unroll
        for (int k = 0; k < 8; ++k) f[k] = ld1(&e[k]);
    }
};

template <class T, bool VEC>
__device__ __forceinline__ void store_chunk(T *row, int col, int D, const float f[8])
{
    if constexpr (VEC) {
        if (col < D) store8(row + col, f);
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (col + 16 * k < D) st1(row + col + 16 * k, f[k]);
    }
}

// Eight weights or gate values of run-time type (1 beyond the row's end, so
// that nothing there turns into a NaN).  vec: in 128-bit loads, if all eight lie
// below column D or all beyond.
template <bool VEC>
__device__ __forceinline__ void param8(const void *p, int f32, int vec, int64_t base, int col, int D, float f[8])
{
    if (VEC && vec) {
        if (col < D) {
            if (f32) {
                const float4 *q = reinterpret_cast<const float4 *>(static_cast<const float *>(p) + base + col);
                const float4 a = __ldg(q), b = __ldg(q + 1);
                f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w; f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
            } else {
                unpack8(__ldg(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p) + base + col)), f);
            }
            return;
        }
    } else {
        // (the type is looked at once, so that the eight loads are under way together)
        if (f32) {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int c = col + kStep<VEC> * k;
                f[k] = c < D ? __ldg(static_cast<const float *>(p) + base + c) : 1.f;
            }
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int c = col + kStep<VEC> * k;
                f[k] = c < D ? bf_one(__ldg(static_cast<const uint16_t *>(p) + base + c)) : 1.f;
            }
        }
        return;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) f[k] = 1.f;
}

__device__ __forceinline__ float warp_sum(float x)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// The sum over a row, the same in every thread.  One barrier per call: between
// two calls with the same `red` buffer every warp passes another call's
// barrier, so the kernels alternate by sum and by row (a row may have one sum
// only).
__device__ __forceinline__ float row_sum(float x, float *red)
{
    const int lane = threadIdx.x & 31;
    x = warp_sum(x);
    if (lane == 0) red[threadIdx.x >> 5] = x;
    __syncthreads();
    return warp_sum(lane < (int)(blockDim.x >> 5) ? red[lane] : 0.f);
}

// exp(-a) for a >= 0 to 2.5 ulps (and through the subnormal numbers, NaN for
// NaN; USUAL: a is at most 87, where the result is a normal number): 2^t by the
// hardware's 2-ulp instruction, t = -a log2(e) rounded, times 1 + r ln 2 for the
// rest r of that product, which a fused multiply-add gives exactly and log2(e)'s
// own lower part completes.  Without r the error grows with a: 100 ulps at 80.
template <bool USUAL = false>
__device__ __forceinline__ float exp_minus(float a)
{
    constexpr float kLog2e = 1.44269502f, kLog2eLow = 1.92596299e-8f, kLn2 = 0.693147182f;
    if (!USUAL) asm("min.NaN.f32 %0, %1, %2;" : "=f"(a) : "f"(a), "f"(200.f));  // an infinity would have no rest
    const float t = __fmul_rn(-a, kLog2e);
    const float r = __fmaf_rn(-a, kLog2eLow, __fmaf_rn(-a, kLog2e, -t));
    float e;
    if (USUAL) asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(t));
    else asm("ex2.approx.f32 %0, %1;" : "=f"(e) : "f"(t));
    return __fmaf_rn(e, __fmul_rn(r, kLn2), e);
}

// s = 1 / (1 + exp(-x)) and its slope s (1 - s), both from e = exp(-|x|) and 1 +
// e, which is between 1 and 2: s = 1 / (1 + e) or e / (1 + e), slope = e / (1 +
// e)^2, within 16 half ulps at every x.  1 - s would lose every bit where s
// rounds to 1.
template <bool USUAL = false>
struct Logistic {
    float s, slope;
    __device__ __forceinline__ explicit Logistic(float x)
    {
        const float e = exp_minus<USUAL>(fabsf(x));
        float q;
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(q) : "f"(1.f + e));  // 1 ulp
        const float t = e * q;
        s = x >= 0.f ? q : t;
        slope = t * q;
    }
};
__device__ __forceinline__ float sigmoid(float x) { return Logistic<>(x).s; }
__device__ __forceinline__ float rstd_of(float ss, const Common &c) { return rsqrtf(fmaf(ss, c.inv_d, c.eps)); }

// Eight gates to their factors or slopes (or both).  Eight of usual size,
// almost always all of them, take the shorter form (16384 x 8192 with a full
// gate: backward 294 us against 298 without it, forward 263 against 266; 292 and
// 257 with __expf and 1 - s).
__device__ __forceinline__ bool usual8(float a, float b, float c, float d, float e, float f, float g, float h)
{
    return max_abs(max_abs(a, b, c), max_abs(d, e, f), max_abs(g, h, 0.f)) <= 87.f;
}
template <bool USUAL>
__device__ __forceinline__ void logistic8_of(V8 &g, V8 &slope)
{
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float2 v = split(g.p[k]);
        const Logistic<USUAL> a(v.x), b(v.y);
        g.p[k] = pair(a.s, b.s);
        slope.p[k] = pair(a.slope, b.slope);
    }
}
__device__ __forceinline__ void logistic8(V8 &g, V8 &slope)
{
    const float2 a = split(g.p[0]), b = split(g.p[1]), c = split(g.p[2]), d = split(g.p[3]);
    if (usual8(a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y)) logistic8_of<true>(g, slope);
    else logistic8_of<false>(g, slope);
}
template <bool SLOPE>
__device__ __forceinline__ void logistic8(float g[8])
{
    if (usual8(g[0], g[1], g[2], g[3], g[4], g[5], g[6], g[7])) {
#pragma unroll
        for (int k = 0; k < 8; ++k) g[k] = SLOPE ? Logistic<true>(g[k]).slope : Logistic<true>(g[k]).s;
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) g[k] = SLOPE ? Logistic<>(g[k]).slope : Logistic<>(g[k]).s;
    }
}

// The gates of a chunk (channel and full gates; else g is left).
template <bool VEC>
__device__ __forceinline__ void raw_gate8(const Common &c, int64_t row, int col, float g[8])
{
    if (c.gate_kind == ZERO1_GATE_CHANNEL) param8<VEC>(c.gate, c.gf32, c.pvec, 0, col, c.D, g);
    else if (c.gate_kind == ZERO1_GATE_FULL) param8<VEC>(c.gate, c.gf32, c.gvec, row * c.ld_gate, col, c.D, g);
}

// Their factors.
template <bool VEC>
__device__ __forceinline__ void gate8(const Common &c, int64_t row, int col, float g[8])
{
    raw_gate8<VEC>(c, row, col, g);
    if (c.sigmoid && c.gate_kind != ZERO1_GATE_TOKEN) logistic8<false>(g);
}

// A token's factor, and its slope.
__device__ __forceinline__ float token_gate(const Common &c, int64_t row, float &slope)
{
    slope = 1.f;
    if (c.gate_kind != ZERO1_GATE_TOKEN) return 1.f;
    const float g = ld_param(c.gate, c.gf32, row * c.ld_gate);
    if (!c.sigmoid) return g;
    const Logistic<> l(g);
    slope = l.slope;
    return l.s;
}
__device__ __forceinline__ float token_gate(const Common &c, int64_t row)
{
    float slope;
    return token_gate(c, row, slope);
}

// Write 8 values of a row into a checkpoint (all 32 lanes take part; values
// beyond the row's end are 0).
template <bool VEC>
__device__ __forceinline__ void pack_chunk(const Ckpt &c, int64_t row, int col, int D, const float f[8])
{
    uint32_t m = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) m = max(m, mag_bits(f[k]));
    const int E = scale_exp(max16(m));
    const float inv = scale_inv(E);
    uint2 q;
    q.x = code4(f[0], f[1], f[2], f[3], inv, E != kNanE);
    q.y = code4(f[4], f[5], f[6], f[7], inv, E != kNanE);
    if (col / kQBlock * kQBlock >= D) return;
    uint8_t *o = c.codes + row * c.ld_codes + col;
    if constexpr (VEC) {
        __stcs(reinterpret_cast<uint2 *>(o), q);
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) o[16 * k] = (uint8_t)((k < 4 ? q.x : q.y) >> (8 * (k & 3)));
    }
    if ((threadIdx.x & 15) == 0) c.exps[(int64_t)(col / kQBlock) * c.ld_exps + row] = (uint8_t)E;
}

template <bool VEC>
__device__ __forceinline__ void load_codes(const Ckpt &c, int64_t row, int col, int D, uint2 &q, int &E)
{
    q = make_uint2(0, 0);
    E = 127;
    if (col >= D) return;
    const uint8_t *p = c.codes + row * c.ld_codes + col;
    if constexpr (VEC) {
        q = __ldcs(reinterpret_cast<const uint2 *>(p));
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (col + 16 * k < D) (k < 4 ? q.x : q.y) |= (uint32_t)p[16 * k] << (8 * (k & 3));
    }
    E = __ldg(c.exps + (int64_t)(col / kQBlock) * c.ld_exps + row);
}

// ----------------------------------------------------------------- ring ----
//
// Rows up to the widths that fit shared memory travel through a ring of shared-memory stages, so that loads
// are in flight through all phases of a row and both of its sums.  A thread
// copies its own columns (cp.async) and reads only those, so the ring needs no
// barrier.  Bulk copies of whole rows were slower: about 12 bytes per cycle and
// SM came in (90 us for the backward pass at 8192 x 4096), however many were in
// flight; so was a slot per thread, whose scattered 16-byte writes took twice
// as long.
//
// What bounds these kernels besides HBM is the number of instructions (a row's
// 8 columns take 200 to 260), so the common mixes of inputs are compiled apart,
// fp32 pairs are used throughout and the weights are kept as fp32 values.  A
// thread owns C chunks of 8 columns; T threads, of up to 128 registers each,
// take a row, and 512 / T blocks share an SM.

constexpr int kOwnRegs = 512;           // threads per SM at 128 registers each
constexpr int kSmemPerSm = 227 * 1024;  // of which each block also takes 1 KB, and 256 bytes for its sums

// Keeps a [D] vector in shared memory as fp32 values, through the logistic
// function if asked: the first four values of each eight, then the last four,
// so that a warp's 16-byte reads touch every bank once.  The eight values that
// reach past column D are read one by one (D need be no multiple of 8): what
// lies behind a vector is not the caller's, and an Inf or NaN kept from there
// would reach the row's sums as 0 * NaN.
template <int T, int C>
__device__ __forceinline__ void keep_vector(unsigned char *kept, const void *src, int f32, int D, int act)
{
    if (!src) return;
    const bool aligned = ((uintptr_t)src & 15) == 0;
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const int col = threadIdx.x * 8 + i * T * 8;
        float f[8];
        param8<true>(src, f32, aligned && col + 8 <= D, 0, col, D, f);
#pragma unroll
        for (int k = 0; k < 8; ++k) f[k] = act ? sigmoid(f[k]) : f[k];
        float4 *q = reinterpret_cast<float4 *>(kept) + i * T + threadIdx.x;
        q[0] = make_float4(f[0], f[1], f[2], f[3]);
        q[C * T] = make_float4(f[4], f[5], f[6], f[7]);
    }
}
template <int T, int C>
__device__ __forceinline__ V8 kept8(const unsigned char *kept, int i)
{
    const float4 *q = reinterpret_cast<const float4 *>(kept) + i * T + threadIdx.x;
    const float4 a = q[0], b = q[C * T];
    return V8{{pair(a.x, a.y), pair(a.z, a.w), pair(b.x, b.y), pair(b.z, b.w)}};
}

// Starts copying eight elements (of 1, 2 or 4 bytes) into a stage.
template <int BYTES>
__device__ __forceinline__ void copy8_ahead(unsigned char *dst, const void *row, int col)
{
    const uint32_t d = (uint32_t)__cvta_generic_to_shared(dst);
    const char *src = static_cast<const char *>(row) + (uint32_t)(col * BYTES);
    if constexpr (BYTES == 1) asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(d), "l"(src) : "memory");
    else asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(d), "l"(src) : "memory");
    if constexpr (BYTES == 4) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(d + 16), "l"(src + 16) : "memory");
}

// The same for rows at any element offset, a 4-byte word at a time: the words
// that hold the thread's eight elements (five for bf16, whose first element
// may be the upper half of a word) go to a slot of an odd number of words.
// Elements from column D on arrive as zeros.  `first`: nothing of the matrix
// lies before this row.
template <int BYTES>
constexpr int kSlot = BYTES == 2 ? 20 : 36;

template <int BYTES>
__device__ __forceinline__ void copy8_words(unsigned char *dst, const void *row, int col, int D, bool first)
{
    const uint32_t d = (uint32_t)__cvta_generic_to_shared(dst);
    const char *src = static_cast<const char *>(row) + (uint32_t)(col * BYTES);
    const int phase = BYTES == 2 ? (int)((uintptr_t)src & 2) : 0;
    int left = (D - col) * BYTES + phase;  // bytes from the first word to the row's end
    src -= phase;
#pragma unroll
    for (int j = 0; j < (BYTES == 2 ? 5 : 8); ++j, left -= 4) {
        if (BYTES == 2 && j == 0 && phase && first && col == 0) {  // the word's lower half is before the matrix
            reinterpret_cast<uint16_t *>(dst)[1] = *reinterpret_cast<const uint16_t *>(src + 2);
            continue;
        }
        const int n = left >= 4 ? 4 : left > 0 ? left : 0;
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(d + 4 * j), "l"(n ? src + 4 * j : src), "r"(n) : "memory");
    }
}

// Eight elements of such a slot; `row` is where the row lies in memory.
template <class T>
__device__ __forceinline__ V8 take8_words(const unsigned char *slot, const void *row)
{
    const uint32_t *w = reinterpret_cast<const uint32_t *>(slot);
    if constexpr (sizeof(T) == 2) {
        const int shift = ((uintptr_t)row & 2) ? 16 : 0;
        return from_bf16(make_uint4(__funnelshift_r(w[0], w[1], shift), __funnelshift_r(w[1], w[2], shift),
                                    __funnelshift_r(w[2], w[3], shift), __funnelshift_r(w[3], w[4], shift)));
    } else {
        const float *f = reinterpret_cast<const float *>(slot);
        return V8{{pair(f[0], f[1]), pair(f[2], f[3]), pair(f[4], f[5]), pair(f[6], f[7])}};
    }
}

// The values below column D, zeros beyond.
__device__ __forceinline__ V8 below(const V8 &v, int col, int D)
{
    if (col + 8 <= D) return v;
    V8 r;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float2 f = split(v.p[k]);
        r.p[k] = pair(col + 2 * k < D ? f.x : 0.f, col + 2 * k + 1 < D ? f.y : 0.f);
    }
    return r;
}

// The ring's accesses to a row of E-byte elements, N columns in all; AL: in
// 128-bit accesses, else at any offset.
template <int T, bool AL>
struct Row {
    template <int E>
    static __host__ __device__ constexpr int bytes(int n) { return AL ? n * E : n / 8 * kSlot<E>; }
    template <int E>
    static __device__ __forceinline__ int at(int i)
    {
        return (i * T + threadIdx.x) * (AL ? 8 * E : kSlot<E>);
    }
    template <int E>
    static __device__ __forceinline__ void copy(unsigned char *region, int i, const void *row, int col, int D, bool first)
    {
        if constexpr (AL) copy8_ahead<E>(region + at<E>(i), row, col);
        else copy8_words<E>(region + at<E>(i), row, col, D, first);
    }
    template <class V>
    static __device__ __forceinline__ V8 take(const unsigned char *region, int i, const V *row)
    {
        if constexpr (AL) return take8<V>(region + at<sizeof(V)>(i), 0);
        else return take8_words<V>(region + at<sizeof(V)>(i), row);
    }
    template <class V>
    static __device__ __forceinline__ void put(V *row, int col, int D, const V8 &v)
    {
        if constexpr (AL) put8(row + col, v);
        else put8_any(row, col, D, v);
    }
};

// Waits until at most the `left` latest groups of copies are still under way.
__device__ __forceinline__ void copies_wait(int left)
{
    if (left <= 1) asm volatile("cp.async.wait_group 1;" ::: "memory");
    else if (left == 2) asm volatile("cp.async.wait_group 2;" ::: "memory");
    else asm volatile("cp.async.wait_group 3;" ::: "memory");
}

// The sum over the block (at most 16 warps), the same in every thread.
template <int T>
__device__ __forceinline__ float block_sum(float x, float *red)
{
    const int lane = threadIdx.x & 31;
    x = warp_sum(x);
    if (lane == 0) red[threadIdx.x >> 5] = x;
    __syncthreads();
    x = red[lane & (T / 32 - 1)];
#pragma unroll
    for (int o = T / 64; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// This thread's chunk i of an input of E-byte elements.
template <int T, int E>
__device__ __forceinline__ int chunk_at(int i)
{
    return (i * T + threadIdx.x) * 8 * E;
}

// As many stages (2 to 4) of `stage` bytes as fit beside `kept` bytes; 0 if not
// even two do.
int stages_that_fit(int T, int kept, int stage)
{
    const int n = (kSmemPerSm / (kOwnRegs / T) - 1280 - kept) / stage;
    return n < 2 ? 0 : n < 4 ? n : 4;
}

// Calls f<T, C>() with the threads and chunks per thread of a row of D columns
// until one launches (returns true).
template <class F>
bool pick_threads(int D, F &&f)
{
    using std::integral_constant;
    if (D <= 256) return f(integral_constant<int, 32>{}, integral_constant<int, 1>{});
    if (D <= 512) return f(integral_constant<int, 64>{}, integral_constant<int, 1>{});
    if (D <= 1024) return f(integral_constant<int, 128>{}, integral_constant<int, 1>{});
    if (D <= 2048) return f(integral_constant<int, 128>{}, integral_constant<int, 2>{});
    if (D <= 4096)
        return f(integral_constant<int, 256>{}, integral_constant<int, 2>{}) ||
               f(integral_constant<int, 512>{}, integral_constant<int, 1>{});
    return f(integral_constant<int, 512>{}, integral_constant<int, 2>{});
}

// Calls f with the gate's shape: 0 none or one value per row, 1 per channel, 2
// per element.
template <class F>
bool pick_gate(int kind, F &&f)
{
    if (kind == ZERO1_GATE_CHANNEL) return f(std::integral_constant<int, 1>{});
    if (kind == ZERO1_GATE_FULL) return f(std::integral_constant<int, 2>{});
    return f(std::integral_constant<int, 0>{});
}

}  // namespace
