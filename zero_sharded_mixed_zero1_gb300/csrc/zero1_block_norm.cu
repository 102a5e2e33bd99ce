// zero1_block_norm.cu - norms before and after a block, fused with the
// block's gate and residual scale: forward and backward.

#include "zero1_block.cuh"

namespace {

constexpr int kMaxCols = ZERO1_BLOCK_NORM_MAX_COLS;
constexpr int kWarpRows = 8;  // rows (one per warp) of a block in the narrow shapes

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

// ---------------------------------------------------------- row geometry ---
//
// A row lives in the registers of one warp (narrow rows) or of one block, V
// elements per thread in chunks of 8.  On the vector path a chunk is 8
// consecutive columns; otherwise its elements are 16 columns apart.  Either
// way 16 neighbouring lanes hold one 128-column checkpoint block per chunk.

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
// that nothing there turns into a NaN).
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
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int c = col + kStep<VEC> * k;
            f[k] = c < D ? ld_param(p, f32, base + c) : 1.f;
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

// The sum over a row, the same in every thread.  Consecutive calls in a block
// alternate between two `red` buffers, so one barrier per call is enough.
template <bool WARP>
__device__ __forceinline__ float row_sum(float x, float *red)
{
    x = warp_sum(x);
    if constexpr (!WARP) {
        const int lane = threadIdx.x & 31;
        if (lane == 0) red[threadIdx.x >> 5] = x;
        __syncthreads();
        x = warp_sum(lane < (int)(blockDim.x >> 5) ? red[lane] : 0.f);
    }
    return x;
}

__device__ __forceinline__ float sigmoid(float x) { return __fdividef(1.f, 1.f + __expf(-x)); }
__device__ __forceinline__ float rstd_of(float ss, const Common &c)
{
    return __frcp_rn(__fsqrt_rn(fmaf(ss, c.inv_d, c.eps)));
}

// The gate's factor for a chunk (channel and full gates; else g is left).
template <bool VEC>
__device__ __forceinline__ void gate8(const Common &c, int64_t row, int col, float g[8])
{
    if (c.gate_kind == ZERO1_GATE_CHANNEL) param8<VEC>(c.gate, c.gf32, c.pvec, 0, col, c.D, g);
    else if (c.gate_kind == ZERO1_GATE_FULL) param8<VEC>(c.gate, c.gf32, c.gvec, row * c.ld_gate, col, c.D, g);
    else return;
    if (c.sigmoid) {
#pragma unroll
        for (int k = 0; k < 8; ++k) g[k] = sigmoid(g[k]);
    }
}

__device__ __forceinline__ float token_gate(const Common &c, int64_t row)
{
    if (c.gate_kind != ZERO1_GATE_TOKEN) return 1.f;
    const float g = ld_param(c.gate, c.gf32, row * c.ld_gate);
    return c.sigmoid ? sigmoid(g) : g;
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

// ------------------------------------------------------------- forward -----
//
// One pass: y and x are read once, both statistics come from registers, and
// r, h and the checkpoints are written once: 10 bytes per bf16 element with
// both checkpoints, 8 without.  HBM is the bound.

template <class TA, class TR, int V, bool VEC, bool WARP>
__global__ void __launch_bounds__(V == 16 && !WARP ? 1024 : 256) k_block_norm_fwd(const Common c, const Fwd a)
{
    constexpr int C = V / 8;
    __shared__ float red[2][32];
    const int tid = WARP ? threadIdx.x & 31 : threadIdx.x;
    const int nthr = WARP ? 32 : blockDim.x;
    const int64_t row0 = WARP ? (int64_t)blockIdx.x * kWarpRows + (threadIdx.x >> 5) : blockIdx.x;
    const int64_t step = WARP ? (int64_t)gridDim.x * kWarpRows : gridDim.x;
    for (int64_t row = row0; row < c.rows; row += step) {
        Chunk<TA, VEC> yq[C];
        Chunk<TR, VEC> xq[C];
        const TA *y = static_cast<const TA *>(a.y) + row * a.ld_y;
        const TR *x = static_cast<const TR *>(a.x) + row * a.ld_x;
#pragma unroll
        for (int i = 0; i < C; ++i) yq[i].load(y, chunk_col<VEC>(i, tid, nthr), c.D);
#pragma unroll
        for (int i = 0; i < C; ++i) xq[i].load(x, chunk_col<VEC>(i, tid, nthr), c.D);
        const float gt = token_gate(c, row);
        float f[C][8];
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < C; ++i) {
            yq[i].get(f[i]);
#pragma unroll
            for (int k = 0; k < 8; ++k) ss = fmaf(f[i][k], f[i][k], ss);
        }
        float rs = 1.f;
        if (c.w_post) {
            rs = rstd_of(row_sum<WARP>(ss, red[0]), c);
            if (tid == 0) a.rstd_post[row] = rs;
        }
        ss = 0.f;
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const int col = chunk_col<VEC>(i, tid, nthr);
            float w[8], g[8], xv[8];
            if (c.w_post) {
                param8<VEC>(c.w_post, c.pf32, c.pvec, 0, col, c.D, w);
#pragma unroll
                for (int k = 0; k < 8; ++k) f[i][k] *= rs;
            }
            if (c.y8.codes) pack_chunk<VEC>(c.y8, row, col, c.D, f[i]);
#pragma unroll
            for (int k = 0; k < 8; ++k) g[k] = gt;
            gate8<VEC>(c, row, col, g);
            xq[i].get(xv);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float u = c.w_post ? f[i][k] * w[k] : f[i][k];
                f[i][k] = fmaf(c.alpha * g[k], u, xv[k]);
            }
            store_chunk<TR, VEC>(static_cast<TR *>(a.r) + row * a.ld_r, col, c.D, f[i]);
#pragma unroll
            for (int k = 0; k < 8; ++k) ss = fmaf(f[i][k], f[i][k], ss);
        }
        if (!c.w_pre) continue;
        rs = rstd_of(row_sum<WARP>(ss, red[1]), c);
        if (tid == 0) a.rstd_pre[row] = rs;
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const int col = chunk_col<VEC>(i, tid, nthr);
            float w[8];
            param8<VEC>(c.w_pre, c.pf32, c.pvec, 0, col, c.D, w);
#pragma unroll
            for (int k = 0; k < 8; ++k) f[i][k] *= rs;
            if (c.r8.codes) pack_chunk<VEC>(c.r8, row, col, c.D, f[i]);
#pragma unroll
            for (int k = 0; k < 8; ++k) f[i][k] *= w[k];
            store_chunk<TA, VEC>(static_cast<TA *>(a.h) + row * a.ld_h, col, c.D, f[i]);
        }
    }
}

// ------------------------------------------------------------ backward -----
//
// One pass: dh, dr and the saved activations are read once, dx and dy written
// once: 10 bytes per bf16 element from both checkpoints, 12 from tensors.
// Each thread keeps the column sums of its own columns over all rows that its
// block visits (in registers, or in shared memory where a row takes 1024
// threads and registers are short); a second kernel adds the blocks' sums in
// block order.

template <class TA, class TR, int V, bool VEC, bool WARP, bool SACC>
__global__ void __launch_bounds__(SACC ? 1024 : (WARP ? 256 : 512)) k_block_norm_bwd(const Common c, const Bwd a)
{
    constexpr int C = V / 8;
    __shared__ float red[2][32];
    extern __shared__ float sacc[];  // SACC: [3][V][threads]; WARP: [D] for the blocks' sum
    const int tid = WARP ? threadIdx.x & 31 : threadIdx.x;
    const int nthr = WARP ? 32 : blockDim.x;
    const int64_t row0 = WARP ? (int64_t)blockIdx.x * kWarpRows + (threadIdx.x >> 5) : blockIdx.x;
    const int64_t step = WARP ? (int64_t)gridDim.x * kWarpRows : gridDim.x;
    float acc[SACC ? 1 : 3][C][8];
    if constexpr (SACC) {
        for (int q = 0; q < 3 * V; ++q) sacc[q * nthr + tid] = 0.f;
    } else {
#pragma unroll
        for (int s = 0; s < 3; ++s)
#pragma unroll
            for (int i = 0; i < C; ++i)
#pragma unroll
                for (int k = 0; k < 8; ++k) acc[s][i][k] = 0.f;
    }
    auto add = [&](int s, int i, int k, float x) {
        if constexpr (SACC) sacc[(s * V + i * 8 + k) * nthr + tid] += x;
        else acc[s][i][k] += x;
    };

    for (int64_t row = row0; row < c.rows; row += step) {
        Chunk<TA, VEC> hq[C], yq[C];
        Chunk<TR, VEC> dq[C], rq[C];
        uint2 y8[C], r8[C];
        int ey[C], er[C];
        const bool pre = c.w_pre, post = c.w_post;
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const int col = chunk_col<VEC>(i, tid, nthr);
            if (pre) {
                hq[i].load(static_cast<const TA *>(a.dh) + row * a.ld_dh, col, c.D);
                if (c.r8.codes) load_codes<VEC>(c.r8, row, col, c.D, r8[i], er[i]);
                else rq[i].load(static_cast<const TR *>(a.r) + row * a.ld_r, col, c.D);
            }
            if (a.dr) dq[i].load(static_cast<const TR *>(a.dr) + row * a.ld_dr, col, c.D);
            if (c.y8.codes) load_codes<VEC>(c.y8, row, col, c.D, y8[i], ey[i]);
            else if (a.y) yq[i].load(static_cast<const TA *>(a.y) + row * a.ld_y, col, c.D);
        }
        const float gt = token_gate(c, row);
        const float rs_pre = pre ? a.rstd_pre[row] : 0.f, rs_post = post ? a.rstd_post[row] : 1.f;
        float d[C][8], rh[C][8];
        float s1 = 0.f;
        if (pre) {
#pragma unroll
            for (int i = 0; i < C; ++i) {
                const int col = chunk_col<VEC>(i, tid, nthr);
                float w[8];
                param8<VEC>(c.w_pre, c.pf32, c.pvec, 0, col, c.D, w);
                hq[i].get(d[i]);
                if (c.r8.codes) {
                    values8(r8[i], scale_of(er[i]), rh[i]);
                } else {
                    rq[i].get(rh[i]);
#pragma unroll
                    for (int k = 0; k < 8; ++k) rh[i][k] *= rs_pre;
                }
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    if (a.need_pre) add(1, i, k, d[i][k] * rh[i][k]);
                    d[i][k] *= w[k];
                    s1 = fmaf(d[i][k], rh[i][k], s1);
                }
            }
            s1 = row_sum<WARP>(s1, red[0]) * c.inv_d;
        }
        float s2 = 0.f;
        float yh[C][8];
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const int col = chunk_col<VEC>(i, tid, nthr);
            float r0[8], g[8], w[8], o[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) r0[k] = 0.f;
            if (a.dr) dq[i].get(r0);
#pragma unroll
            for (int k = 0; k < 8; ++k) d[i][k] = pre ? fmaf(rs_pre, fmaf(-rh[i][k], s1, d[i][k]), r0[k]) : r0[k];
            store_chunk<TR, VEC>(static_cast<TR *>(a.dx) + row * a.ld_dx, col, c.D, d[i]);
#pragma unroll
            for (int k = 0; k < 8; ++k) yh[i][k] = 0.f;
            if (c.y8.codes) {
                values8(y8[i], scale_of(ey[i]), yh[i]);
            } else if (a.y) {
                yq[i].get(yh[i]);
#pragma unroll
                for (int k = 0; k < 8; ++k) yh[i][k] *= rs_post;
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) { g[k] = 1.f; w[k] = 1.f; }
            gate8<VEC>(c, row, col, g);
            if (post) param8<VEC>(c.w_post, c.pf32, c.pvec, 0, col, c.D, w);
            // p = a d u, the gradient of the gate's factor; d becomes a g d, the
            // gradient of u
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float ad = c.alpha * d[i][k];
                const float p = ad * (w[k] * yh[i][k]);
                if (a.need_gate && c.gate_kind == ZERO1_GATE_CHANNEL) add(2, i, k, p);
                o[k] = p * (c.sigmoid ? g[k] * (1.f - g[k]) : 1.f);
                d[i][k] = ad * g[k];
                s2 = fmaf(g[k], p, s2);
            }
            if (a.need_gate && c.gate_kind == ZERO1_GATE_FULL) {
                if (VEC && a.dgvec) {
                    if (c.gf32) store_chunk<float, true>(static_cast<float *>(a.dgate) + row * a.ld_dgate, col, c.D, o);
                    else store_chunk<uint16_t, true>(static_cast<uint16_t *>(a.dgate) + row * a.ld_dgate, col, c.D, o);
                } else {
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const int cc = col + kStep<VEC> * k;
                        if (cc >= c.D) continue;
                        if (c.gf32) st1(static_cast<float *>(a.dgate) + row * a.ld_dgate + cc, o[k]);
                        else st1(static_cast<uint16_t *>(a.dgate) + row * a.ld_dgate + cc, o[k]);
                    }
                }
            }
        }
        const bool tok = a.need_gate && c.gate_kind == ZERO1_GATE_TOKEN;
        if (post || tok) s2 = row_sum<WARP>(s2, red[1]);
        if (tok && tid == 0) {
            const float dg = c.sigmoid ? s2 * gt * (1.f - gt) : s2;
            if (c.wf32) static_cast<float *>(a.dgate)[row * a.ld_dgate] = dg;
            else static_cast<uint16_t *>(a.dgate)[row * a.ld_dgate] = to_bf16(dg);
        }
        s2 *= c.inv_d * gt;  // a token gate's factor is the same over the row
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const int col = chunk_col<VEC>(i, tid, nthr);
            float w[8];
            if (post) param8<VEC>(c.w_post, c.pf32, c.pvec, 0, col, c.D, w);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float dyh = d[i][k] * gt;
                if (a.need_post) add(0, i, k, dyh * yh[i][k]);
                d[i][k] = post ? rs_post * fmaf(-yh[i][k], s2, dyh * w[k]) : dyh;
            }
            store_chunk<TA, VEC>(static_cast<TA *>(a.dy) + row * a.ld_dy, col, c.D, d[i]);
        }
    }

    // this block's column sums
#pragma unroll
    for (int s = 0; s < 3; ++s) {
        const bool need = s == 0 ? a.need_post : s == 1 ? a.need_pre
                                                        : a.need_gate && c.gate_kind == ZERO1_GATE_CHANNEL;
        if (!need) continue;
        float *part = a.part + ((int64_t)s * gridDim.x + blockIdx.x) * c.D;
        if constexpr (WARP) {  // the warps add up in turn
            for (int w = 0; w < kWarpRows; ++w) {
                if ((int)(threadIdx.x >> 5) == w) {
#pragma unroll
                    for (int i = 0; i < C; ++i)
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            const int cc = chunk_col<VEC>(i, tid, nthr) + kStep<VEC> * k;
                            if (cc < c.D) sacc[cc] = (w ? sacc[cc] : 0.f) + acc[s][i][k];
                        }
                }
                __syncthreads();
            }
            for (int cc = threadIdx.x; cc < c.D; cc += blockDim.x) part[cc] = sacc[cc];
            __syncthreads();
        } else {
#pragma unroll
            for (int i = 0; i < C; ++i)
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const int cc = chunk_col<VEC>(i, tid, nthr) + kStep<VEC> * k;
                    if (cc < c.D) part[cc] = SACC ? sacc[(s * V + i * 8 + k) * nthr + tid] : acc[SACC ? 0 : s][i][k];
                }
        }
    }
}

// ------------------------------------------------------- staged backward ---
//
// Rows of more than 512 columns that 128-bit accesses can address, up to the
// widths whose rows fit shared memory.  The inputs of R rows at a time travel
// through a ring of shared-memory stages, so that loads are in flight through
// all phases of a row and both of its sums.  A thread copies its own columns
// (cp.async) and reads only those, so the ring needs no barrier.  Bulk copies
// of whole rows were slower: about 12 bytes per cycle and SM came in (90 us at
// 8192 x 4096), however many were in flight.
//
// A block of at most 512 threads keeps up to 128 registers per thread: the
// column sums, and what one phase leaves to the next.  A thread owns C chunks
// of 8 columns of each of the R rows; two units of work per thread (R C = 2)
// share one reading of the weights and one barrier per sum.

struct Ring {
    int stages, stage_bytes, row_bytes;
    int at_dh, at_dr, at_y, at_r, at_gate;       // offsets in a staged row
    int by_dh, by_dr, by_y, by_r, by_gate;       // bytes of a row's inputs (0: none)
    int at_wpre, at_wpost, at_wgate, at_stage;   // offsets in shared memory
};

constexpr int kStagedThreads = 512;

// Keeps a [D] vector (D a multiple of 8) in shared memory as fp32 values,
// through the logistic function if asked: the first four values of each eight,
// then the last four, so that a warp's 16-byte reads touch every bank once.
__device__ __forceinline__ void keep_vector(float *dst, const void *src, int f32, int D, int act)
{
    if (!src) return;
    const bool vec = ((uintptr_t)src & 15) == 0;
    for (int c = threadIdx.x * 8; c < D; c += blockDim.x * 8) {
        float f[8];
        param8<true>(src, f32, vec, 0, c, D, f);
#pragma unroll
        for (int k = 0; k < 8; ++k) f[k] = act ? sigmoid(f[k]) : f[k];
        *reinterpret_cast<float4 *>(dst + c / 2) = make_float4(f[0], f[1], f[2], f[3]);
        *reinterpret_cast<float4 *>(dst + D / 2 + c / 2) = make_float4(f[4], f[5], f[6], f[7]);
    }
}
__device__ __forceinline__ V8 kept8(const unsigned char *kept, int col, int D)
{
    const float4 a = *reinterpret_cast<const float4 *>(kept + col * 2), b = *reinterpret_cast<const float4 *>(kept + D * 2 + col * 2);
    return V8{{pair(a.x, a.y), pair(a.z, a.w), pair(b.x, b.y), pair(b.z, b.w)}};
}

// Loads that stay where they are written, ahead of the wait for a stage: the
// compiler would move plain ones down to their use a group later, and their
// latency with them (24 us of 90 at 8192 x 4096).
__device__ __forceinline__ float ld_ahead(const float *p)
{
    float x;
    asm volatile("ld.global.nc.f32 %0, [%1];" : "=f"(x) : "l"(p));
    return x;
}
__device__ __forceinline__ uint16_t ld_ahead(const uint16_t *p)
{
    uint16_t x;
    asm volatile("ld.global.nc.u16 %0, [%1];" : "=h"(x) : "l"(p));
    return x;
}
__device__ __forceinline__ uint16_t ld_ahead(const uint8_t *p)
{
    uint16_t x;
    asm volatile("{ .reg .u16 t; ld.global.nc.u8 t, [%1]; mov.u16 %0, t; }" : "=h"(x) : "l"(p));
    return x;
}

// What a thread needs of a group of rows besides the staged bytes, fetched a
// group ahead.
template <int C, int R>
struct RowScalars {
    float rs_pre[R], rs_post[R], gate[R];
    uint16_t ey[C], er[C];  // the scale bytes of the group's rows
};

// Those of the group that starts at row (a row within the matrix; a missing
// second row gets the first one's values).
template <int C, int R>
__device__ __forceinline__ void load_scalars(const Common &c, bool pre, bool post, const float *rstd_pre, const float *rstd_post,
                                             const uint8_t *const (&ey)[C], const uint8_t *const (&er)[C], int64_t row,
                                             RowScalars<C, R> &s)
{
    const int more = row + 1 < c.rows ? 1 : 0;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        s.rs_pre[r] = pre ? ld_ahead(rstd_pre + row + r * more) : 0.f;
        s.rs_post[r] = post ? ld_ahead(rstd_post + row + r * more) : 1.f;
        s.gate[r] = c.gate_kind == ZERO1_GATE_TOKEN ? ld_param(c.gate, c.gf32, (row + r * more) * c.ld_gate) : 1.f;
    }
#pragma unroll
    for (int i = 0; i < C; ++i) {
        if (R == 2) {  // row is even, and the scales of a block are padded to 128 rows
            if (ey[i]) s.ey[i] = ld_ahead(reinterpret_cast<const uint16_t *>(ey[i] + row));
            if (er[i]) s.er[i] = ld_ahead(reinterpret_cast<const uint16_t *>(er[i] + row));
            if (!more) {
                s.ey[i] = (uint16_t)((s.ey[i] & 255) * 257);
                s.er[i] = (uint16_t)((s.er[i] & 255) * 257);
            }
        } else {
            if (ey[i]) s.ey[i] = ld_ahead(ey[i] + row);
            if (er[i]) s.er[i] = ld_ahead(er[i] + row);
        }
    }
}

// A thread's column of scales, or NULL.
__device__ __forceinline__ const uint8_t *scale_column(const Ckpt &k, int col, int D)
{
    return k.codes && col < D ? k.exps + (int64_t)(col / kQBlock) * k.ld_exps : nullptr;
}

// The sums of R rows over the block (at most 16 warps), the same in every thread.
template <int R>
__device__ __forceinline__ void block_sums(float x[R], float *red)
{
    const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    if constexpr (R == 2) {
        // from the first step on, the lower lanes carry row 0 and the upper ones row 1
        const bool hi = lane >= 16;
        const float got = __shfl_xor_sync(0xffffffffu, hi ? x[0] : x[1], 16);
        float y = (hi ? x[1] : x[0]) + got;
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
        if ((lane & 15) == 0) red[(lane & 16) + (threadIdx.x >> 5)] = y;
        __syncthreads();
        y = (lane & 15) < warps ? red[lane] : 0.f;
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
        x[0] = __shfl_sync(0xffffffffu, y, 0);
        x[1] = __shfl_sync(0xffffffffu, y, 16);
    } else {
        float y = warp_sum(x[0]);
        if (lane == 0) red[threadIdx.x >> 5] = y;
        __syncthreads();
        y = (lane & 15) < warps ? red[lane & 15] : 0.f;
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
        x[0] = y;
    }
}

// Starts copying N bytes (8 or 16) to shared memory; zeros if `there` is false.
template <int N>
__device__ __forceinline__ void copy_ahead(unsigned char *dst, const void *src, bool there)
{
    const uint32_t d = (uint32_t)__cvta_generic_to_shared(dst);
    const int n = there ? N : 0;
    if constexpr (N == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(d), "l"(src), "r"(n) : "memory");
    else asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(d), "l"(src), "r"(n) : "memory");
}
// Eight elements of a row.
template <class T>
__device__ __forceinline__ void copy8_ahead(unsigned char *row, const T *src, int col, bool there)
{
    copy_ahead<16>(row + col * sizeof(T), src + col, there);
    if (sizeof(T) == 4) copy_ahead<16>(row + col * sizeof(T) + 16, src + col + 4, there);
}
__device__ __forceinline__ void copies_end_group() { asm volatile("cp.async.commit_group;" ::: "memory"); }

// Waits until at most the `left` latest groups of copies are still under way.
__device__ __forceinline__ void copies_wait(int left)
{
    if (left <= 1) asm volatile("cp.async.wait_group 1;" ::: "memory");
    else if (left == 2) asm volatile("cp.async.wait_group 2;" ::: "memory");
    else asm volatile("cp.async.wait_group 3;" ::: "memory");
}

// GATE: 0 none or one value per row, 1 per channel, 2 per element.  SAVED: 1
// both norms and dr are there and both saved activations are checkpoints, 2
// the same with tensors, 0 any other mix, decided at run time.
template <class TA, class TR, int C, int R, int GATE, int SAVED>
__global__ void __launch_bounds__(kStagedThreads, 1) k_block_norm_bwd_staged(const Common c, const Bwd a, const Ring g)
{
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ float red[2][2][32];
    const int tid = threadIdx.x, stride = blockDim.x * 8;
    const bool pre = SAVED || c.w_pre, post = SAVED || c.w_post, dr = SAVED || a.dr;
    const bool r8 = SAVED ? SAVED == 1 : c.r8.codes != nullptr, y8 = SAVED ? SAVED == 1 : c.y8.codes != nullptr;
    const bool ysaved = SAVED || g.by_y;
    const bool tok = GATE == 0 && a.need_gate;
    const int64_t groups = (c.rows + R - 1) / R;
    // Starts the copies of a group of rows; past the last group, an empty group
    // of copies that keeps the count.
    auto fetch = [&](int64_t group, int st) {
        if (group < groups) {
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const bool there = r == 0 || group * R + r < c.rows;
                const int64_t row = group * R + (there ? r : 0);
                unsigned char *b = smem + g.at_stage + st * g.stage_bytes + r * g.row_bytes;
#pragma unroll
                for (int i = 0; i < C; ++i) {
                    const int col = tid * 8 + i * stride;
                    if (col >= c.D) continue;
                    if (pre) {
                        copy8_ahead(b + g.at_dh, static_cast<const TA *>(a.dh) + row * a.ld_dh, col, there);
                        if (r8) copy_ahead<8>(b + g.at_r + col, c.r8.codes + row * c.r8.ld_codes + col, there);
                        else copy8_ahead(b + g.at_r, static_cast<const TR *>(a.r) + row * a.ld_r, col, there);
                    }
                    if (dr) copy8_ahead(b + g.at_dr, static_cast<const TR *>(a.dr) + row * a.ld_dr, col, there);
                    if (y8) copy_ahead<8>(b + g.at_y + col, c.y8.codes + row * c.y8.ld_codes + col, there);
                    else if (ysaved) copy8_ahead(b + g.at_y, static_cast<const TA *>(a.y) + row * a.ld_y, col, there);
                    if (GATE == 2) {
                        if (c.gf32) copy8_ahead(b + g.at_gate, static_cast<const float *>(c.gate) + row * c.ld_gate, col, there);
                        else copy8_ahead(b + g.at_gate, static_cast<const uint16_t *>(c.gate) + row * c.ld_gate, col, there);
                    }
                }
            }
        }
        copies_end_group();
    };
    for (int k = 0; k + 1 < g.stages; ++k) fetch(blockIdx.x + (int64_t)k * gridDim.x, k);
    keep_vector(reinterpret_cast<float *>(smem + g.at_wpre), c.w_pre, c.pf32, c.D, 0);
    keep_vector(reinterpret_cast<float *>(smem + g.at_wpost), c.w_post, c.pf32, c.D, 0);
    if (GATE == 1) keep_vector(reinterpret_cast<float *>(smem + g.at_wgate), c.gate, c.gf32, c.D, c.sigmoid);
    V8 acc_post[C], acc_pre[C], acc_gate[GATE == 1 ? C : 1];
    const uint8_t *ey[C], *er[C];
#pragma unroll
    for (int i = 0; i < C; ++i) {
        acc_post[i] = acc_pre[i] = acc_gate[GATE == 1 ? i : 0] = splat8(0.f);
        ey[i] = scale_column(c.y8, tid * 8 + i * stride, c.D);
        er[i] = scale_column(c.r8, tid * 8 + i * stride, c.D);
    }
    RowScalars<C, R> cur, next;
    load_scalars<C, R>(c, pre, post, a.rstd_pre, a.rstd_post, ey, er, (int64_t)blockIdx.x * R, cur);
    __syncthreads();

    int st = 0, flip = 0;
    for (int64_t group = blockIdx.x; group < groups; group += gridDim.x) {
        const int64_t row0 = group * R;
        {
            const int64_t following = group + gridDim.x;
            load_scalars<C, R>(c, pre, post, a.rstd_pre, a.rstd_post, ey, er, (following < groups ? following : group) * R, next);
        }
        // the stage that this thread has read a group ago is filled again
        fetch(group + (int64_t)(g.stages - 1) * gridDim.x, st == 0 ? g.stages - 1 : st - 1);
        copies_wait(g.stages - 1);
        const unsigned char *base = smem + g.at_stage + st * g.stage_bytes;
        const bool both = R == 1 || row0 + 1 < c.rows;  // a missing second row counts as zeros
        V8 d[C][R], h[C][R];  // h: the saved row, first rh, then yh

        float s[R] = {};
        if (pre) {
#pragma unroll
            for (int i = 0; i < C; ++i) {
                const int col = tid * 8 + i * stride;
                if (col >= c.D) continue;
                const V8 w = kept8(smem + g.at_wpre, col, c.D);
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const unsigned char *b = base + r * g.row_bytes;
                    d[i][r] = take8<TA>(b + g.at_dh, col);
                    if (r8) h[i][r] = take_codes(b + g.at_r + col, scale_of((cur.er[i] >> (8 * r)) & 255));
                    else h[i][r] = mul8(take8<TR>(b + g.at_r, col), cur.rs_pre[r]);
                    acc_pre[i] = fma8(d[i][r], h[i][r], acc_pre[i]);
                    d[i][r] = mul8(d[i][r], w);
                    s[r] += dot8(d[i][r], h[i][r]);
                }
            }
            block_sums<R>(s, red[flip][0]);
        }

        // x: the gradient of r; then p = a x u, the gradient of the gate's
        // factor, and d = a g x, the gradient of u
        float t[R] = {}, gt[R];
#pragma unroll
        for (int r = 0; r < R; ++r)
            gt[r] = GATE || c.gate_kind != ZERO1_GATE_TOKEN ? 1.f : c.sigmoid ? sigmoid(cur.gate[r]) : cur.gate[r];
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const int col = tid * 8 + i * stride;
            if (col >= c.D) continue;
            const V8 w = post ? kept8(smem + g.at_wpost, col, c.D) : splat8(1.f);
            V8 gc = w;
            if (GATE == 1) gc = kept8(smem + g.at_wgate, col, c.D);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const unsigned char *b = base + r * g.row_bytes;
                const bool there = r == 0 || both;
                V8 x = dr ? take8<TR>(b + g.at_dr, col) : splat8(0.f);
                if (pre) x = fma8(fma8(h[i][r], -s[r] * c.inv_d, d[i][r]), cur.rs_pre[r], x);
                if (there) put8(static_cast<TR *>(a.dx) + (row0 + r) * a.ld_dx + col, x);
                if (y8) h[i][r] = take_codes(b + g.at_y + col, scale_of((cur.ey[i] >> (8 * r)) & 255));
                else if (ysaved) h[i][r] = mul8(take8<TA>(b + g.at_y, col), cur.rs_post[r]);
                else h[i][r] = splat8(0.f);
                const V8 u = mul8(w, h[i][r]);
                if (GATE == 0) {
                    t[r] += dot8(x, u);  // times a: the gradient of a token's gate
                    d[i][r] = mul8(x, c.alpha * gt[r]);
                } else {
                    if (GATE == 2) {
                        gc = take8(b + g.at_gate, c.gf32, col);
                        if (c.sigmoid) gc = map8(gc, [](float v) { return sigmoid(v); });
                    }
                    const V8 ax = mul8(x, c.alpha), p = mul8(ax, u);
                    if (GATE == 1) acc_gate[GATE == 1 ? i : 0] = add8(acc_gate[GATE == 1 ? i : 0], p);
                    t[r] += dot8(gc, p);
                    d[i][r] = mul8(ax, gc);
                    if (GATE == 2 && a.need_gate && there) {
                        const V8 o = c.sigmoid ? mul8(p, map8(gc, [](float v) { return v * (1.f - v); })) : p;
                        if (c.gf32) put8(static_cast<float *>(a.dgate) + (row0 + r) * a.ld_dgate + col, o);
                        else put8(static_cast<uint16_t *>(a.dgate) + (row0 + r) * a.ld_dgate + col, o);
                    }
                }
                acc_post[i] = fma8(d[i][r], h[i][r], acc_post[i]);
            }
        }
        if (post || tok) block_sums<R>(t, red[flip][1]);
        if (GATE == 0) {
#pragma unroll
            for (int r = 0; r < R; ++r) {
                t[r] *= c.alpha;
                if (tok && tid == r && (r == 0 || both)) {
                    const float dg = c.sigmoid ? t[r] * gt[r] * (1.f - gt[r]) : t[r];
                    if (c.wf32) static_cast<float *>(a.dgate)[(row0 + r) * a.ld_dgate] = dg;
                    else static_cast<uint16_t *>(a.dgate)[(row0 + r) * a.ld_dgate] = to_bf16(dg);
                }
                t[r] *= gt[r];
            }
        }
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const int col = tid * 8 + i * stride;
            if (col >= c.D) continue;
            const V8 w = post ? kept8(smem + g.at_wpost, col, c.D) : splat8(1.f);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                if (post) d[i][r] = mul8(fma8(h[i][r], -t[r] * c.inv_d, mul8(d[i][r], w)), cur.rs_post[r]);
                if (r == 0 || both) put8(static_cast<TA *>(a.dy) + (row0 + r) * a.ld_dy + col, d[i][r]);
            }
        }
        cur = next;
        flip ^= 1;
        if (++st == g.stages) st = 0;
    }
    const int64_t plane = (int64_t)gridDim.x * c.D;
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const int col = tid * 8 + i * stride;
        if (col >= c.D) continue;
        float4 *part = reinterpret_cast<float4 *>(a.part + (int64_t)blockIdx.x * c.D + col);
        auto put = [&](float4 *p, const V8 &v) {
            const float2 x = split(v.p[0]), y = split(v.p[1]), z = split(v.p[2]), w = split(v.p[3]);
            p[0] = make_float4(x.x, x.y, y.x, y.y);
            p[1] = make_float4(z.x, z.y, w.x, w.y);
        };
        if (a.need_post) put(part, acc_post[i]);
        if (a.need_pre) put(part + plane / 4, acc_pre[i]);
        if (GATE == 1 && a.need_gate) put(part + plane / 2, acc_gate[GATE == 1 ? i : 0]);
    }
}

// Adds the blocks' partial column sums in block order: 32 columns per block,
// 8 slices of the partials each summed in order and then joined in order.
struct Finish {
    const float *part;
    int64_t nparts;
    int D, f32, accumulate;
    void *out[3];       // dw_post, dw_pre, dgate (NULL: not wanted)
    const void *gate;   // a sigmoid channel gate, else NULL
    int gf32;
};

__global__ void __launch_bounds__(256) k_block_norm_finish(const Finish f)
{
    wait_prior_grid();
    __shared__ float sum[8][32];
    const int s = blockIdx.y;
    if (!f.out[s]) return;
    const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5;
    const int col = blockIdx.x * 32 + lane;
    const float *p = f.part + (int64_t)s * f.nparts * f.D + col;
    const int64_t per = (f.nparts + 7) / 8, b = slice * per, e = b + per < f.nparts ? b + per : f.nparts;
    float x = 0.f;
    if (col < f.D) {
#pragma unroll 8
        for (int64_t q = b; q < e; ++q) x += p[q * f.D];
    }
    sum[slice][lane] = x;
    __syncthreads();
    if (slice || col >= f.D) return;
#pragma unroll
    for (int q = 1; q < 8; ++q) x += sum[q][lane];
    if (s == 2 && f.gate) {
        const float g = sigmoid(ld_param(f.gate, f.gf32, col));
        x *= g * (1.f - g);
    }
    if (f.f32) {
        float *o = static_cast<float *>(f.out[s]) + col;
        *o = f.accumulate ? *o + x : x;
    } else {
        uint16_t *o = static_cast<uint16_t *>(f.out[s]) + col;
        *o = to_bf16(f.accumulate ? bf_one(*o) + x : x);
    }
}

// --------------------------------------------------------------- launch ----

// Threads of a block for D columns: narrow rows take a warp each.
int row_threads(int64_t D) { return D <= 512 ? 256 : (int)round_up(D, 512) / 16; }

// Blocks of the backward kernel: one resident wave at most, with about 512
// threads per SM at work.
int64_t bwd_blocks(int64_t rows, int64_t D, int sms)
{
    const int64_t per_sm = D <= 512 ? 2 : D <= 4096 ? 4096 / round_up(D, 256) : 1;
    const int64_t work = D <= 512 ? (rows + kWarpRows - 1) / kWarpRows : D <= 4096 ? (rows + 1) / 2 : rows;
    return work < per_sm * sms ? work : per_sm * sms;
}

int check_cfg(const zero1_block_norm_t *cfg, bool has_gate, bool has_post, bool has_pre, const char *call)
{
    if (!cfg) return z1_fail(ZERO1_EINVAL, "%s: the configuration is NULL", call);
    if (cfg->rows < 0 || cfg->cols < 1)
        return z1_fail(ZERO1_EINVAL, "%s: %lld rows, %lld columns", call, (long long)cfg->rows, (long long)cfg->cols);
    if (cfg->cols > kMaxCols || cfg->rows > (INT64_C(1) << 40))
        return z1_fail(ZERO1_ERANGE, "%s: %lld rows of %lld columns (at most %d columns)", call, (long long)cfg->rows,
                       (long long)cfg->cols, kMaxCols);
    if (!(cfg->eps > 0.f) || !std::isfinite(cfg->eps)) return z1_fail(ZERO1_EINVAL, "%s: eps must be finite and > 0", call);
    if (!std::isfinite(cfg->residual_scale)) return z1_fail(ZERO1_EINVAL, "%s: residual_scale is not finite", call);
    int rc;
    if ((rc = check_dtype(cfg->act_dtype, call, "act_dtype")) || (rc = check_dtype(cfg->res_dtype, call, "res_dtype")) ||
        (rc = check_dtype(cfg->param_dtype, call, "param_dtype")) ||
        (rc = check_dtype(cfg->gate_dtype, call, "gate_dtype")) ||
        (rc = check_dtype(cfg->grad_dtype, call, "grad_dtype")))
        return rc;
    if (cfg->act_dtype == ZERO1_DTYPE_F32 && cfg->res_dtype != ZERO1_DTYPE_F32)
        return z1_fail(ZERO1_EINVAL, "%s: fp32 activations need an fp32 residual stream", call);
    if (cfg->gate_kind < ZERO1_GATE_NONE || cfg->gate_kind > ZERO1_GATE_FULL ||
        (cfg->gate_act != ZERO1_GATE_LINEAR && cfg->gate_act != ZERO1_GATE_SIGMOID))
        return z1_fail(ZERO1_EINVAL, "%s: unknown gate kind %d or activation %d", call, cfg->gate_kind, cfg->gate_act);
    if (cfg->rows > 0 && has_gate != (cfg->gate_kind != ZERO1_GATE_NONE))
        return z1_fail(ZERO1_EINVAL, "%s: gate kind %d with a %s gate", call, cfg->gate_kind, has_gate ? "non-NULL" : "NULL");
    (void)has_post;
    (void)has_pre;
    return ZERO1_OK;
}

// The gate as a matrix of the call.
Mat gate_mat(const zero1_block_norm_t *cfg, const void *p, int64_t ld, int es, const char *what)
{
    switch (cfg->gate_kind) {
    case ZERO1_GATE_CHANNEL: return mat(p, 1, cfg->cols, 0, es, what);
    case ZERO1_GATE_TOKEN: return mat(p, cfg->rows, 1, ld, es, what);
    case ZERO1_GATE_FULL: return mat(p, cfg->rows, cfg->cols, ld, es, what);
    default: return Mat{nullptr, 0, 0, 0, what};
    }
}

int check_saved(const zero1_block_norm_t *cfg, const zero1_checkpoint8_t *k, const char *call, const char *what)
{
    int rc = check_ckpt(k, call, what);
    if (rc != ZERO1_OK) return rc;
    if (k->rows != cfg->rows || k->cols != cfg->cols)
        return z1_fail(ZERO1_EINVAL, "%s: %s is %lld x %lld, not %lld x %lld", call, what, (long long)k->rows,
                       (long long)k->cols, (long long)cfg->rows, (long long)cfg->cols);
    return ZERO1_OK;
}

// EINVAL if an output overlaps another output or an input.  in_place[o] names
// the input that output o may coincide with (-1: none).
int check_overlaps(const Mat *out, const int *in_place, int nout, const Mat *in, int nin, const char *call)
{
    for (int o = 0; o < nout; ++o) {
        for (int q = o + 1; q < nout; ++q)
            if (mats_overlap(out[o], out[q]))
                return z1_fail(ZERO1_EINVAL, "%s: %s and %s overlap", call, out[o].what, out[q].what);
        for (int q = 0; q < nin; ++q) {
            if (!mats_overlap(out[o], in[q])) continue;
            if (in_place[o] == q && out[o].p == in[q].p && out[o].pitch == in[q].pitch && out[o].width == in[q].width)
                continue;
            return z1_fail(ZERO1_EINVAL, "%s: %s and %s overlap", call, out[o].what, in[q].what);
        }
    }
    return ZERO1_OK;
}

Common common_of(const zero1_block_norm_t *cfg, const void *w_post, const void *w_pre, const void *gate, int64_t ld_gate,
                 const zero1_checkpoint8_t *y8, const zero1_checkpoint8_t *r8)
{
    Common c{};
    c.rows = cfg->rows;
    c.D = (int)cfg->cols;
    c.eps = cfg->eps;
    c.alpha = cfg->residual_scale;
    c.inv_d = (float)(1.0 / (double)cfg->cols);
    c.gate_kind = cfg->gate_kind;
    c.sigmoid = cfg->gate_act == ZERO1_GATE_SIGMOID && cfg->gate_kind != ZERO1_GATE_NONE;
    c.pf32 = cfg->param_dtype == ZERO1_DTYPE_F32;
    c.gf32 = cfg->gate_dtype == ZERO1_DTYPE_F32;
    c.wf32 = cfg->grad_dtype == ZERO1_DTYPE_F32;
    c.w_post = w_post;
    c.w_pre = w_pre;
    c.gate = gate;
    c.ld_gate = cfg->rows > 1 ? ld_gate : 0;
    const void *chan = cfg->gate_kind == ZERO1_GATE_CHANNEL ? gate : nullptr;
    c.pvec = ((((uintptr_t)w_post) | (uintptr_t)w_pre | (uintptr_t)chan) & 15) == 0;
    c.gvec = vec_ok(gate_mat(cfg, gate, ld_gate, esize(cfg->gate_dtype), "gate"));
    if (y8) c.y8 = Ckpt{y8->codes, y8->exps, y8->ld_codes, y8->ld_exps};
    if (r8) c.r8 = Ckpt{r8->codes, r8->exps, r8->ld_codes, r8->ld_exps};
    return c;
}

template <class TA, class TR, int V, bool VEC, bool WARP>
int launch_fwd(const Common &c, const Fwd &a, int threads, int sms, cudaStream_t st)
{
    auto kernel = k_block_norm_fwd<TA, TR, V, VEC, WARP>;
    const int per_sm = blocks_per_sm(reinterpret_cast<const void *>(kernel), threads);
    const int64_t work = WARP ? (c.rows + kWarpRows - 1) / kWarpRows : c.rows;
    const int64_t grid = work < (int64_t)sms * per_sm ? work : (int64_t)sms * per_sm;
    kernel<<<(unsigned)grid, threads, 0, st>>>(c, a);
    z1_note_launch(reinterpret_cast<const void *>(kernel), (int)grid, per_sm, threads, 0);
    return launch_status("block norm forward launch");
}

template <class TA, class TR, bool VEC>
int pick_fwd(const Common &c, const Fwd &a, int sms, cudaStream_t st)
{
    const int threads = row_threads(c.D);
    if (c.D <= 256) return launch_fwd<TA, TR, 8, VEC, true>(c, a, threads, sms, st);
    if (c.D <= 512) return launch_fwd<TA, TR, 16, VEC, true>(c, a, threads, sms, st);
    return launch_fwd<TA, TR, 16, VEC, false>(c, a, threads, sms, st);
}

template <class TA, class TR, int V, bool VEC, bool WARP, bool SACC>
int launch_bwd(const Common &c, const Bwd &a, int threads, int64_t grid, cudaStream_t st)
{
    auto kernel = k_block_norm_bwd<TA, TR, V, VEC, WARP, SACC>;
    const int smem = SACC ? 3 * V * threads * 4 : WARP ? c.D * 4 : 0;
    if (SACC) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return z1_fail(ZERO1_ECUDA, "block norm backward: %s", cudaGetErrorString(e));
    }
    kernel<<<(unsigned)grid, threads, smem, st>>>(c, a);
    z1_note_launch(reinterpret_cast<const void *>(kernel), (int)grid, 1, threads, 0);
    return launch_status("block norm backward launch");
}

constexpr int kStagedSmem = 220 * 1024;

// The stages of R rows for the staged kernel; false if they do not fit.
bool ring_of(const Common &c, const Bwd &a, int ea, int er, int R, Ring *g)
{
    *g = Ring{};
    int at = 0;
    auto place = [&](int *where, int *bytes, int64_t n) {
        *where = at;
        *bytes = (int)n;
        at += (int)round_up(n, 128);
    };
    const int D = c.D, eg = c.gf32 ? 4 : 2;
    const int64_t codes = D;
    place(&g->at_dh, &g->by_dh, c.w_pre ? D * ea : 0);
    place(&g->at_dr, &g->by_dr, a.dr ? D * er : 0);
    place(&g->at_y, &g->by_y, c.y8.codes ? codes : a.y ? D * ea : 0);
    place(&g->at_r, &g->by_r, c.r8.codes ? codes : c.w_pre ? D * er : 0);
    place(&g->at_gate, &g->by_gate, c.gate_kind == ZERO1_GATE_FULL ? D * eg : 0);
    g->row_bytes = at;
    g->stage_bytes = at * R;
    at = 0;
    int unused;
    place(&g->at_wpre, &unused, c.w_pre ? D * 4 : 0);
    place(&g->at_wpost, &unused, c.w_post ? D * 4 : 0);
    place(&g->at_wgate, &unused, c.gate_kind == ZERO1_GATE_CHANNEL ? D * 4 : 0);
    g->at_stage = at;
    g->stages = (kStagedSmem - at) / (g->stage_bytes > 0 ? g->stage_bytes : 1);
    if (g->stages > 4) g->stages = 4;
    return g->stages >= 2;
}

template <class TA, class TR, int C, int R>
int launch_bwd_staged(const Common &c, const Bwd &a, const Ring &g, int threads, int64_t grid, cudaStream_t st)
{
    auto go = [&](auto kernel) {
        const int smem = g.at_stage + g.stages * g.stage_bytes;
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return z1_fail(ZERO1_ECUDA, "block norm backward: %s", cudaGetErrorString(e));
        kernel<<<(unsigned)grid, threads, smem, st>>>(c, a, g);
        z1_note_launch(reinterpret_cast<const void *>(kernel), (int)grid, 1, threads, 0);
        return launch_status("block norm backward launch");
    };
    const int codes = (c.y8.codes != nullptr) + (c.r8.codes != nullptr);
    const int saved = !c.w_pre || !c.w_post || !a.dr ? 0 : codes == 2 ? 1 : codes == 0 ? 2 : 0;
    auto with = [&](auto gate) {
        constexpr int G = decltype(gate)::value;
        if (saved == 1) return go(k_block_norm_bwd_staged<TA, TR, C, R, G, 1>);
        if (saved == 2) return go(k_block_norm_bwd_staged<TA, TR, C, R, G, 2>);
        return go(k_block_norm_bwd_staged<TA, TR, C, R, G, 0>);
    };
    if (c.gate_kind == ZERO1_GATE_CHANNEL) return with(std::integral_constant<int, 1>{});
    if (c.gate_kind == ZERO1_GATE_FULL) return with(std::integral_constant<int, 2>{});
    return with(std::integral_constant<int, 0>{});
}

template <class TA, class TR, bool VEC>
int pick_bwd(const Common &c, const Bwd &a, int64_t grid, cudaStream_t st)
{
    const int threads = row_threads(c.D);
    if constexpr (VEC) {
        Ring g;
        const bool fits = c.D > 512 && c.D <= 8192 && (c.gate_kind != ZERO1_GATE_FULL || (c.gvec && (!a.need_gate || a.dgvec)));
        const int n = (int)round_up(c.D, 256) / 8;
        const int ea = sizeof(TA), er = sizeof(TR);
        if (fits && n <= kStagedThreads) {
            if (ring_of(c, a, ea, er, 2, &g)) return launch_bwd_staged<TA, TR, 1, 2>(c, a, g, n, grid, st);
            if (ring_of(c, a, ea, er, 1, &g)) return launch_bwd_staged<TA, TR, 1, 1>(c, a, g, n, grid, st);
        } else if (fits && ring_of(c, a, ea, er, 1, &g)) {
            return launch_bwd_staged<TA, TR, 2, 1>(c, a, g, (int)round_up(c.D, 512) / 16, grid, st);
        }
    }
    if (c.D <= 256) return launch_bwd<TA, TR, 8, VEC, true, false>(c, a, threads, grid, st);
    if (c.D <= 512) return launch_bwd<TA, TR, 16, VEC, true, false>(c, a, threads, grid, st);
    if (c.D <= 8192) return launch_bwd<TA, TR, 16, VEC, false, false>(c, a, threads, grid, st);
    return launch_bwd<TA, TR, 16, VEC, false, true>(c, a, threads, grid, st);
}

// Calls f(TA, TR, VEC) for the run-time types.
template <class F>
int dispatch_types(const zero1_block_norm_t *cfg, bool vec, F &&f)
{
    auto with = [&](auto v) {
        if (cfg->act_dtype == ZERO1_DTYPE_F32) return f(float{}, float{}, v);
        if (cfg->res_dtype == ZERO1_DTYPE_F32) return f(uint16_t{}, float{}, v);
        return f(uint16_t{}, uint16_t{}, v);
    };
    return vec ? with(std::true_type{}) : with(std::false_type{});
}

}  // namespace

extern "C" int zero1_block_norm_forward(const zero1_block_norm_t *cfg, const zero1_block_norm_forward_t *io,
                                        zero1_stream_t stream)
{
    Z1Trace trace("zero1_block_norm_forward");
    const char *call = "block norm forward";
    if (!io) return z1_fail(ZERO1_EINVAL, "%s: the buffers are NULL", call);
    int rc = check_cfg(cfg, io->gate != nullptr, io->w_post != nullptr, io->w_pre != nullptr, call);
    if (rc != ZERO1_OK || cfg->rows == 0) return rc;
    const int64_t T = cfg->rows, D = cfg->cols;
    const int ea = esize(cfg->act_dtype), er = esize(cfg->res_dtype), ep = esize(cfg->param_dtype),
              eg = esize(cfg->gate_dtype);
    const Mat in[] = {mat(io->x, T, D, io->ld_x, er, "x"), mat(io->y, T, D, io->ld_y, ea, "y"),
                      mat(io->w_post, 1, D, 0, ep, "w_post"), mat(io->w_pre, 1, D, 0, ep, "w_pre"),
                      gate_mat(cfg, io->gate, io->ld_gate, eg, "gate")};
    const Mat out[] = {mat(io->r, T, D, io->ld_r, er, "r"), mat(io->h, T, D, io->ld_h, ea, "h"),
                       mat(io->rstd_post, 1, T, 0, 4, "rstd_post"), mat(io->rstd_pre, 1, T, 0, 4, "rstd_pre"),
                       codes_mat(io->y8, "the codes of y8"), exps_mat(io->y8, "the exps of y8"),
                       codes_mat(io->r8, "the codes of r8"), exps_mat(io->r8, "the exps of r8")};
    const int in_place[] = {0, -1, -1, -1, -1, -1, -1, -1};
    if ((rc = check_mat(in[0], er, false, call)) || (rc = check_mat(in[1], ea, false, call)) ||
        (rc = check_mat(out[0], er, true, call)) || (io->gate && (rc = check_mat(in[4], eg, false, call))))
        return rc;
    if (io->w_post && ((rc = check_natural(io->w_post, ep, "w_post")) || (rc = check_mat(out[2], 4, true, call)))) return rc;
    if (io->w_pre && ((rc = check_natural(io->w_pre, ep, "w_pre")) || (rc = check_mat(out[1], ea, true, call)) ||
                      (rc = check_mat(out[3], 4, true, call))))
        return rc;
    if (!io->w_post && io->rstd_post) return z1_fail(ZERO1_EINVAL, "%s: rstd_post without w_post", call);
    if (!io->w_pre && (io->h || io->rstd_pre || io->r8))
        return z1_fail(ZERO1_EINVAL, "%s: h, rstd_pre or r8 without w_pre", call);
    if (io->y8 && (rc = check_saved(cfg, io->y8, call, "y8")) != ZERO1_OK) return rc;
    if (io->r8 && (rc = check_saved(cfg, io->r8, call, "r8")) != ZERO1_OK) return rc;
    if ((rc = check_overlaps(out, in_place, 8, in, 5, call)) != ZERO1_OK) return rc;
    const int sms = sm_count();
    if (sms == 0) return z1_fail(ZERO1_ECUDA, "%s: no CUDA device", call);
    const Common c = common_of(cfg, io->w_post, io->w_pre, io->gate, io->ld_gate, io->y8, io->r8);
    const Fwd a{io->y, io->x, io->r, io->h, io->rstd_post, io->rstd_pre, io->ld_y, io->ld_x, io->ld_r, io->ld_h};
    const bool vec = D % 8 == 0 && vec_ok(in[0]) && vec_ok(in[1]) && vec_ok(out[0]) && vec_ok(out[1]);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    return dispatch_types(cfg, vec, [&](auto ta, auto tr, auto v) {
        return pick_fwd<decltype(ta), decltype(tr), decltype(v)::value>(c, a, sms, st);
    });
}

extern "C" int zero1_block_norm_workspace(const zero1_block_norm_t *cfg, int64_t *bytes)
{
    const char *call = "block norm workspace";
    if (!bytes) return z1_fail(ZERO1_EINVAL, "%s: bytes is NULL", call);
    int rc = check_cfg(cfg, cfg && cfg->gate_kind != ZERO1_GATE_NONE, true, true, call);
    if (rc != ZERO1_OK) return rc;
    const int sms = sm_count();
    if (sms == 0) return z1_fail(ZERO1_ECUDA, "%s: no CUDA device", call);
    *bytes = 3 * bwd_blocks(cfg->rows, cfg->cols, sms) * cfg->cols * 4;
    return ZERO1_OK;
}

extern "C" int zero1_block_norm_backward(const zero1_block_norm_t *cfg, const zero1_block_norm_backward_t *io,
                                         void *workspace, int64_t workspace_bytes, zero1_stream_t stream)
{
    Z1Trace trace("zero1_block_norm_backward");
    const char *call = "block norm backward";
    if (!io) return z1_fail(ZERO1_EINVAL, "%s: the buffers are NULL", call);
    const bool post = io->w_post, pre = io->w_pre;
    int rc = check_cfg(cfg, io->gate != nullptr, post, pre, call);
    if (rc != ZERO1_OK) return rc;
    const int64_t T = cfg->rows, D = cfg->cols;
    const int ea = esize(cfg->act_dtype), er = esize(cfg->res_dtype), ep = esize(cfg->param_dtype),
              eg = esize(cfg->gate_dtype), ew = esize(cfg->grad_dtype);
    const int edg = cfg->gate_kind == ZERO1_GATE_FULL ? eg : ew;
    const Mat in[] = {mat(io->dr, T, D, io->ld_dr, er, "dr"), mat(io->dh, T, D, io->ld_dh, ea, "dh"),
                      mat(io->y, T, D, io->ld_y, ea, "y"), mat(io->r, T, D, io->ld_r, er, "r"),
                      mat(io->w_post, 1, D, 0, ep, "w_post"), mat(io->w_pre, 1, D, 0, ep, "w_pre"),
                      gate_mat(cfg, io->gate, io->ld_gate, eg, "gate"),
                      mat(io->rstd_post, 1, T, 0, 4, "rstd_post"), mat(io->rstd_pre, 1, T, 0, 4, "rstd_pre"),
                      codes_mat(io->y8, "the codes of y8"), exps_mat(io->y8, "the exps of y8"),
                      codes_mat(io->r8, "the codes of r8"), exps_mat(io->r8, "the exps of r8")};
    Mat work{workspace, 1, workspace_bytes, workspace_bytes, "the workspace"};
    const Mat out[] = {mat(io->dx, T, D, io->ld_dx, er, "dx"), mat(io->dy, T, D, io->ld_dy, ea, "dy"),
                       mat(io->dw_post, 1, D, 0, ew, "dw_post"), mat(io->dw_pre, 1, D, 0, ew, "dw_pre"),
                       gate_mat(cfg, io->dgate, io->ld_dgate, edg, "dgate"), work};
    const int in_place[] = {0, 1, -1, -1, -1, -1};
    if (!post && (io->dw_post || io->rstd_post)) return z1_fail(ZERO1_EINVAL, "%s: dw_post or rstd_post without w_post", call);
    if (!pre && (io->dw_pre || io->rstd_pre || io->dh || io->r || io->r8))
        return z1_fail(ZERO1_EINVAL, "%s: dw_pre, rstd_pre, dh, r or r8 without w_pre", call);
    if (io->dgate && cfg->gate_kind == ZERO1_GATE_NONE) return z1_fail(ZERO1_EINVAL, "%s: dgate without a gate", call);
    const bool need_y = post || io->dgate;
    if (T > 0) {
        if ((rc = check_mat(out[0], er, true, call)) || (rc = check_mat(out[1], ea, true, call)) ||
            (io->dr && (rc = check_mat(in[0], er, false, call))) || (io->gate && (rc = check_mat(in[6], eg, false, call))))
            return rc;
        if (pre) {
            if ((rc = check_mat(in[1], ea, false, call)) || (rc = check_natural(io->w_pre, ep, "w_pre")) ||
                (rc = check_mat(in[8], 4, false, call)))
                return rc;
            if ((io->r != nullptr) == (io->r8 != nullptr))
                return z1_fail(ZERO1_EINVAL, "%s: exactly one of r and r8 is needed", call);
            if (io->r8 ? (rc = check_saved(cfg, io->r8, call, "r8")) : (rc = check_mat(in[3], er, false, call))) return rc;
        }
        if (post && ((rc = check_natural(io->w_post, ep, "w_post")) || (rc = check_mat(in[7], 4, false, call)))) return rc;
        if (io->y && io->y8) return z1_fail(ZERO1_EINVAL, "%s: both y and y8", call);
        if (need_y) {
            if (!io->y && !io->y8) return z1_fail(ZERO1_EINVAL, "%s: y or y8 is needed", call);
            if (io->y8 ? (rc = check_saved(cfg, io->y8, call, "y8")) : (rc = check_mat(in[2], ea, false, call))) return rc;
        }
        if (!pre && !io->dr) return z1_fail(ZERO1_EINVAL, "%s: neither dh nor dr", call);
    }
    if ((io->dw_post && (rc = check_natural(io->dw_post, ew, "dw_post"))) ||
        (io->dw_pre && (rc = check_natural(io->dw_pre, ew, "dw_pre"))) ||
        (io->dgate && (rc = check_mat(out[4], edg, true, call))))
        return rc;
    const int sms = sm_count();
    if (sms == 0) return z1_fail(ZERO1_ECUDA, "%s: no CUDA device", call);
    const int64_t grid = bwd_blocks(T, D, sms);
    const bool chan = io->dgate && cfg->gate_kind == ZERO1_GATE_CHANNEL;
    const bool sums = io->dw_post || io->dw_pre || chan;
    const int64_t need = sums ? 3 * grid * D * 4 : 0;
    if (need > 0) {
        if (!workspace || workspace_bytes < need)
            return z1_fail(ZERO1_EINVAL, "%s: workspace of %lld bytes, needs %lld", call,
                           (long long)(workspace ? workspace_bytes : 0), (long long)need);
        if ((uintptr_t)workspace & 15) return z1_fail(ZERO1_EALIGN, "%s: the workspace is not 16-byte aligned", call);
    }
    if ((rc = check_overlaps(out, in_place, 6, in, 13, call)) != ZERO1_OK) return rc;

    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (T > 0) {
        const Common c = common_of(cfg, io->w_post, io->w_pre, io->gate, io->ld_gate, io->y8, io->r8);
        Bwd a{};
        a.dh = io->dh; a.dr = io->dr; a.y = need_y ? io->y : nullptr; a.r = io->r;
        a.rstd_post = io->rstd_post; a.rstd_pre = io->rstd_pre;
        a.dy = io->dy; a.dx = io->dx; a.dgate = io->dgate;
        a.ld_dh = io->ld_dh; a.ld_dr = io->ld_dr; a.ld_y = io->ld_y; a.ld_r = io->ld_r;
        a.ld_dy = io->ld_dy; a.ld_dx = io->ld_dx; a.ld_dgate = T > 1 ? io->ld_dgate : 0;
        a.need_post = io->dw_post != nullptr; a.need_pre = io->dw_pre != nullptr; a.need_gate = io->dgate != nullptr;
        a.dgvec = vec_ok(out[4]);
        a.part = static_cast<float *>(workspace);
        const bool vec = D % 8 == 0 && vec_ok(in[0]) && vec_ok(in[1]) && vec_ok(in[2]) && vec_ok(in[3]) &&
                         vec_ok(out[0]) && vec_ok(out[1]);
        rc = dispatch_types(cfg, vec, [&](auto ta, auto tr, auto v) {
            return pick_bwd<decltype(ta), decltype(tr), decltype(v)::value>(c, a, grid, st);
        });
        if (rc != ZERO1_OK) return rc;
    }
    if (!sums) return ZERO1_OK;
    Finish f{};
    f.part = static_cast<const float *>(workspace);
    f.nparts = grid;
    f.D = (int)D;
    f.f32 = cfg->grad_dtype == ZERO1_DTYPE_F32;
    f.accumulate = cfg->accumulate != 0;
    f.out[0] = io->dw_post;
    f.out[1] = io->dw_pre;
    f.out[2] = chan ? io->dgate : nullptr;
    f.gate = chan && cfg->gate_act == ZERO1_GATE_SIGMOID ? io->gate : nullptr;
    f.gf32 = cfg->gate_dtype == ZERO1_DTYPE_F32;
    cudaLaunchConfig_t lc = {};
    lc.gridDim = dim3((unsigned)((D + 31) / 32), 3);
    lc.blockDim = dim3(256);
    lc.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    lc.attrs = at;
    lc.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&lc, k_block_norm_finish, f);
    if (e != cudaSuccess) return pdl_fail(e, "block norm backward: column sums");
    return ZERO1_OK;
}
