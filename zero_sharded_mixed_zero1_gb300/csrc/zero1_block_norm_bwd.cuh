// zero1_block_norm_bwd.cuh - the backward kernels of the block norms
// (library-internal; each source that includes this compiles one pair of types).
#pragma once

#include "zero1_block_norm.cuh"

namespace {

// ------------------------------------------------------------ backward -----
//
// One pass: dh, dr and the saved activations are read once, dx and dy written
// once: 10 bytes per bf16 element from both checkpoints, 12 from tensors.
// Each thread keeps the column sums of its own columns over all rows that its
// block visits (in registers, or in shared memory where a row takes 1024
// threads and registers are short); a second kernel adds the blocks' sums in
// block order.  This direct kernel takes the rows that do not fit the ring of
// the staged one below (which ones: at the choice of kernel there).

template <class TA, class TR, bool VEC, bool SACC>
__global__ void __launch_bounds__(SACC ? 1024 : 512) k_block_norm_bwd(const Common c, const Bwd a)
{
    constexpr int C = 2, V = 8 * C;
    __shared__ float red[2][2][32];  // by the row's parity and sum
    extern __shared__ float sacc[];  // SACC: [3][V][threads]
    const int tid = threadIdx.x, nthr = blockDim.x;
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

    int flip = 0;
    for (int64_t row = blockIdx.x; row < c.rows; row += gridDim.x, flip ^= 1) {
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
        float gt_slope;
        const float gt = token_gate(c, row, gt_slope);
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
            s1 = row_sum(s1, red[flip][0]) * c.inv_d;
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
                o[k] = p;
                d[i][k] = ad * g[k];
                s2 = fmaf(g[k], p, s2);
            }
            if (a.need_gate && c.gate_kind == ZERO1_GATE_FULL) {
                if (c.sigmoid) {  // (the slopes from the gates again: registers are short)
                    float slope[8];
                    raw_gate8<VEC>(c, row, col, slope);
                    logistic8<true>(slope);
#pragma unroll
                    for (int k = 0; k < 8; ++k) o[k] *= slope[k];
                }
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
        if (post || tok) s2 = row_sum(s2, red[flip][1]);
        if (tok && tid == 0) {
            const float dg = s2 * gt_slope;
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
#pragma unroll
        for (int i = 0; i < C; ++i)
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int cc = chunk_col<VEC>(i, tid, nthr) + kStep<VEC> * k;
                if (cc < c.D) part[cc] = SACC ? sacc[(s * V + i * 8 + k) * nthr + tid] : acc[SACC ? 0 : s][i][k];
            }
    }
}

// ------------------------------------------------------- staged backward ---
//
// The same sums as above, with a thread's column sums in registers.  Measured
// on GB300: from checkpoints 8192 x 4096 70 us (4.8 TB/s, 0.71 of the measured
// copy rate; 63 us without the joining of the column sums), 16384 x 8192 with
// an elementwise sigmoid gate 294 us (6.4 TB/s, 0.95), from tensors 8192 x 4096
// 73 us (0.82), 32768 x 768 83 us (0.81).  Two barriers per row and 16 warps
// per SM leave the schedulers idle half of the time (0.45 instructions per
// cycle each); more warps would need fewer registers than the column sums take.

// A row's statistics and scale bytes travel through the ring as well: plain
// loads a row ahead ended in waits that the compiler put where it liked (20 to
// 100 us on the larger sizes).  Each warp has 16 words per stage: rstd_pre,
// rstd_post, and from word 4 on the aligned words around the scale bytes of
// its 128-column blocks, two per chunk, those of y8 first.  This lane copies
// word `lane`.
template <int T, int C>
struct RowWords {
    const char *from = nullptr;
    int bytes_per_row = 1;

    __device__ __forceinline__ RowWords(const Common &c, const float *rstd_pre, const float *rstd_post)
    {
        const int lane = threadIdx.x & 31, k = lane - 4;
        if (lane < 2) {
            from = reinterpret_cast<const char *>(lane == 0 ? rstd_pre : rstd_post);
            bytes_per_row = 4;
        } else if (k >= 0 && k < 4 * C) {
            const Ckpt &q = k < 2 * C ? c.y8 : c.r8;
            const int col = (threadIdx.x / 32 * 32 + (k % 2) * 16) * 8 + k / 2 % C * T * 8;
            if (q.codes && col < c.D) from = reinterpret_cast<const char *>(q.exps + (int64_t)(col / kQBlock) * q.ld_exps);
        }
    }
    __device__ __forceinline__ void copy_ahead(uint32_t *words, int64_t row) const
    {
        if (!from) return;
        const uint32_t d = (uint32_t)__cvta_generic_to_shared(words + (threadIdx.x & 31));
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(d), "l"(from + ((row * bytes_per_row) & ~INT64_C(3)))
                     : "memory");
    }
    // The scale of this thread's chunk i: of y8, or (half 1) of r8.
    static __device__ __forceinline__ float scale(const uint32_t *words, int64_t row, int half, int i)
    {
        const uint32_t w = words[4 + 2 * (C * half + i) + (threadIdx.x >> 4 & 1)];
        return scale_of((w >> (8 * ((int)row & 3))) & 255);
    }
};

// Where a row's inputs lie in a stage of T threads with C chunks of 8 columns.
// SAVED: 1 both norms and dr are there and both saved activations are
// checkpoints, 2 the same with tensors, 0 any other mix, decided at run time.
template <class TA, class TR, int T, int C, int SAVED, bool AL>
struct Stage {
    using Ld = Row<T, AL>;
    static constexpr int n = 8 * C * T;
    static constexpr int A = Ld::template bytes<sizeof(TA)>(n), B = Ld::template bytes<sizeof(TR)>(n);
    static constexpr int dh = 0, dr = dh + A, y = dr + B;
    static constexpr int r = y + (SAVED == 1 ? n : A);
    static constexpr int words = r + (SAVED == 1 ? n : B);
    static constexpr int words_bytes = SAVED == 2 ? 16 : 64;  // of a warp
    static constexpr int gate = words + T / 32 * words_bytes;
};

// GATE: 0 none or one value per row, 1 per channel, 2 per element.  FULL: the
// row has exactly 8 C T columns.
template <class TA, class TR, int T, int C, int GATE, int SAVED, bool FULL, bool AL>
__global__ void __launch_bounds__(T, kOwnRegs / T)
k_block_norm_bwd_staged(const Common c, const Bwd a, const int stages, const int stage_bytes)
{
    using S = Stage<TA, TR, T, C, SAVED, AL>;
    using Ld = Row<T, AL>;
    constexpr int A = sizeof(TA), B = sizeof(TR), kVector = S::n * 4;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ float red[2][2][16];
    const int tid = threadIdx.x;
    const bool pre = SAVED || c.w_pre, post = SAVED || c.w_post, dr = SAVED || a.dr;
    const bool r8 = SAVED ? SAVED == 1 : c.r8.codes != nullptr, y8 = SAVED ? SAVED == 1 : c.y8.codes != nullptr;
    const bool ysaved = SAVED || y8 || a.y;
    const bool tok = GATE == 0 && a.need_gate;
    unsigned char *kept = smem;  // w_pre, w_post, the channel gate's factor
    unsigned char *ring = smem + (GATE == 1 ? 3 : 2) * kVector;
    auto in = [&](int i) { return FULL || tid * 8 + i * T * 8 < c.D; };

    const RowWords<T, C> row_words(c, a.rstd_pre, a.rstd_post);
    auto words_of = [&](unsigned char *stage) { return reinterpret_cast<uint32_t *>(stage + S::words + tid / 32 * S::words_bytes); };

    // Starts the copies of a row; past the last row, an empty group that keeps the count.
    auto fetch = [&](int64_t row, unsigned char *to) {
        if (row < c.rows) {
            row_words.copy_ahead(words_of(to), row);
            const TA *dh = static_cast<const TA *>(a.dh) + row * a.ld_dh;
            const TR *ddr = static_cast<const TR *>(a.dr) + row * a.ld_dr;
            const void *y = y8 ? (const void *)(c.y8.codes + row * c.y8.ld_codes)
                               : (const void *)(static_cast<const TA *>(a.y) + row * a.ld_y);
            const void *r = r8 ? (const void *)(c.r8.codes + row * c.r8.ld_codes)
                               : (const void *)(static_cast<const TR *>(a.r) + row * a.ld_r);
            const char *gate = static_cast<const char *>(c.gate) + row * c.ld_gate * (c.gf32 ? 4 : 2);
#pragma unroll
            for (int i = 0; i < C; ++i) {
                const int col = tid * 8 + i * T * 8;
                if (!in(i)) continue;
                if (pre) {
                    Ld::template copy<A>(to + S::dh, i, dh, col, c.D, row * a.ld_dh == 0);
                    if (r8) copy8_ahead<1>(to + S::r + chunk_at<T, 1>(i), r, col);
                    else Ld::template copy<B>(to + S::r, i, r, col, c.D, row * a.ld_r == 0);
                }
                if (dr) Ld::template copy<B>(to + S::dr, i, ddr, col, c.D, row * a.ld_dr == 0);
                if (y8) copy8_ahead<1>(to + S::y + chunk_at<T, 1>(i), y, col);
                else if (ysaved) Ld::template copy<A>(to + S::y, i, y, col, c.D, row * a.ld_y == 0);
                if (GATE == 2) {
                    if (c.gf32) Ld::template copy<4>(to + S::gate, i, gate, col, c.D, row * c.ld_gate == 0);
                    else Ld::template copy<2>(to + S::gate, i, gate, col, c.D, row * c.ld_gate == 0);
                }
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    for (int k = 0; k + 1 < stages; ++k) fetch(blockIdx.x + (int64_t)k * gridDim.x, ring + k * stage_bytes);

    keep_vector<T, C>(kept, c.w_pre, c.pf32, c.D, 0);
    keep_vector<T, C>(kept + kVector, c.w_post, c.pf32, c.D, 0);
    if (GATE == 1) keep_vector<T, C>(kept + 2 * kVector, c.gate, c.gf32, c.D, c.sigmoid);
    V8 acc_post[C], acc_pre[C], acc_gate[GATE == 1 ? C : 1];
#pragma unroll
    for (int i = 0; i < C; ++i) acc_post[i] = acc_pre[i] = acc_gate[GATE == 1 ? i : 0] = splat8(0.f);

    int st = 0, flip = 0;
    for (int64_t row = blockIdx.x; row < c.rows; row += gridDim.x) {
        float gt = 1.f, gt_slope = 1.f;
        if (GATE == 0 && c.gate_kind == ZERO1_GATE_TOKEN) gt = token_gate(c, row, gt_slope);
        // the stage that this warp has read a row ago is filled again
        __syncwarp();
        fetch(row + (int64_t)(stages - 1) * gridDim.x, ring + (st == 0 ? stages - 1 : st - 1) * stage_bytes);
        copies_wait(stages - 1);
        __syncwarp();
        unsigned char *b = ring + st * stage_bytes;
        const uint32_t *words = words_of(b);
        V8 d[C], h[C];  // h: the saved row, first rh, then yh

        const float rs_pre = pre ? __uint_as_float(words[0]) : 0.f, rs_post = post ? __uint_as_float(words[1]) : 1.f;
        float s = 0.f;
        if (pre) {
#pragma unroll
            for (int i = 0; i < C; ++i) {
                if (!in(i)) continue;
                const V8 w = kept8<T, C>(kept, i);
                d[i] = Ld::take(b + S::dh, i, static_cast<const TA *>(a.dh) + row * a.ld_dh);
                if (r8) h[i] = take_codes(b + S::r + chunk_at<T, 1>(i), row_words.scale(words, row, 1, i));
                else h[i] = mul8(Ld::take(b + S::r, i, static_cast<const TR *>(a.r) + row * a.ld_r), rs_pre);
                if (!AL) h[i] = below(h[i], tid * 8 + i * T * 8, c.D);
                acc_pre[i] = fma8(d[i], h[i], acc_pre[i]);
                d[i] = mul8(d[i], w);
                s += dot8(d[i], h[i]);
            }
            s = block_sum<T>(s, red[flip][0]) * -c.inv_d;
        }

        // x: the gradient of r; then p = a x u, the gradient of the gate's
        // factor, and d = a g x, the gradient of u
        float t = 0.f;
        TR *dx = static_cast<TR *>(a.dx) + row * a.ld_dx;
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const int col = tid * 8 + i * T * 8;
            if (!in(i)) continue;
            V8 x = dr ? Ld::take(b + S::dr, i, static_cast<const TR *>(a.dr) + row * a.ld_dr) : splat8(0.f);
            if (pre) x = fma8(fma8(h[i], s, d[i]), rs_pre, x);
            Ld::put(dx, col, c.D, x);
            if (y8) h[i] = take_codes(b + S::y + chunk_at<T, 1>(i), row_words.scale(words, row, 0, i));
            else if (ysaved) h[i] = mul8(Ld::take(b + S::y, i, static_cast<const TA *>(a.y) + row * a.ld_y), rs_post);
            else h[i] = splat8(0.f);
            if (!AL) h[i] = below(h[i], col, c.D);
            const V8 u = post ? mul8(kept8<T, C>(kept + kVector, i), h[i]) : h[i];
            if (GATE == 0) {
                t += dot8(x, u);  // times a: the gradient of a token's gate
                d[i] = mul8(x, c.alpha * gt);
            } else {
                V8 gc, slope;
                if (GATE == 1) {
                    gc = kept8<T, C>(kept + 2 * kVector, i);
                } else {
                    gc = c.gf32 ? Ld::take(b + S::gate, i, static_cast<const float *>(c.gate) + row * c.ld_gate)
                                : Ld::take(b + S::gate, i, static_cast<const uint16_t *>(c.gate) + row * c.ld_gate);
                    if (c.sigmoid) logistic8(gc, slope);
                }
                const V8 ax = mul8(x, c.alpha), p = mul8(ax, u);
                if (GATE == 1) acc_gate[GATE == 1 ? i : 0] = add8(acc_gate[GATE == 1 ? i : 0], p);
                t += dot8(gc, p);
                d[i] = mul8(ax, gc);
                if (GATE == 2 && a.need_gate) {
                    const V8 o = c.sigmoid ? mul8(p, slope) : p;
                    if (c.gf32) Ld::put(static_cast<float *>(a.dgate) + row * a.ld_dgate, col, c.D, o);
                    else Ld::put(static_cast<uint16_t *>(a.dgate) + row * a.ld_dgate, col, c.D, o);
                }
            }
            acc_post[i] = fma8(d[i], h[i], acc_post[i]);
        }
        if (post || tok) t = block_sum<T>(t, red[flip][1]);
        if (GATE == 0) {
            t *= c.alpha;
            if (tok && tid == 0) {
                const float dg = t * gt_slope;
                if (c.wf32) static_cast<float *>(a.dgate)[row * a.ld_dgate] = dg;
                else static_cast<uint16_t *>(a.dgate)[row * a.ld_dgate] = to_bf16(dg);
            }
            t *= gt;
        }
        t *= -c.inv_d;
        TA *dy = static_cast<TA *>(a.dy) + row * a.ld_dy;
#pragma unroll
        for (int i = 0; i < C; ++i) {
            if (!in(i)) continue;
            if (post) d[i] = mul8(fma8(h[i], t, mul8(d[i], kept8<T, C>(kept + kVector, i))), rs_post);
            Ld::put(dy, tid * 8 + i * T * 8, c.D, d[i]);
        }
        flip ^= 1;
        if (++st == stages) st = 0;
    }
    const int64_t plane = (int64_t)gridDim.x * c.D;
#pragma unroll
    for (int i = 0; i < C; ++i) {
        if (!in(i)) continue;
        const int col = tid * 8 + i * T * 8;
        if (!AL) {
            float *part = a.part + (int64_t)blockIdx.x * c.D;
            if (a.need_post) put8_any(part, col, c.D, acc_post[i]);
            if (a.need_pre) put8_any(part + plane, col, c.D, acc_pre[i]);
            if (GATE == 1 && a.need_gate) put8_any(part + 2 * plane, col, c.D, acc_gate[GATE == 1 ? i : 0]);
            continue;
        }
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

template <class TA, class TR, bool VEC, bool SACC>
int launch_bwd(const Common &c, const Bwd &a, int64_t grid, cudaStream_t st)
{
    auto kernel = k_block_norm_bwd<TA, TR, VEC, SACC>;
    const int threads = row_threads(c.D), smem = SACC ? 3 * 16 * threads * 4 : 0;
    if (SACC) {
        static std::atomic<uint64_t> done{0};
        const cudaError_t e = allow_smem(kernel, 3 * 16 * 1024 * 4, done);
        if (e != cudaSuccess) return z1_fail(ZERO1_ECUDA, "block norm backward: %s", cudaGetErrorString(e));
    }
    kernel<<<(unsigned)grid, threads, smem, st>>>(c, a);
    z1_note_launch(reinterpret_cast<const void *>(kernel), (int)grid, 1, threads, 0);
    return launch_status("block norm backward launch");
}

template <class TA, class TR, bool VEC>
int direct_bwd(const Common &c, const Bwd &a, int64_t grid, cudaStream_t st)
{
    if (c.D <= 8192) return launch_bwd<TA, TR, VEC, false>(c, a, grid, st);
    return launch_bwd<TA, TR, VEC, true>(c, a, grid, st);
}

// One resident wave of staged blocks (`grid`); false, with nothing launched, if
// a row does not fit: two stages, which are sized for 8 C T columns and, but for
// SAVED = 1, for tensors, beside two or three vectors of as many fp32 values.
template <class TA, class TR, int T, int C, int GATE, int SAVED, bool FULL, bool AL>
bool launch_bwd_staged(const Common &c, const Bwd &a, int64_t grid, cudaStream_t st, int *rc)
{
    auto kernel = k_block_norm_bwd_staged<TA, TR, T, C, GATE, SAVED, FULL, AL>;
    using S = Stage<TA, TR, T, C, SAVED, AL>;
    constexpr int kept = (GATE == 1 ? 3 : 2) * S::n * 4;
    const int stage = S::gate + (GATE != 2 ? 0 : c.gf32 ? S::Ld::template bytes<4>(S::n) : S::Ld::template bytes<2>(S::n));
    const int stages = stages_that_fit(T, kept, stage);
    if (stages == 0) return false;
    const int smem = kept + stages * stage;
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = allow_smem(kernel, kSmemPerSm - 1024, done);
    if (e != cudaSuccess) {
        *rc = z1_fail(ZERO1_ECUDA, "block norm backward: %s", cudaGetErrorString(e));
        return true;
    }
    kernel<<<(unsigned)grid, T, smem, st>>>(c, a, stages, stage);
    z1_note_launch(reinterpret_cast<const void *>(kernel), (int)grid, kOwnRegs / T, T, 0);
    *rc = launch_status("block norm backward launch");
    return true;
}

// The mixes in use are compiled apart (SAVED) for rows of exactly 8 C T columns,
// 256 to 8192 in powers of two; any other row takes the run-time mix.  us on the
// device, compiled apart and as a run-time mix, 33.6 million bf16 elements,
// without a gate and with a channel gate:
//   columns   from checkpoints         from tensors
//   1024      66 / 83    69 / 87       74 / 84    75 / 88
//   2048      67 / 72    69 / 198      76 / 73   154 / 154
//   4096      67 / 73    71 / 104      73 / 72    74 / 105
//   8192      75 / 71    68 / 210      70 / 73    72 / 167
// The long times are rows that do not fit the ring and run on the direct kernel:
//   - above 8192 columns, all (398 to 654);
//   - at 1025 to 2048 and 4097 to 8192 columns: bf16 with a channel or full gate
//     (5120: 293 from checkpoints, 221 from tensors; without a gate 90) but for
//     the mixes compiled apart at 2048 (checkpoints) and 8192 columns; an fp32
//     residual stream or fp32 activations (353 to 506) but for 2048 and 8192 columns
//     from checkpoints with bf16 activations and without such a gate (83, 85); and
//     rows off the 128-bit path;
//   - up to 256 columns, fp32 activations off the 128-bit path with a full fp32 gate.
template <class TA, class TR>
bool backward_staged(const Common &c, const Bwd &a, bool vec, int64_t grid, cudaStream_t st, int *rc)
{
    if (c.D > 8192) return false;
    if (c.gate_kind == ZERO1_GATE_FULL && (!c.gvec || (a.need_gate && !a.dgvec))) vec = false;
    const int codes = (c.y8.codes != nullptr) + (c.r8.codes != nullptr);
    const int kinds = !c.w_pre || !c.w_post || !a.dr ? 0 : codes == 2 ? 1 : codes == 0 ? 2 : 0;
    return pick_threads(c.D, [&](auto t, auto n) {
        constexpr int T = decltype(t)::value, C = decltype(n)::value;
        return pick_gate(c.gate_kind, [&](auto gate) {
            constexpr int G = decltype(gate)::value;
            if (!vec) return launch_bwd_staged<TA, TR, T, C, G, 0, false, false>(c, a, grid, st, rc);
            if constexpr (sizeof(TA) == 2 && !(T == 512 && C == 1)) {
                const int saved = c.D == 8 * C * T ? kinds : 0;
                if (saved == 1) return launch_bwd_staged<TA, TR, T, C, G, 1, true, true>(c, a, grid, st, rc);
                if (saved == 2) return launch_bwd_staged<TA, TR, T, C, G, 2, true, true>(c, a, grid, st, rc);
            }
            return launch_bwd_staged<TA, TR, T, C, G, 0, false, true>(c, a, grid, st, rc);
        });
    });
}

}  // namespace

template <class TA, class TR>
int z1bn::run_backward(const Common &c, const Bwd &a, bool vec, int64_t grid, cudaStream_t st)
{
    int rc;
    if (backward_staged<TA, TR>(c, a, vec, grid, st, &rc)) return rc;
    return vec ? direct_bwd<TA, TR, true>(c, a, grid, st) : direct_bwd<TA, TR, false>(c, a, grid, st);
}
