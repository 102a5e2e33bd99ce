// zero1_block_norm_fwd.cuh - the forward kernels of the block norms
// (library-internal; each source that includes this compiles one pair of types).
#pragma once

#include "zero1_block_norm.cuh"

namespace {

// ------------------------------------------------------------- forward -----
//
// One pass: y and x are read once, both statistics come from registers, and
// r, h and the checkpoints are written once: 10 bytes per bf16 element with
// both checkpoints, 8 without.  HBM is the bound.  This direct kernel takes
// the rows that do not fit the ring of the staged one below: above 8192
// columns (94 to 111 us for 33.6 million bf16 elements with checkpoints, where
// the ring takes 57 to 67 up to 4096 and at 8192), at 1025 to 2048 columns fp32
// activations with a channel or full gate and an fp32 residual stream with a
// full fp32 gate, and from 4097 on those of them that are off the 128-bit path
// or have a full fp32 gate beside fp32 activations.

template <class TA, class TR, bool VEC>
__global__ void __launch_bounds__(1024) k_block_norm_fwd(const Common c, const Fwd a)
{
    constexpr int C = 2;
    __shared__ float red[2][2][32];  // by the row's parity and sum
    const int tid = threadIdx.x, nthr = blockDim.x;
    int flip = 0;
    for (int64_t row = blockIdx.x; row < c.rows; row += gridDim.x, flip ^= 1) {
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
            rs = rstd_of(row_sum(ss, red[flip][0]), c);
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
        rs = rstd_of(row_sum(ss, red[flip][1]), c);
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

// ------------------------------------------------------- staged forward ----
//
// Measured on GB300 with both checkpoints, bf16: 8192 x 4096 59 us (5.7 TB/s of
// the 10 bytes per element, 0.85 of the measured copy rate; the direct kernel
// took 75), 32768 x 768 with an fp32 residual stream 54 us (0.83).  What is
// lost is the first rows' latency and, with 16 warps per SM, the waits for
// shuffles and shared memory (0.43 instructions per cycle and scheduler).
//
// KEPT: 1 both norms are there and both checkpoints wanted, 2 both norms and
// no checkpoint, 0 any other mix, decided at run time.  FULL: the row has
// exactly 8 C T columns.

template <class TA, class TR, int T, int C, int GATE, int KEPT, bool FULL, bool AL>
__global__ void __launch_bounds__(T, kOwnRegs / T)
k_block_norm_fwd_staged(const Common c, const Fwd a, const int stages, const int stage_bytes)
{
    using Ld = Row<T, AL>;
    constexpr int A = sizeof(TA), B = sizeof(TR), N = 8 * C * T, kVector = N * 4;
    constexpr int at_y = 0, at_x = Ld::template bytes<A>(N), at_gate = at_x + Ld::template bytes<B>(N);
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ float red[2][2][16];
    const int tid = threadIdx.x;
    const bool post = KEPT || c.w_post, pre = KEPT || c.w_pre;
    const bool y8 = KEPT ? KEPT == 1 : c.y8.codes != nullptr, r8 = KEPT ? KEPT == 1 : c.r8.codes != nullptr;
    unsigned char *kept = smem;  // w_post, w_pre, the channel gate's factor
    unsigned char *ring = smem + (GATE == 1 ? 3 : 2) * kVector;
    auto in = [&](int i) { return FULL || tid * 8 + i * T * 8 < c.D; };

    auto fetch = [&](int64_t row, unsigned char *to) {
        if (row < c.rows) {
            const TA *y = static_cast<const TA *>(a.y) + row * a.ld_y;
            const TR *x = static_cast<const TR *>(a.x) + row * a.ld_x;
            const char *gate = static_cast<const char *>(c.gate) + row * c.ld_gate * (c.gf32 ? 4 : 2);
#pragma unroll
            for (int i = 0; i < C; ++i) {
                const int col = tid * 8 + i * T * 8;
                if (!in(i)) continue;
                Ld::template copy<A>(to + at_y, i, y, col, c.D, row * a.ld_y == 0);
                Ld::template copy<B>(to + at_x, i, x, col, c.D, row * a.ld_x == 0);
                if (GATE == 2) {
                    if (c.gf32) Ld::template copy<4>(to + at_gate, i, gate, col, c.D, row * c.ld_gate == 0);
                    else Ld::template copy<2>(to + at_gate, i, gate, col, c.D, row * c.ld_gate == 0);
                }
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    // Codes of a chunk, and their block's scale from one of its 16 lanes.
    auto keep = [&](const Ckpt &k, int64_t row, int i, const V8 &v) {
        const int col = tid * 8 + i * T * 8;
        int E;
        const uint2 q = encode8(v, E);
        if (!FULL && col / kQBlock * kQBlock >= c.D) return;
        __stcs(reinterpret_cast<uint2 *>(k.codes + row * k.ld_codes + col), q);
        if ((tid & 15) == 0) k.exps[(int64_t)(col / kQBlock) * k.ld_exps + row] = (uint8_t)E;
    };
    for (int k = 0; k + 1 < stages; ++k) fetch(blockIdx.x + (int64_t)k * gridDim.x, ring + k * stage_bytes);
    keep_vector<T, C>(kept, c.w_post, c.pf32, c.D, 0);
    keep_vector<T, C>(kept + kVector, c.w_pre, c.pf32, c.D, 0);
    if (GATE == 1) keep_vector<T, C>(kept + 2 * kVector, c.gate, c.gf32, c.D, c.sigmoid);

    int st = 0, flip = 0;
    for (int64_t row = blockIdx.x; row < c.rows; row += gridDim.x) {
        float gt = 1.f;
        if (GATE == 0 && c.gate_kind == ZERO1_GATE_TOKEN) gt = token_gate(c, row);
        // what this thread has read a row ago is filled again
        fetch(row + (int64_t)(stages - 1) * gridDim.x, ring + (st == 0 ? stages - 1 : st - 1) * stage_bytes);
        copies_wait(stages - 1);
        const unsigned char *b = ring + st * stage_bytes;
        V8 v[C];
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < C; ++i) {
            v[i] = in(i) ? Ld::take(b + at_y, i, static_cast<const TA *>(a.y) + row * a.ld_y) : splat8(0.f);
            if (post) s += dot8(v[i], v[i]);
        }
        float rs = 1.f;
        if (post) {
            rs = rstd_of(block_sum<T>(s, red[flip][0]), c);
            if (tid == 0) a.rstd_post[row] = rs;
        }
        s = 0.f;
        TR *r = static_cast<TR *>(a.r) + row * a.ld_r;
#pragma unroll
        for (int i = 0; i < C; ++i) {
            if (post) v[i] = mul8(v[i], rs);
            if (y8) keep(c.y8, row, i, v[i]);
            if (!in(i)) continue;
            if (post) v[i] = mul8(v[i], kept8<T, C>(kept, i));
            if (GATE == 1) {
                v[i] = mul8(v[i], kept8<T, C>(kept + 2 * kVector, i));
            } else if (GATE == 2) {
                V8 g = c.gf32 ? Ld::take(b + at_gate, i, static_cast<const float *>(c.gate) + row * c.ld_gate)
                              : Ld::take(b + at_gate, i, static_cast<const uint16_t *>(c.gate) + row * c.ld_gate);
                if (c.sigmoid) {
                    V8 slope;
                    logistic8(g, slope);
                }
                v[i] = mul8(v[i], g);
            }
            v[i] = fma8(v[i], c.alpha * gt, Ld::take(b + at_x, i, static_cast<const TR *>(a.x) + row * a.ld_x));
            Ld::put(r, tid * 8 + i * T * 8, c.D, v[i]);
            if (pre) s += dot8(v[i], v[i]);
        }
        if (pre) {
            rs = rstd_of(block_sum<T>(s, red[flip][1]), c);
            if (tid == 0) a.rstd_pre[row] = rs;
            TA *h = static_cast<TA *>(a.h) + row * a.ld_h;
#pragma unroll
            for (int i = 0; i < C; ++i) {
                v[i] = mul8(v[i], rs);
                if (r8) keep(c.r8, row, i, v[i]);
                if (in(i)) Ld::put(h, tid * 8 + i * T * 8, c.D, mul8(v[i], kept8<T, C>(kept + kVector, i)));
            }
        }
        flip ^= 1;
        if (++st == stages) st = 0;
    }
}

// Every resident block, one row at a time.
template <class TA, class TR, bool VEC>
int launch_fwd(const Common &c, const Fwd &a, int sms, cudaStream_t st)
{
    auto kernel = k_block_norm_fwd<TA, TR, VEC>;
    const int threads = row_threads(c.D);
    const int per_sm = blocks_per_sm(reinterpret_cast<const void *>(kernel), threads);
    const int64_t grid = c.rows < (int64_t)sms * per_sm ? c.rows : (int64_t)sms * per_sm;
    kernel<<<(unsigned)grid, threads, 0, st>>>(c, a);
    z1_note_launch(reinterpret_cast<const void *>(kernel), (int)grid, per_sm, threads, 0);
    return launch_status("block norm forward launch");
}

// One resident wave of staged blocks; false, with nothing launched, if a row
// does not fit.
template <class TA, class TR, int T, int C, int GATE, int KEPT, bool FULL, bool AL>
bool launch_fwd_staged(const Common &c, const Fwd &a, int sms, cudaStream_t st, int *rc)
{
    auto kernel = k_block_norm_fwd_staged<TA, TR, T, C, GATE, KEPT, FULL, AL>;
    using Ld = Row<T, AL>;
    constexpr int N = 8 * C * T, kept = (GATE == 1 ? 3 : 2) * N * 4;
    const int stage = Ld::template bytes<sizeof(TA)>(N) + Ld::template bytes<sizeof(TR)>(N) +
                      (GATE != 2 ? 0 : c.gf32 ? Ld::template bytes<4>(N) : Ld::template bytes<2>(N));
    const int stages = stages_that_fit(T, kept, stage);
    if (stages == 0) return false;
    const int smem = kept + stages * stage;
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = allow_smem(kernel, kSmemPerSm - 1024, done);
    if (e != cudaSuccess) {
        *rc = z1_fail(ZERO1_ECUDA, "block norm forward: %s", cudaGetErrorString(e));
        return true;
    }
    const int64_t wave = (int64_t)sms * (kOwnRegs / T);
    const int64_t grid = c.rows < wave ? c.rows : wave;
    kernel<<<(unsigned)grid, T, smem, st>>>(c, a, stages, stage);
    z1_note_launch(reinterpret_cast<const void *>(kernel), (int)grid, kOwnRegs / T, T, 0);
    *rc = launch_status("block norm forward launch");
    return true;
}

// The mixes in use are compiled apart (KEPT) for rows of exactly 8 C T columns; any
// other row takes the run-time mix.  us on the device, compiled apart and as a
// run-time mix, 33.6 million bf16 elements, without a gate and with a channel
// gate:
//   columns   with checkpoints         without
//   1024      56 / 69    60 / 69       44 / 51    45 / 52
//   2048      60 / 56    60 / 58       48 / 48    48 / 46
//   4096      57 / 58    58 / 62       46 / 46    45 / 44
//   8192      63 / 61    67 / 65       43 / 43    48 / 48
template <class TA, class TR>
bool forward_staged(const Common &c, const Fwd &a, bool vec, int sms, cudaStream_t st, int *rc)
{
    if (c.D > 8192) return false;
    if (c.gate_kind == ZERO1_GATE_FULL && !c.gvec) vec = false;
    const int codes = (c.y8.codes != nullptr) + (c.r8.codes != nullptr);
    const int kinds = !c.w_pre || !c.w_post ? 0 : codes == 2 ? 1 : codes == 0 ? 2 : 0;
    return pick_threads(c.D, [&](auto t, auto n) {
        constexpr int T = decltype(t)::value, C = decltype(n)::value;
        return pick_gate(c.gate_kind, [&](auto gate) {
            constexpr int G = decltype(gate)::value;
            if (!vec) return launch_fwd_staged<TA, TR, T, C, G, 0, false, false>(c, a, sms, st, rc);
            if constexpr (sizeof(TA) == 2 && !(T == 512 && C == 1)) {
                const int kept = c.D == 8 * C * T ? kinds : 0;
                if (kept == 1) return launch_fwd_staged<TA, TR, T, C, G, 1, true, true>(c, a, sms, st, rc);
                if (kept == 2) return launch_fwd_staged<TA, TR, T, C, G, 2, true, true>(c, a, sms, st, rc);
            }
            return launch_fwd_staged<TA, TR, T, C, G, 0, false, true>(c, a, sms, st, rc);
        });
    });
}

}  // namespace

template <class TA, class TR>
int z1bn::run_forward(const Common &c, const Fwd &a, bool vec, int sms, cudaStream_t st)
{
    int rc;
    if (forward_staged<TA, TR>(c, a, vec, sms, st, &rc)) return rc;
    return vec ? launch_fwd<TA, TR, true>(c, a, sms, st) : launch_fwd<TA, TR, false>(c, a, sms, st);
}
