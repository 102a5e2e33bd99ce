// zero1_clip.cu - the global gradient norm and clipping: over a list of tensors,
// and in the sharded step.
//
//   norm = sqrt(sum of g^2 over all gradients),  c = min(1, max_norm / (norm + 1e-6))
//
// Sums of squares: eight elements in fp32, up to sixteen such sums in fp32, the
// rest in doubles, in an order that sizes and alignment fix.  Eight squares that leave
// [2^-100, 2^100] (which fp32 would flush or overflow) are taken again, scaled by
// 2^100 or 2^-100: every finite gradient counts with about 24 bits.

#include <algorithm>
#include <vector>

#include "zero1_block.cuh"

namespace {

// ------------------------------------------------------- sums of squares ---

constexpr float kLow = 7.88860905e-31f, kHigh = 1.26765060e30f;  // 2^-100, 2^100

__device__ __forceinline__ float squares8(const float f[8])
{
    float a = __fmul_rn(f[0], f[0]), b = __fmul_rn(f[1], f[1]);
#pragma unroll
    for (int k = 2; k < 8; k += 2) {
        a = __fmaf_rn(f[k], f[k], a);
        b = __fmaf_rn(f[k + 1], f[k + 1], b);
    }
    return __fadd_rn(a, b);
}

struct SumSq {
    float near = 0.f;  // of squares in the usual range, since the last flush
    double sum = 0.0;

    __device__ __forceinline__ void add8(float f[8])
    {
        float p = squares8(f);
        if (p >= kLow && p <= kHigh) {
            near = __fadd_rn(near, p);
            return;
        }
        const float scale = p < kLow ? kHigh : kLow;  // (NaN and Inf take the second, and stay)
#pragma unroll
        for (int k = 0; k < 8; ++k) f[k] = __fmul_rn(f[k], scale);
        p = squares8(f);
        if (p == 0.f) return;  // eight zeros
        const double back = scale == kHigh ? 0x1p-200 : 0x1p200;
        sum = __fma_rn((double)p, back, sum);
    }
    __device__ __forceinline__ void add1(float f)
    {
        sum = __fma_rn((double)f, (double)f, sum);
    }
    // At the latest after sixteen calls of add8.
    __device__ __forceinline__ void flush()
    {
        sum = __dadd_rn(sum, (double)near);
        near = 0.f;
    }
};

__device__ __forceinline__ double warp_sum(double x)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x = __dadd_rn(x, __shfl_xor_sync(0xffffffffu, x, o));
    return x;
}

// The sum over the block, in thread 0.  `red` is free again after the next
// barrier.
__device__ __forceinline__ double block_sum(double x, double *red)
{
    const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    x = warp_sum(x);
    if (lane == 0) red[threadIdx.x >> 5] = x;
    __syncthreads();
    if (threadIdx.x < 32) x = warp_sum(lane < warps ? red[lane] : 0.0);
    return x;
}

// norm and c from the sum of squares; c is 1 where the norm is not finite.
struct Clip {
    double norm;
    float c;
    __device__ __forceinline__ Clip(double sumsq, double max_norm)
    {
        norm = __dsqrt_rn(sumsq);
        const double q = __ddiv_rn(max_norm, __dadd_rn(norm, 1e-6));
        c = q < 1.0 && isfinite(norm) ? __double2float_rn(q) : 1.f;
    }
};

// ------------------------------------------------------ lists of tensors ---

// Tensors per launch: their table travels in the kernel's arguments, of which a
// launch copies all, so that short lists take a smaller one.
constexpr int kGroup = 512, kShort = 48;
constexpr int kListBlock = 256;
constexpr int kUnroll = 4;      // vectors of 8 elements in flight per thread

// Elements of a chunk, the unit that blocks share a list out by.
constexpr int kChunkVecs = 256, kChunk = 8 * kChunkVecs;

struct Entry {
    const void *p;
    void *out;
    int64_t numel;
    int32_t first;   // chunk
    int16_t f32;
    int16_t head;    // elements before the first 16-byte boundary; -1: out lies otherwise, one element at a time
};
template <int N>
struct Table {
    int count, chunks;
    Entry e[N];
};
static_assert(sizeof(Table<kGroup>) + 64 <= 32764, "kernel arguments");

// Each block takes an equal, contiguous run of the list's chunks, piece by piece of
// a tensor, so that there is one sum over the block per piece and not per chunk (872
// million bf16 elements: 257 us, with chunks of 64 Ki elements in turn 285).
__host__ __device__ __forceinline__ int64_t first_chunk(int block, int grid, int chunks) { return (int64_t)block * chunks / grid; }
__host__ __device__ __forceinline__ int block_of(int chunk, int grid, int chunks)
{
    return (int)(((int64_t)(chunk + 1) * grid - 1) / chunks);
}

template <int N>
__device__ __forceinline__ int entry_of(const Table<N> &t, int chunk)
{
    int lo = 0, hi = t.count - 1;  // the last entry whose first chunk is at most this (empty tensors have none)
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (t.e[mid].first <= chunk) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}
template <int N>
__device__ __forceinline__ int end_of(const Table<N> &t, int k)
{
    return k + 1 < t.count ? t.e[k + 1].first : t.chunks;
}

// Calls vecs(v, end) for chunks [b, e) of a tensor, a thread's vectors v, v +
// kListBlock and so on (kUnroll of them, below end) at a time, and one(element) for
// those before the first vector and after the last, with the tensor's first and last
// chunk.  FROM_END: the last vectors first.
template <bool FROM_END, class Vecs, class One>
__device__ __forceinline__ void walk_chunks(const Entry &t, int64_t b, int64_t e, int64_t chunks, Vecs &&vecs, One &&one)
{
    constexpr int64_t kStep = kUnroll * kListBlock;
    const int64_t nvec = (t.numel - t.head) / 8, begin = min(nvec, b * kChunkVecs), end = min(nvec, e * kChunkVecs);
    if (FROM_END)
        for (int64_t v = begin + (end - begin + kStep - 1) / kStep * kStep - kStep; v >= begin; v -= kStep) vecs(v + threadIdx.x, end);
    else
        for (int64_t v = begin; v < end; v += kStep) vecs(v + threadIdx.x, end);
    if (b == 0 && (int)threadIdx.x < t.head) one(threadIdx.x);
    if (e == chunks) {
        const int64_t j = t.head + nvec * 8 + threadIdx.x;
        if (j < t.numel) one(j);
    }
}

template <class T>
__device__ __forceinline__ void sum_chunks(const Entry &t, int64_t b, int64_t e, int64_t chunks, SumSq &s)
{
    const T *p = static_cast<const T *>(t.p);
    int since = 0;
    walk_chunks<false>(
        t, b, e, chunks,
        [&](int64_t v, int64_t end) {
            Raw8<T> q[kUnroll];
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                const int64_t at = v + u * kListBlock;
                if (at < end) q[u].load(p + t.head + at * 8);
                else q[u].zero();
            }
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                float f[8];
                q[u].get(f);
                s.add8(f);
            }
            if (++since == 4) {
                s.flush();
                since = 0;
            }
        },
        [&](int64_t j) { s.add1(ld1(p + j)); });
    s.flush();
}

// A piece is known by its block's number and its tensor's: with each step along the
// list one of the two grows, so their sum is a place of its own.
template <int N>
__global__ void __launch_bounds__(kListBlock, 4) k_list_sumsq(const __grid_constant__ Table<N> t, double *part)
{
    wait_prior_grid();
    let_next_grid_start();
    __shared__ double red[2][32];
    int flip = 0;
    const int end = (int)first_chunk(blockIdx.x + 1, gridDim.x, t.chunks);
    int c = (int)first_chunk(blockIdx.x, gridDim.x, t.chunks);
    for (int k = entry_of(t, c); c < end; ++k) {
        const Entry &e = t.e[k];
        const int next = min(end, end_of(t, k));
        if (next <= c) continue;  // (an empty tensor)
        SumSq s;
        if (e.f32) sum_chunks<float>(e, c - e.first, next - e.first, end_of(t, k) - e.first, s);
        else sum_chunks<uint16_t>(e, c - e.first, next - e.first, end_of(t, k) - e.first, s);
        const double x = block_sum(s.sum, red[flip]);
        if (threadIdx.x == 0) part[blockIdx.x + k] = x;
        flip ^= 1;
        c = next;
    }
}

// Adds the pieces: a warp to a tensor, lanes in strides and then joined in order;
// tensors in order of their warps.  `grid`: of the kernel above.
template <int N>
__global__ void __launch_bounds__(1024) k_list_finish(const __grid_constant__ Table<N> t, int grid, const double *part, double *sumsq,
                                                      float *norms, int add)
{
    wait_prior_grid();
    let_next_grid_start();
    __shared__ double red[32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    double total = 0.0;
    for (int k = warp; k < t.count; k += warps) {
        double x = 0.0;
        const int chunks = end_of(t, k) - t.e[k].first;
        if (chunks > 0) {
            const int b = block_of(t.e[k].first, grid, t.chunks), e = block_of(end_of(t, k) - 1, grid, t.chunks);
            for (int q = b; q <= e; q += 4 * 32) {
                double v[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) v[j] = q + 32 * j + lane <= e ? part[q + 32 * j + lane + k] : 0.0;
#pragma unroll
                for (int j = 0; j < 4; ++j) x = __dadd_rn(x, v[j]);
            }
            x = warp_sum(x);
        }
        if (norms && lane == 0) norms[k] = __double2float_rn(__dsqrt_rn(x));
        total = __dadd_rn(total, x);
    }
    const double x = block_sum(lane == 0 ? total : 0.0, red);
    if (threadIdx.x == 0) *sumsq = add ? __dadd_rn(*sumsq, x) : x;
}

// Eight elements as they lie in memory, by plain loads: what is read here may be
// written here.
template <class T>
struct Plain8;
template <>
struct Plain8<uint16_t> {
    uint4 q;
    __device__ __forceinline__ void load(const uint16_t *p) { q = *reinterpret_cast<const uint4 *>(p); }
    __device__ __forceinline__ void get(float f[8]) const { unpack8(q, f); }
};
template <>
struct Plain8<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float *p)
    {
        a = reinterpret_cast<const float4 *>(p)[0];
        b = reinterpret_cast<const float4 *>(p)[1];
    }
    __device__ __forceinline__ void get(float f[8]) const
    {
        f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w; f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    }
};

template <class T>
__device__ __forceinline__ void clip_chunks(const Entry &t, int64_t b, int64_t e, int64_t chunks, float c)
{
    const T *p = static_cast<const T *>(t.p);
    T *o = static_cast<T *>(t.out);
    if (t.head < 0) {
        const int64_t end = min(t.numel, e * kChunk);
        for (int64_t j = b * kChunk + threadIdx.x; j < end; j += kListBlock) st1(o + j, __fmul_rn(ld1(p + j), c));
        return;
    }
    // from the end: what the sum of squares read last is still in L2
    walk_chunks<true>(
        t, b, e, chunks,
        [&](int64_t v, int64_t end) {
            Plain8<T> q[kUnroll];
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                const int64_t at = v + u * kListBlock;
                if (at < end) q[u].load(p + t.head + at * 8);
            }
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                const int64_t at = v + u * kListBlock;
                if (at >= end) continue;
                float f[8];
                q[u].get(f);
#pragma unroll
                for (int j = 0; j < 8; ++j) f[j] = __fmul_rn(f[j], c);
                store8(o + t.head + at * 8, f);
            }
        },
        [&](int64_t j) { st1(o + j, __fmul_rn(ld1(p + j), c)); });
}

template <int N>
__global__ void __launch_bounds__(kListBlock, 4)
k_list_clip(const __grid_constant__ Table<N> t, const double *sumsq, double max_norm, float *norm, int in_place)
{
    wait_prior_grid();
    let_next_grid_start();
    __shared__ float coef;
    if (threadIdx.x == 0) {
        const Clip c(*sumsq, max_norm);
        coef = c.c;
        if (norm && blockIdx.x == 0) *norm = __double2float_rn(c.norm);
    }
    __syncthreads();
    const float c = coef;
    if (in_place && c == 1.f) return;
    int end = (int)first_chunk(blockIdx.x + 1, gridDim.x, t.chunks);
    const int begin = (int)first_chunk(blockIdx.x, gridDim.x, t.chunks);
    for (int k = end > begin ? entry_of(t, end - 1) : 0; end > begin; --k) {
        const Entry &e = t.e[k];
        const int from = max(begin, e.first);
        if (from >= end) continue;  // (an empty tensor)
        if (e.f32) clip_chunks<float>(e, from - e.first, end - e.first, end_of(t, k) - e.first, c);
        else clip_chunks<uint16_t>(e, from - e.first, end - e.first, end_of(t, k) - e.first, c);
        end = from;
    }
}

// --------------------------------------------------------- sharded step ----

constexpr int kShardParts = 2048;  // blocks of k_shard_sumsq at most

// Sum of squares of g = (rank-order sum of the replicas) * inv over the real
// elements; the sums are kept when `sums` is not NULL (+0 on padding).  A stream
// of 2M bytes per element, and 4 more for the sums.
template <int MT>
__global__ void __launch_bounds__(kBlock, MT > 0 ? 4 : 3)
k_shard_sumsq(const __grid_constant__ GradPtrs g, int M, const Walk w, float inv, float *sums, double *part)
{
    wait_prior_grid();
    let_next_grid_start();
    __shared__ double red[32];
    const int64_t tid = grid_tid(), nthr = grid_threads();
    SumSq acc;
    int since = 0;
    for (int64_t i = tid; i < w.nvec; i += nthr) {
        const int64_t j = w.head + i * kVec;
        float s[kVec];
        sum8<MT>(g, M, j, s);
        if (sums) st_stream8(sums + j, s, w.w32);
#pragma unroll
        for (int k = 0; k < kVec; ++k) s[k] = __fmul_rn(s[k], inv);
        acc.add8(s);
        if (++since == 16) {
            acc.flush();
            since = 0;
        }
    }
    acc.flush();
    const int64_t ns = w.L - w.nvec * kVec;
    for (int64_t q = tid; q < ns; q += nthr) {
        const int64_t j = scalar_index(w, q);
        float s = 0.f;
        if (j < w.nv) {
            s = sum1(g, M, j);
            acc.add1(__fmul_rn(s, inv));
        }
        if (sums) sums[j] = s;
    }
    const double x = block_sum(acc.sum, red);
    if (threadIdx.x == 0) part[blockIdx.x] = x;
}

__global__ void __launch_bounds__(256) k_shard_finish(const double *part, int parts, double *sumsq, int add)
{
    wait_prior_grid();
    let_next_grid_start();
    __shared__ double red[32];
    double x = 0.0, v[kShardParts / 256];
#pragma unroll
    for (int j = 0; j < kShardParts / 256; ++j) {
        const int c = threadIdx.x + 256 * j;
        v[j] = c < parts ? part[c] : 0.0;
    }
#pragma unroll
    for (int j = 0; j < kShardParts / 256; ++j) x = __dadd_rn(x, v[j]);
    x = block_sum(x, red);
    if (threadIdx.x == 0) *sumsq = add ? __dadd_rn(*sumsq, x) : x;
}

struct State {
    const float *w, *m, *v;
    float *w_out, *m_out, *v_out;
    uint16_t *params;
};

__device__ __forceinline__ void clipped8(float s[kVec], const F8 &w, const F8 &m, const F8 &v, int64_t j, const State &t,
                                         const Z1Consts &c, float coef, bool wide)
{
    float ww[kVec], mm[kVec], vv[kVec];
    unpack_f8(w, ww);
    unpack_f8(m, mm);
    unpack_f8(v, vv);
#pragma unroll
    for (int k = 0; k < kVec; ++k) adamw1(__fmul_rn(__fmul_rn(s[k], c.inv), coef), c, ww[k], mm[k], vv[k]);
    st_stream8(t.w_out + j, ww, wide);
    st_stream8(t.m_out + j, mm, wide);
    st_stream8(t.v_out + j, vv, wide);
    __stcs(reinterpret_cast<uint4 *>(t.params + j), make_uint4(pack_bf16x2(ww[0], ww[1]), pack_bf16x2(ww[2], ww[3]),
                                                              pack_bf16x2(ww[4], ww[5]), pack_bf16x2(ww[6], ww[7])));
}

// The fused step's update with g = (sum * inv) * c, c from the sum of squares;
// nothing is written but the flag if that is not finite.  KEPT: the sums come
// from the first pass, 4 bytes per element, instead of the M gradients again.
template <int MT, bool KEPT>
__global__ void __launch_bounds__(kBlock, MT == 0 && !KEPT ? 3 : 4)
k_step_clipped(const __grid_constant__ GradPtrs g, int M, const float *sums, const State t, const Walk w, const Z1Consts c,
               const double *sumsq, double max_norm, float *norm, uint32_t *flag, int wide)
{
    wait_prior_grid();
    let_next_grid_start();
    __shared__ float shared_coef;
    __shared__ int bad;
    if (threadIdx.x == 0) {
        const double q = *sumsq;
        const Clip k(q, max_norm);
        shared_coef = k.c;
        bad = !isfinite(q);
        if (blockIdx.x == 0) {
            if (norm) *norm = __double2float_rn(k.norm);
            if (bad && flag) atomicOr(flag, 1u);
        }
    }
    __syncthreads();
    if (bad) return;
    const float coef = shared_coef;
    const int64_t tid = grid_tid(), nthr = grid_threads();
    const bool w32 = w.w32 != 0;
    // from the end: what the first pass read or wrote last is still in L2
    for (int64_t i = w.nvec - 1 - tid; i >= 0; i -= nthr) {
        const int64_t j = w.head + i * kVec;
        float s[kVec];
        if constexpr (KEPT) {
            const F8 q = ld_cs8(sums + j, w32), sw = ld_state8(t.w + j, w32), sm = ld_state8(t.m + j, w32), sv = ld_state8(t.v + j, w32);
            unpack_f8(q, s);
            clipped8(s, sw, sm, sv, j, t, c, coef, wide);
        } else if constexpr (MT > 0) {
            uint4 q[MT];
#pragma unroll
            for (int r = 0; r < MT; ++r) q[r] = ld_stream_u4(g.p[r] + j);
            const F8 sw = ld_state8(t.w + j, w32), sm = ld_state8(t.m + j, w32), sv = ld_state8(t.v + j, w32);
            unpack8(q[0], s);
#pragma unroll
            for (int r = 1; r < MT; ++r) add8(q[r], s);
            clipped8(s, sw, sm, sv, j, t, c, coef, wide);
        } else {
            const F8 sw = ld_state8(t.w + j, w32), sm = ld_state8(t.m + j, w32), sv = ld_state8(t.v + j, w32);
            sum8<0>(g, M, j, s);
            clipped8(s, sw, sm, sv, j, t, c, coef, wide);
        }
    }
    const int64_t ns = w.L - w.nvec * kVec;
    for (int64_t q = tid; q < ns; q += nthr) {
        const int64_t j = scalar_index(w, q);
        float s = 0.f;
        if (j < w.nv) {
            if constexpr (KEPT) s = sums[j];
            else s = sum1(g, M, j);
        }
        float ww = t.w[j], mm = t.m[j], vv = t.v[j];
        adamw1(__fmul_rn(__fmul_rn(s, c.inv), coef), c, ww, mm, vv);
        t.w_out[j] = ww;
        t.m_out[j] = mm;
        t.v_out[j] = vv;
        if (j < w.nv) t.params[j] = to_bf16(ww);
    }
}

// ------------------------------------------------------------ host side ----

// The clipped step's launch shapes: on large ranges the fused step's for M (M = 8, 124
// million elements: 768 us against 811 at full occupancy, 770 against 842 in place), and
// for kept sums three blocks of 192 per SM (551 us; two of 256 552, five of 128 586,
// four of 256 586, six of 128 615; in place 560, 567, 665, 641, 656); at full occupancy
// on small ones.
constexpr int64_t kSmallVecs = 1 << 18;
constexpr Shape kKeptShape{1, 3, 192};
static_assert(shape_ok(kKeptShape), "launch shape");

int64_t chunks_of(const zero1_tensor_t &t) { return (t.numel + kChunk - 1) / kChunk; }

int check_list(const zero1_tensor_t *t, int32_t count, const char *call, const char *what, int64_t *total)
{
    if (count < 0 || (count > 0 && !t)) return z1_fail(ZERO1_EINVAL, "%s: %d %s, list %s", call, count, what, t ? "given" : "NULL");
    *total = 0;
    for (int k = 0; k < count; ++k) {
        int rc = check_dtype(t[k].dtype, call, "dtype");
        if (rc != ZERO1_OK) return rc;
        if (t[k].numel < 0) return z1_fail(ZERO1_EINVAL, "%s: %s[%d] has %lld elements", call, what, k, (long long)t[k].numel);
        if (t[k].numel > (INT64_C(1) << 40) || (*total += t[k].numel) > (INT64_C(1) << 40))
            return z1_fail(ZERO1_ERANGE, "%s: more than 2^40 elements", call);
        if (t[k].numel == 0) continue;
        if (!t[k].data) return z1_fail(ZERO1_EINVAL, "%s: %s[%d] is NULL", call, what, k);
        if ((rc = check_natural(t[k].data, esize(t[k].dtype), what)) != ZERO1_OK) return rc;
    }
    return ZERO1_OK;
}

// Groups of at most kGroup tensors, with their chunks.  outs may be NULL.  `run`
// launches one group.
template <int N, class F>
int each_group_of(const zero1_tensor_t *t, const zero1_tensor_t *outs, int32_t count, F &&run)
{
    for (int at = 0; at < count;) {
        Table<N> tab;
        int64_t chunks = 0;
        int n = 0;
        for (; at + n < count && n < N && chunks <= INT32_MAX / 2; ++n) {
            const zero1_tensor_t &x = t[at + n];
            const int es = esize(x.dtype);
            Entry &e = tab.e[n];
            e.p = x.data;
            e.out = outs ? outs[at + n].data : x.data;
            e.numel = x.numel;
            e.first = (int32_t)chunks;
            e.f32 = x.dtype == ZERO1_DTYPE_F32;
            const int64_t head = (16 - ((uintptr_t)x.data & 15)) % 16 / es;
            e.head = (int16_t)(head < x.numel ? head : x.numel);
            if (outs && (((uintptr_t)e.out ^ (uintptr_t)e.p) & 15)) e.head = -1;
            chunks += chunks_of(x);
        }
        tab.count = n;
        tab.chunks = (int)chunks;
        const int rc = run(tab, at);
        if (rc != ZERO1_OK) return rc;
        at += n;
    }
    return ZERO1_OK;
}

template <class F>
int each_group(const zero1_tensor_t *t, const zero1_tensor_t *outs, int32_t count, F &&run)
{
    return count <= kShort ? each_group_of<kShort>(t, outs, count, run) : each_group_of<kGroup>(t, outs, count, run);
}

// Blocks per SM of the list kernels (872 million bf16 elements: sums of squares 257 us
// with four, 281 with three, 354 with two; clipping to other tensors 542, 530 and 586).
constexpr int kSumsqWave = 4, kClipWave = 3;

int list_grid(const void *kernel, int chunks, int wave, int sms)
{
    const int64_t most = (int64_t)sms * wave;
    const int grid = chunks < most ? (chunks < 1 ? 1 : chunks) : (int)most;
    z1_note_launch(kernel, grid, wave, kListBlock, 0);
    return grid;
}

template <int N>
auto sumsq_of(const Table<N> &)
{
    return k_list_sumsq<N>;
}
template <int N>
auto finish_of(const Table<N> &)
{
    return k_list_finish<N>;
}
template <int N>
auto clip_of(const Table<N> &)
{
    return k_list_clip<N>;
}

// EINVAL if two of the extents share a byte.
int check_apart(std::vector<Extent> &x, const char *call)
{
    bool sorted = true;
    for (size_t k = 1; k < x.size() && sorted; ++k) sorted = (uintptr_t)x[k - 1].p + x[k - 1].bytes <= (uintptr_t)x[k].p;
    if (sorted) return ZERO1_OK;
    std::sort(x.begin(), x.end(), [](const Extent &a, const Extent &b) { return (uintptr_t)a.p < (uintptr_t)b.p; });
    for (size_t k = 1; k < x.size(); ++k)
        if (overlap(x[k - 1], x[k])) return z1_fail(ZERO1_EINVAL, "%s: %s and %s overlap", call, x[k - 1].what, x[k].what);
    return ZERO1_OK;
}

// The outputs must lie apart, and apart from every input but their own.
int check_outs(const zero1_tensor_t *t, const zero1_tensor_t *outs, int32_t count, const double *sumsq, const float *norm, const char *call)
{
    try {
        std::vector<Extent> w;
        w.reserve((size_t)count * 2 + 2);
        auto push = [&](const zero1_tensor_t &x, const char *what) {
            if (x.numel > 0) w.push_back(Extent{x.data, x.numel * esize(x.dtype), what});
        };
        for (int k = 0; k < count; ++k) push(outs[k], "an output");
        w.push_back(Extent{sumsq, 8, "sumsq"});
        if (norm) w.push_back(Extent{norm, 4, "norm"});
        const size_t written = w.size();
        int rc = check_apart(w, call);
        if (rc != ZERO1_OK || outs == t) return rc;
        // inputs that are not their own output, among the (now sorted or ascending) outputs
        std::sort(w.begin(), w.end(), [](const Extent &a, const Extent &b) { return (uintptr_t)a.p < (uintptr_t)b.p; });
        for (int k = 0; k < count; ++k) {
            if (t[k].numel == 0) continue;
            const Extent in{t[k].data, t[k].numel * esize(t[k].dtype), "a tensor"};
            size_t lo = 0, hi = written;  // the first output that ends behind the tensor's start
            while (lo < hi) {
                const size_t mid = (lo + hi) / 2;
                if ((uintptr_t)w[mid].p + w[mid].bytes <= (uintptr_t)in.p) lo = mid + 1;
                else hi = mid;
            }
            if (lo < written && overlap(w[lo], in) && !(t[k].data == outs[k].data && w[lo].p == in.p && w[lo].bytes == in.bytes))
                return z1_fail(ZERO1_EINVAL, "%s: tensors[%d] and %s that is not its own overlap", call, k, w[lo].what);
        }
        return ZERO1_OK;
    } catch (const std::bad_alloc &) {
        return z1_fail(ZERO1_ERANGE, "%s: no host memory for a list of %d tensors", call, count);
    }
}

int check_max_norm(float max_norm, const char *call)
{
    if (!(max_norm > 0.f) || !std::isfinite(max_norm)) return z1_fail(ZERO1_EINVAL, "%s: max_norm must be finite and > 0", call);
    return ZERO1_OK;
}

int check_scalar(const void *p, int es, bool needed, const char *call, const char *what)
{
    if (!p) return needed ? z1_fail(ZERO1_EINVAL, "%s: %s is NULL", call, what) : ZERO1_OK;
    return check_natural(p, es, what);
}

// Doubles for the pieces of any group of a list: fewer than its blocks and its
// tensors together.
int64_t most_pieces(int32_t count, int sms) { return (int64_t)sms * kSumsqWave + (count < kGroup ? count : kGroup); }

}  // namespace

extern "C" int zero1_grad_sumsq_workspace(const zero1_tensor_t *tensors, int32_t count, int64_t *bytes)
{
    const char *call = "gradient norm workspace";
    if (!bytes) return z1_fail(ZERO1_EINVAL, "%s: bytes is NULL", call);
    int64_t total;
    const int rc = check_list(tensors, count, call, "tensors", &total);
    if (rc != ZERO1_OK) return rc;
    const int sms = sm_count();
    if (sms == 0) return z1_fail(ZERO1_ECUDA, "%s: no CUDA device", call);
    *bytes = 8 * most_pieces(count, sms);
    return ZERO1_OK;
}

extern "C" int zero1_grad_sumsq(const zero1_tensor_t *tensors, int32_t count, double *sumsq, float *norms, int32_t accumulate,
                                void *workspace, int64_t workspace_bytes, zero1_stream_t stream)
{
    Z1Trace trace("zero1_grad_sumsq");
    const char *call = "gradient norm";
    int64_t total;
    int rc;
    if ((rc = check_list(tensors, count, call, "tensors", &total)) || (rc = check_scalar(sumsq, 8, true, call, "sumsq")) ||
        (rc = check_scalar(norms, 4, false, call, "norms")))
        return rc;
    const Extent out[] = {{sumsq, 8, "sumsq"}, {norms, 4 * (int64_t)count, "norms"}, {workspace, workspace_bytes, "the workspace"}};
    for (int a = 0; a < 3; ++a) {
        for (int b = a + 1; b < 3; ++b)
            if (overlap(out[a], out[b])) return z1_fail(ZERO1_EINVAL, "%s: %s and %s overlap", call, out[a].what, out[b].what);
        for (int k = 0; k < count; ++k)
            if (overlap(out[a], Extent{tensors[k].data, tensors[k].numel * esize(tensors[k].dtype), ""}))
                return z1_fail(ZERO1_EINVAL, "%s: %s and tensors[%d] overlap", call, out[a].what, k);
    }
    const int sms = sm_count();
    if (sms == 0) return z1_fail(ZERO1_ECUDA, "%s: no CUDA device", call);
    const int64_t need = 8 * most_pieces(count, sms);
    if (!workspace || workspace_bytes < need)
        return z1_fail(ZERO1_EINVAL, "%s: workspace of %lld bytes, needs %lld", call, (long long)(workspace ? workspace_bytes : 0),
                       (long long)need);
    if ((uintptr_t)workspace & 7) return z1_fail(ZERO1_EALIGN, "%s: the workspace is not 8-byte aligned", call);
    if (in_host_memory(workspace)) return z1_fail(ZERO1_EINVAL, "%s: the workspace must be device memory", call);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    double *part = static_cast<double *>(workspace);
    auto finish = [&](const auto &tab, int at, int grid) -> int {
        const cudaError_t e = launch_after(finish_of(tab), dim3(1), tab.count <= 8 ? 256 : 1024, 0, st, tab, grid, (const double *)part, sumsq,
                                           norms ? norms + at : nullptr, accumulate || at > 0 ? 1 : 0);
        return e == cudaSuccess ? ZERO1_OK : pdl_fail(e, call);
    };
    if (count == 0) {
        Table<kShort> none;
        none.count = none.chunks = 0;
        return finish(none, 0, 1);
    }
    return each_group(tensors, nullptr, count, [&](const auto &tab, int at) -> int {
        int grid = 1;
        if (tab.chunks > 0) {
            const auto kernel = sumsq_of(tab);
            grid = list_grid(reinterpret_cast<const void *>(kernel), tab.chunks, kSumsqWave, sms);
            const cudaError_t e = launch_after(kernel, dim3(grid), kListBlock, 0, st, tab, part);
            if (e != cudaSuccess) return pdl_fail(e, call);
        }
        return finish(tab, at, grid);
    });
}

extern "C" int zero1_grad_clip(const zero1_tensor_t *tensors, const zero1_tensor_t *outs, int32_t count, const double *sumsq,
                               float max_norm, float *norm, zero1_stream_t stream)
{
    Z1Trace trace("zero1_grad_clip");
    const char *call = "gradient clipping";
    int64_t total;
    int rc;
    if ((rc = check_list(tensors, count, call, "tensors", &total)) || (rc = check_scalar(sumsq, 8, true, call, "sumsq")) ||
        (rc = check_scalar(norm, 4, false, call, "norm")) || (rc = check_max_norm(max_norm, call)))
        return rc;
    if (outs) {
        int64_t same;
        if ((rc = check_list(outs, count, call, "outs", &same)) != ZERO1_OK) return rc;
        for (int k = 0; k < count; ++k)
            if (outs[k].numel != tensors[k].numel || outs[k].dtype != tensors[k].dtype)
                return z1_fail(ZERO1_EINVAL, "%s: outs[%d] is not like tensors[%d]", call, k, k);
    }
    if ((rc = check_outs(tensors, outs ? outs : tensors, count, sumsq, norm, call)) != ZERO1_OK) return rc;
    const int sms = sm_count();
    if (sms == 0) return z1_fail(ZERO1_ECUDA, "%s: no CUDA device", call);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    auto run = [&](const auto &tab, int at) -> int {
        const auto kernel = clip_of(tab);
        const int grid = list_grid(reinterpret_cast<const void *>(kernel), tab.chunks, kClipWave, sms);
        const cudaError_t e = launch_after(kernel, dim3(grid), kListBlock, 0, st, tab, sumsq, (double)max_norm,
                                           at == 0 ? norm : nullptr, outs ? 0 : 1);
        return e == cudaSuccess ? ZERO1_OK : pdl_fail(e, call);
    };
    if (count == 0) {
        Table<kShort> none;
        none.count = none.chunks = 0;
        return norm ? run(none, 0) : ZERO1_OK;
    }
    return each_group(tensors, outs, count, run);
}

extern "C" int zero1_shard_grad_sumsq_workspace(int64_t *bytes)
{
    if (!bytes) return z1_fail(ZERO1_EINVAL, "shard gradient norm workspace: bytes is NULL");
    *bytes = 8 * kShardParts;
    return ZERO1_OK;
}

extern "C" int zero1_shard_grad_sumsq(const zero1_plan_t *plan, int32_t shard_begin, int32_t shard_end, const void *const *grads,
                                      const zero1_adamw_t *hp, double *sumsq, float *sums, int32_t accumulate, void *workspace,
                                      int64_t workspace_bytes, zero1_stream_t stream)
{
    Z1Trace trace("zero1_shard_grad_sumsq");
    const char *call = "shard gradient norm";
    Z1Range r;
    int rc = z1_range(plan, shard_begin, shard_end, &r);
    Z1Consts c;
    if (rc != ZERO1_OK || (rc = z1_adamw_constants(hp, plan->M, &c))) return rc;
    GradPtrs g{};
    if (r.nv > 0 && (rc = load_grads(plan, grads, &g, call)) != ZERO1_OK) return rc;
    if ((rc = check_scalar(sumsq, 8, true, call, "sumsq")) || (rc = check_scalar(sums, 4, false, call, "sums"))) return rc;
    const Extent out[] = {{sumsq, 8, "sumsq"}, {sums, r.L * 4, "sums"}, {workspace, 8 * kShardParts, "the workspace"}};
    if ((rc = check_disjoint(out, 3, g, plan->M, r.nv, call)) != ZERO1_OK) return rc;
    if (!workspace || workspace_bytes < 8 * kShardParts)
        return z1_fail(ZERO1_EINVAL, "%s: workspace of %lld bytes, needs %d", call, (long long)(workspace ? workspace_bytes : 0),
                       8 * kShardParts);
    if ((uintptr_t)workspace & 7) return z1_fail(ZERO1_EALIGN, "%s: the workspace is not 8-byte aligned", call);
    if (in_host_memory(workspace)) return z1_fail(ZERO1_EINVAL, "%s: the workspace must be device memory", call);
    ArrayRef arr[ZERO1_MAX_REPLICAS + 1];
    int n = 0;
    if (sums) arr[n++] = {sums, 4};
    for (int k = 0; k < plan->M; ++k) arr[n++] = {g.p[k], 2};
    const Walk w = make_walk(r.L, r.nv, arr, n);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    double *part = static_cast<double *>(workspace);
    const int M = plan->M;
    cudaError_t e = cudaSuccess;
    int grid = 0;
    dispatch_m(M, [&](auto mt) {
        constexpr int MT = decltype(mt)::value;
        grid = std::min(grid_for(k_shard_sumsq<MT>, w), kShardParts);
        e = launch_pdl(k_shard_sumsq<MT>, grid, kBlock, st, g, M, w, c.inv, sums, part);
    });
    if (e != cudaSuccess) return pdl_fail(e, call);
    e = launch_pdl(k_shard_finish, 1, 256, st, (const double *)part, grid, sumsq, accumulate ? 1 : 0);
    if (e != cudaSuccess) return pdl_fail(e, call);
    return launch_status(call);
}

extern "C" int zero1_step_clipped(const zero1_plan_t *plan, int32_t shard_begin, int32_t shard_end, const void *const *grads,
                                  const float *sums, const float *master, const float *m, const float *v, float *master_out,
                                  float *m_out, float *v_out, void *params, const zero1_adamw_t *hp, const double *sumsq,
                                  float max_norm, float *norm, uint32_t *overflow_flag, zero1_stream_t stream)
{
    Z1Trace trace("zero1_step_clipped");
    const char *call = "clipped step";
    Z1Range r;
    int rc = z1_range(plan, shard_begin, shard_end, &r);
    Z1Consts c;
    if (rc != ZERO1_OK || (rc = z1_adamw_constants(hp, plan->M, &c)) || (rc = check_max_norm(max_norm, call))) return rc;
    if (!master || !m || !v || !master_out || !m_out || !v_out)
        return z1_fail(ZERO1_EINVAL, "%s: master, m, v and where they go must be non-NULL", call);
    if (r.nv > 0 && !params) return z1_fail(ZERO1_EINVAL, "%s: params must be non-NULL when the range holds parameters", call);
    GradPtrs g{};
    if (r.nv > 0 && !sums && (rc = load_grads(plan, grads, &g, call)) != ZERO1_OK) return rc;
    const int M = sums ? 0 : plan->M;  // gradient buffers that are read
    const float *const in[] = {master, m, v};
    float *const to[] = {master_out, m_out, v_out};
    const char *const names[] = {"master", "m", "v"}, *const names_out[] = {"master_out", "m_out", "v_out"};
    for (int k = 0; k < 3; ++k)
        if ((rc = check_natural(in[k], 4, names[k])) || (rc = check_natural(to[k], 4, names_out[k]))) return rc;
    if ((rc = check_natural(params, 2, "params")) || (rc = check_scalar(sums, 4, false, call, "sums")) ||
        (rc = check_scalar(sumsq, 8, true, call, "sumsq")) || (rc = check_scalar(norm, 4, false, call, "norm")) ||
        (rc = check_scalar(overflow_flag, 4, false, call, "overflow_flag")))
        return rc;
    const Extent out[] = {{master_out, r.L * 4, "master_out"}, {m_out, r.L * 4, "m_out"}, {v_out, r.L * 4, "v_out"},
                          {params, r.nv * 2, "params"}, {norm, 4, "norm"}, {overflow_flag, 4, "overflow_flag"}};
    if ((rc = check_disjoint(out, 6, g, M, r.nv, call)) != ZERO1_OK) return rc;
    const Extent rest[] = {{master, r.L * 4, "master"}, {m, r.L * 4, "m"}, {v, r.L * 4, "v"}, {sums, r.L * 4, "sums"}, {sumsq, 8, "sumsq"}};
    for (int o = 0; o < 6; ++o)
        for (int k = 0; k < 5; ++k)
            if (overlap(out[o], rest[k]) && !(o == k && o < 3 && out[o].p == rest[k].p))
                return z1_fail(ZERO1_EINVAL, "%s: %s and %s overlap", call, out[o].what, rest[k].what);
    ArrayRef arr[ZERO1_MAX_REPLICAS + 8] = {{master, 4}, {m, 4}, {v, 4}, {master_out, 4}, {m_out, 4}, {v_out, 4}, {params, 2}};
    int n = 7;
    if (sums) arr[n++] = {sums, 4};
    for (int k = 0; k < M; ++k) arr[n++] = {g.p[k], 2};
    const Walk w = make_walk(r.L, r.nv, arr, n);
    const State t{master, m, v, master_out, m_out, v_out, static_cast<uint16_t *>(params)};
    const int wide = w.w32 && (kWideStoresInPlace || master_out != master);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e = cudaSuccess;
    if (sums) {
        auto kernel = k_step_clipped<1, true>;
        const bool small = w.nvec <= kSmallVecs;
        const int block = small ? kBlock : kKeptShape.block;
        e = launch_pdl(kernel, grid_for(kernel, w, small ? 0 : kKeptShape.per_sm, block), block, st, g, 1, sums, t, w, c, sumsq, (double)max_norm, norm, overflow_flag, wide);
    } else {
        dispatch_m(M, [&](auto mt) {
            constexpr int MT = decltype(mt)::value;
            auto kernel = k_step_clipped<MT, false>;
            const bool small = w.nvec <= kSmallVecs || MT == 0;
            const int block = small ? kBlock : fused_shape(MT).block;
            e = launch_pdl(kernel, grid_for(kernel, w, small ? 0 : fused_shape(MT).per_sm, block), block, st, g, M, sums, t, w, c, sumsq, (double)max_norm, norm, overflow_flag, wide);
        });
    }
    if (e != cudaSuccess) return pdl_fail(e, call);
    return launch_status(call);
}
