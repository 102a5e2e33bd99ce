// zero1_block.cuh - helpers shared by the training-block operators: typed
// 8-element loads and stores, the 8-bit checkpoint code, and the host-side
// checks of matrices and checkpoints (library-internal).
#pragma once

#include "zero1_checks.h"
#include "zero1_device.cuh"

// A checkpoint as the kernels take it (codes NULL: none).
namespace z1bn {
struct Ckpt {
    uint8_t *codes, *exps;
    int64_t ld_codes, ld_exps;
};
}  // namespace z1bn

namespace {

using z1bn::Ckpt;

constexpr int kQBlock = 128;  // columns that share a checkpoint scale
constexpr int kMinE = 8;      // biased exponents of the scales: 127 - 119 .. 127 + 119
constexpr int kMaxE = 246;
constexpr int kNanE = 255;

// Lets the next kernel's blocks start as soon as there is room for them; they wait
// for this grid's end in their own wait_prior_grid().
__device__ __forceinline__ void let_next_grid_start() { asm volatile("griddepcontrol.launch_dependents;"); }

// ------------------------------------------------------- typed elements ----

__device__ __forceinline__ float ld1(const uint16_t *p) { return bf_one(*p); }
__device__ __forceinline__ float ld1(const float *p) { return *p; }
__device__ __forceinline__ void st1(uint16_t *p, float x) { *p = to_bf16(x); }
__device__ __forceinline__ void st1(float *p, float x) { *p = x; }

// Eight consecutive elements as they lie in memory: one 16-byte access for
// bf16, two for fp32.
template <class T>
struct Raw8;
template <>
struct Raw8<uint16_t> {
    uint4 q;
    __device__ __forceinline__ void load(const uint16_t *p) { q = ld_stream_u4(p); }
    __device__ __forceinline__ void get(float f[8]) const { unpack8(q, f); }
    __device__ __forceinline__ void zero() { q = make_uint4(0, 0, 0, 0); }
};
template <>
struct Raw8<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float *p)
    {
        a = __ldcs(reinterpret_cast<const float4 *>(p));
        b = __ldcs(reinterpret_cast<const float4 *>(p) + 1);
    }
    __device__ __forceinline__ void get(float f[8]) const
    {
        f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w; f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    }
    __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
};

__device__ __forceinline__ void store8(uint16_t *p, const float f[8])
{
    __stcs(reinterpret_cast<uint4 *>(p), make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]),
                                                    pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7])));
}
__device__ __forceinline__ void store8(float *p, const float f[8])
{
    st_stream(p, f[0], f[1], f[2], f[3]);
    st_stream(p + 4, f[4], f[5], f[6], f[7]);
}

// One value of a small vector (weights, gates) whose type is only known at
// run time; the branch is the same for the whole grid.
__device__ __forceinline__ float ld_param(const void *p, int f32, int64_t i)
{
    return f32 ? __ldg(static_cast<const float *>(p) + i) : bf_one(__ldg(static_cast<const uint16_t *>(p) + i));
}

// ------------------------------------------------------ logistic function --

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
// -------------------------------------------------- 8-bit checkpoint code --

// Largest magnitude seen, as the bits of |x|: integer order is the order of
// the magnitudes, with Inf and NaN above every finite value.
__device__ __forceinline__ uint32_t mag_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }

// Biased scale exponent of a block from its largest magnitude 1.m * 2^(b-127):
// 448 = 1.75 * 2^8, so b - 8, one more if the mantissa is above 1.75.
__device__ __forceinline__ int scale_exp(uint32_t amax)
{
    const int e = (int)(amax >> 23) - 8 + ((amax & 0x7fffffu) > 0x600000u ? 1 : 0);
    return amax >= 0x7f800000u ? kNanE : min(max(e, kMinE), kMaxE);
}

// 2^(127 - E), the factor that brings a block's values to the codes' range
// (0 for a block that stands for NaN, whose codes are 0).
__device__ __forceinline__ float scale_inv(int E) { return E == kNanE ? 0.f : __uint_as_float((uint32_t)(254 - E) << 23); }

// 2^(E - 127), the factor from codes to values (NaN for 255).
__device__ __forceinline__ float scale_of(int E)
{
    return __uint_as_float(E == kNanE ? 0x7fc00000u : (uint32_t)E << 23);
}

// Two values to two e4m3 codes, round to nearest even, saturating.
__device__ __forceinline__ uint32_t code2(float lo, float hi)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// Four codes of a scaled block; `ok` false for a block that stands for NaN.
__device__ __forceinline__ uint32_t code4(float a, float b, float c, float d, float inv, bool ok)
{
    const uint32_t q = code2(__fmul_rn(a, inv), __fmul_rn(b, inv)) |
                       (code2(__fmul_rn(c, inv), __fmul_rn(d, inv)) << 16);
    return ok ? q : 0u;
}

// Two codes to two values (an fp16 holds every e4m3 value exactly).
__device__ __forceinline__ float2 value2(uint16_t q)
{
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(q));
    float2 f;
    asm("{ .reg .f16 l, h; mov.b32 {l, h}, %2; cvt.f32.f16 %0, l; cvt.f32.f16 %1, h; }"
        : "=f"(f.x), "=f"(f.y)
        : "r"(h));
    return f;
}

__device__ __forceinline__ void values8(uint2 q, float scale, float f[8])
{
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const uint32_t w = k < 2 ? q.x : q.y;
        const float2 v = value2((uint16_t)(k & 1 ? w >> 16 : w & 0xffffu));
        f[2 * k] = __fmul_rn(v.x, scale);
        f[2 * k + 1] = __fmul_rn(v.y, scale);
    }
}

__device__ __forceinline__ uint32_t max16(uint32_t a)
{
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) a = max(a, __shfl_xor_sync(0xffffffffu, a, o));
    return a;
}

// ------------------------------------------------------------ fp32 pairs ---
//
// Eight fp32 values as four packed pairs: the .f32x2 instructions do two
// roundings each, the same ones as their scalar forms.

__device__ __forceinline__ uint64_t pair(float a, float b)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float2 split(uint64_t p)
{
    float2 f;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(p));
    return f;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

struct V8 {
    uint64_t p[4];
};

__device__ __forceinline__ V8 splat8(float x)
{
    const uint64_t p = pair(x, x);
    return V8{{p, p, p, p}};
}
__device__ __forceinline__ V8 mul8(const V8 &a, const V8 &b)
{
    return V8{{mul2(a.p[0], b.p[0]), mul2(a.p[1], b.p[1]), mul2(a.p[2], b.p[2]), mul2(a.p[3], b.p[3])}};
}
__device__ __forceinline__ V8 mul8(const V8 &a, float s)
{
    const uint64_t p = pair(s, s);
    return V8{{mul2(a.p[0], p), mul2(a.p[1], p), mul2(a.p[2], p), mul2(a.p[3], p)}};
}
__device__ __forceinline__ V8 fma8(const V8 &a, const V8 &b, const V8 &c)
{
    return V8{{fma2(a.p[0], b.p[0], c.p[0]), fma2(a.p[1], b.p[1], c.p[1]), fma2(a.p[2], b.p[2], c.p[2]),
               fma2(a.p[3], b.p[3], c.p[3])}};
}
__device__ __forceinline__ V8 fma8(const V8 &a, float s, const V8 &c)
{
    const uint64_t p = pair(s, s);
    return V8{{fma2(a.p[0], p, c.p[0]), fma2(a.p[1], p, c.p[1]), fma2(a.p[2], p, c.p[2]), fma2(a.p[3], p, c.p[3])}};
}
__device__ __forceinline__ V8 add8(const V8 &a, const V8 &b)
{
    return V8{{add2(a.p[0], b.p[0]), add2(a.p[1], b.p[1]), add2(a.p[2], b.p[2]), add2(a.p[3], b.p[3])}};
}
// The sum of a . b.
__device__ __forceinline__ float dot8(const V8 &a, const V8 &b)
{
    const uint64_t x = fma2(a.p[1], b.p[1], mul2(a.p[0], b.p[0])), y = fma2(a.p[3], b.p[3], mul2(a.p[2], b.p[2]));
    const float2 s = split(add2(x, y));
    return s.x + s.y;
}

__device__ __forceinline__ V8 from_bf16(const uint4 q)
{
    return V8{{pair(bf_lo(q.x), bf_hi(q.x)), pair(bf_lo(q.y), bf_hi(q.y)), pair(bf_lo(q.z), bf_hi(q.z)),
               pair(bf_lo(q.w), bf_hi(q.w))}};
}

// Eight values of a row in shared memory.
template <class T>
__device__ __forceinline__ V8 take8(const unsigned char *row, int col)
{
    if constexpr (sizeof(T) == 2) {
        return from_bf16(*reinterpret_cast<const uint4 *>(row + col * 2));
    } else {
        const float4 a = *reinterpret_cast<const float4 *>(row + col * 4), b = *reinterpret_cast<const float4 *>(row + col * 4 + 16);
        return V8{{pair(a.x, a.y), pair(a.z, a.w), pair(b.x, b.y), pair(b.z, b.w)}};
    }
}
__device__ __forceinline__ V8 take8(const unsigned char *row, int f32, int col)
{
    return f32 ? take8<float>(row, col) : take8<uint16_t>(row, col);
}

// The values of eight codes.
__device__ __forceinline__ V8 take_codes(const unsigned char *p, float scale)
{
    const uint2 q = *reinterpret_cast<const uint2 *>(p);
    const uint64_t s = pair(scale, scale);
    const float2 a = value2((uint16_t)q.x), b = value2((uint16_t)(q.x >> 16)), c = value2((uint16_t)q.y),
                 d = value2((uint16_t)(q.y >> 16));
    return V8{{mul2(pair(a.x, a.y), s), mul2(pair(b.x, b.y), s), mul2(pair(c.x, c.y), s), mul2(pair(d.x, d.y), s)}};
}

__device__ __forceinline__ void put8(uint16_t *p, const V8 &v)
{
    const float2 a = split(v.p[0]), b = split(v.p[1]), c = split(v.p[2]), d = split(v.p[3]);
    __stcs(reinterpret_cast<uint4 *>(p),
           make_uint4(pack_bf16x2(a.x, a.y), pack_bf16x2(b.x, b.y), pack_bf16x2(c.x, c.y), pack_bf16x2(d.x, d.y)));
}
__device__ __forceinline__ void put8(float *p, const V8 &v)
{
    const float2 a = split(v.p[0]), b = split(v.p[1]), c = split(v.p[2]), d = split(v.p[3]);
    st_stream(p, a.x, a.y, b.x, b.y);
    st_stream(p + 4, c.x, c.y, d.x, d.y);
}

// Stores eight elements at any element offset, those from column D on left out.
__device__ __forceinline__ void put8_any(uint16_t *row, int64_t col, int64_t D, const V8 &v)
{
    uint16_t *p = row + col;
    const float2 a = split(v.p[0]), b = split(v.p[1]), c = split(v.p[2]), d = split(v.p[3]);
    const uint32_t q[4] = {pack_bf16x2(a.x, a.y), pack_bf16x2(b.x, b.y), pack_bf16x2(c.x, c.y), pack_bf16x2(d.x, d.y)};
    if (col + 8 > D) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (col + k < D) p[k] = (uint16_t)(k & 1 ? q[k / 2] >> 16 : q[k / 2]);
    } else if ((uintptr_t)p & 2) {
        p[0] = (uint16_t)q[0];
#pragma unroll
        for (int k = 0; k < 3; ++k) *reinterpret_cast<uint32_t *>(p + 1 + 2 * k) = __funnelshift_r(q[k], q[k + 1], 16);
        p[7] = (uint16_t)(q[3] >> 16);
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) *reinterpret_cast<uint32_t *>(p + 2 * k) = q[k];
    }
}
__device__ __forceinline__ void put8_any(float *row, int64_t col, int64_t D, const V8 &v)
{
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float2 f = split(v.p[k]);
        if (col + 2 * k < D) row[col + 2 * k] = f.x;
        if (col + 2 * k + 1 < D) row[col + 2 * k + 1] = f.y;
    }
}

// Eight bf16 elements at any element offset, zeros from column D on, by the
// aligned words that hold them.  `first`: nothing of the matrix lies before
// this row.
__device__ __forceinline__ uint4 load8_any(const uint16_t *row, int64_t col, int64_t D, bool first)
{
    const uint16_t *p = row + col;
    const int odd = (int)(((uintptr_t)p & 2) >> 1);
    const uint32_t *q = reinterpret_cast<const uint32_t *>(p - odd);
    const int64_t left = D - col + odd;  // elements from the first word to the row's end
    uint32_t w[5];
#pragma unroll
    for (int j = 0; j < 5; ++j) {
        w[j] = 0;
        if (j == 0 && odd && first && col == 0) w[j] = (uint32_t)p[0] << 16;
        else if (left >= 2 * j + 2) w[j] = __ldg(q + j);
        else if (left == 2 * j + 1) w[j] = reinterpret_cast<const uint16_t *>(q + j)[0];
    }
    return make_uint4(__funnelshift_r(w[0], w[1], 16 * odd), __funnelshift_r(w[1], w[2], 16 * odd),
                      __funnelshift_r(w[2], w[3], 16 * odd), __funnelshift_r(w[3], w[4], 16 * odd));
}

// The larger magnitude of three, NaN if one is.
__device__ __forceinline__ float max_abs(float a, float b, float c)
{
    float r;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// Eight values of a 128-column block that 16 lanes hold, as codes; the block's
// biased scale exponent in E.
__device__ __forceinline__ uint2 encode8(const V8 &v, int &E)
{
    const float2 a = split(v.p[0]), b = split(v.p[1]), c = split(v.p[2]), d = split(v.p[3]);
    const float m = max_abs(max_abs(a.x, a.y, b.x), max_abs(b.y, c.x, c.y), max_abs(d.x, d.y, 0.f));
    E = scale_exp(max16(mag_bits(m)));
    const float inv = scale_inv(E);
    const V8 q = mul8(v, inv);
    const float2 e = split(q.p[0]), f = split(q.p[1]), g = split(q.p[2]), h = split(q.p[3]);
    const uint2 r = make_uint2(code2(e.x, e.y) | code2(f.x, f.y) << 16, code2(g.x, g.y) | code2(h.x, h.y) << 16);
    return E == kNanE ? make_uint2(0, 0) : r;
}

// ------------------------------------------------------------ host checks --

int64_t round_up(int64_t n, int64_t m) { return (n + m - 1) / m * m; }
int esize(int dtype) { return dtype == ZERO1_DTYPE_F32 ? 4 : 2; }

int check_dtype(int32_t d, const char *call, const char *what)
{
    if (d != ZERO1_DTYPE_BF16 && d != ZERO1_DTYPE_F32)
        return z1_fail(ZERO1_EINVAL, "%s: unknown %s %d", call, what, d);
    return ZERO1_OK;
}

// A matrix of a call: `rows` rows of `width` bytes, `pitch` bytes apart.
struct Mat {
    const void *p;
    int64_t rows, width, pitch;
    const char *what;
};

// `n` elements in bytes, INT64_MAX or -1 where they do not fit (check_mat then
// refuses the matrix: a stride that wrapped round would pass for a short one).
int64_t in_bytes(int64_t n, int es) { return n < 0 ? -1 : n > INT64_MAX / es ? INT64_MAX : n * es; }

Mat mat(const void *p, int64_t rows, int64_t cols, int64_t ld, int es, const char *what)
{
    return Mat{p, rows, in_bytes(cols, es), in_bytes(rows > 1 ? ld : cols, es), what};
}

// Whether two matrices share a byte.  Of equal pitch they may be interleaved
// (column ranges of one wider matrix).
bool mats_overlap(const Mat &a, const Mat &b)
{
    if (!a.p || !b.p || a.rows <= 0 || b.rows <= 0 || a.width <= 0 || b.width <= 0) return false;
    const Extent ea{a.p, (a.rows - 1) * a.pitch + a.width, ""}, eb{b.p, (b.rows - 1) * b.pitch + b.width, ""};
    if (!overlap(ea, eb)) return false;
    if (a.rows > 1 && b.rows > 1 && a.pitch == b.pitch && a.pitch > 0) {
        const int64_t p = a.pitch;
        int64_t d = ((intptr_t)b.p - (intptr_t)a.p) % p;
        if (d < 0) d += p;
        return !(d >= a.width && d + b.width <= p);
    }
    return true;
}

// A matrix argument: present, aligned to its elements, a stride that fits.
int check_mat(const Mat &m, int es, bool out, const char *call)
{
    if (m.rows == 0) return ZERO1_OK;
    if (!m.p) return z1_fail(ZERO1_EINVAL, "%s: %s is NULL", call, m.what);
    if (m.pitch < 0 || (out && m.pitch < m.width))
        return z1_fail(ZERO1_EINVAL, m.pitch < 0 ? "%s: %s: negative row stride" : "%s: %s: row stride of %lld elements", call,
                       m.what, (long long)(m.pitch / es));
    if (m.rows > 1 && m.pitch > INT64_MAX / m.rows)
        return z1_fail(ZERO1_ERANGE, "%s: %s: size overflows", call, m.what);
    return check_natural(m.p, es, m.what);
}

int check_ckpt(const zero1_checkpoint8_t *c, const char *call, const char *what)
{
    if (!c) return z1_fail(ZERO1_EINVAL, "%s: %s is NULL", call, what);
    if (c->rows < 0 || c->cols < 1)
        return z1_fail(ZERO1_EINVAL, "%s: %s: %lld rows, %lld columns", call, what, (long long)c->rows,
                       (long long)c->cols);
    if (c->rows > (INT64_C(1) << 40) || c->cols > (INT64_C(1) << 40))
        return z1_fail(ZERO1_ERANGE, "%s: %s: size not supported", call, what);
    if (c->rows == 0) return ZERO1_OK;
    if (!c->codes || !c->exps) return z1_fail(ZERO1_EINVAL, "%s: %s: NULL codes or exps", call, what);
    if (((uintptr_t)c->codes | (uintptr_t)c->exps | (uintptr_t)c->ld_codes | (uintptr_t)c->ld_exps) & 15)
        return z1_fail(ZERO1_EALIGN, "%s: %s: codes, exps and their strides must be multiples of 16 bytes", call, what);
    if (c->ld_codes < round_up(c->cols, kQBlock) || c->ld_exps < round_up(c->rows, kQBlock))
        return z1_fail(ZERO1_EINVAL, "%s: %s: strides %lld, %lld are too short", call, what, (long long)c->ld_codes,
                       (long long)c->ld_exps);
    if (c->ld_codes > INT64_MAX / c->rows || c->ld_exps > INT64_MAX / (round_up(c->cols, kQBlock) / kQBlock))
        return z1_fail(ZERO1_ERANGE, "%s: %s: size overflows", call, what);
    return ZERO1_OK;
}

Mat codes_mat(const zero1_checkpoint8_t *c, const char *what)
{
    return c ? Mat{c->codes, c->rows, round_up(c->cols, kQBlock), c->ld_codes, what} : Mat{nullptr, 0, 0, 0, what};
}
Mat exps_mat(const zero1_checkpoint8_t *c, const char *what)
{
    return c ? Mat{c->exps, round_up(c->cols, kQBlock) / kQBlock, c->rows, c->ld_exps, what}
             : Mat{nullptr, 0, 0, 0, what};
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

// Rows that the 128-bit path can address.
bool vec_ok(const Mat &m) { return !m.p || ((((uintptr_t)m.p) | (uintptr_t)m.pitch) & 15) == 0; }

// Lets a kernel use up to `bytes` of dynamic shared memory; asked of the
// runtime once per kernel and device.
template <class K>
cudaError_t allow_smem(K kernel, int bytes, std::atomic<uint64_t> &done)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = UINT64_C(1) << (dev & 63);
    if (dev < 64 && (done.load(std::memory_order_relaxed) & bit)) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess && dev < 64) done.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

// launch_pdl with any grid and dynamic shared memory: the kernel calls
// wait_prior_grid() before it touches global memory.
template <class K, class... Args>
cudaError_t launch_after(K kernel, dim3 grid, int block, int smem, cudaStream_t st, Args... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)block);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace
