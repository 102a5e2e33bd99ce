// zero1_checkpoint.cu - 8-bit activation checkpoints: pack a matrix into e4m3
// codes with a power-of-two scale per row and 128 columns, and unpack it.

#include "zero1_block.cuh"

namespace {

// Both kernels are one pass over the matrix: 3 bytes per bf16 element (2 + 1)
// plus 1/128 of scales, bound by HBM (8192 x 14336 bf16: pack 6.0, unpack 6.3
// TB/s).  A thread owns 8 columns of kRows consecutive rows, so that 16 lanes
// hold one 128-column block (its maximum is four shuffles), kRows 16-byte loads
// are in flight per thread, and the four scale bytes of a column block leave as
// one 32-bit store.  Off the 128-bit path a thread's columns are 16 apart, but
// consecutive where bf16 is packed: the aligned words that hold them are read
// (20000 x 3001: 130 -> 63 us; written that way they took longer, 49 -> 54 us).
constexpr int kRows = 4;
constexpr int kThreads = 256;

struct Tiles {
    int64_t rows, cols;
    int tx;  // threads across columns: 16, 32, .. 256; a block covers 8 * tx columns, kRows * 256 / tx rows
};

template <class T, bool VEC>
__global__ void __launch_bounds__(kThreads) k_ckpt_pack(const T *__restrict__ x, int64_t ld, Tiles s, Ckpt c)
{
    const int64_t kp = (s.cols + kQBlock - 1) / kQBlock * kQBlock;
    const int64_t row0 = ((int64_t)blockIdx.x * (kThreads / s.tx) + threadIdx.x / s.tx) * kRows;
    constexpr bool kNext = VEC || sizeof(T) == 2;  // the thread's 8 columns are consecutive, else 16 apart
    const int64_t v = (int64_t)blockIdx.y * s.tx + threadIdx.x % s.tx;
    const int64_t col0 = kNext ? v * 8 : v / 16 * kQBlock + v % 16;
    V8 f[kRows];
    if constexpr (VEC) {  // all loads before the first use
        Raw8<T> q[kRows];
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            q[r].zero();
            if (row0 + r < s.rows && col0 < s.cols) q[r].load(x + (row0 + r) * ld + col0);
        }
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            float e[8];
            q[r].get(e);
            f[r] = V8{{pair(e[0], e[1]), pair(e[2], e[3]), pair(e[4], e[5]), pair(e[6], e[7])}};
        }
    } else {
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            const T *row = x + (row0 + r) * ld;
            f[r] = splat8(0.f);
            if (row0 + r >= s.rows || col0 >= s.cols) continue;
            if constexpr (kNext) {
                f[r] = from_bf16(load8_any(row, col0, s.cols, (row0 + r) * ld == 0));
            } else {
                float e[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) e[k] = col0 + 16 * k < s.cols ? ld1(row + col0 + 16 * k) : 0.f;
                f[r] = V8{{pair(e[0], e[1]), pair(e[2], e[3]), pair(e[4], e[5]), pair(e[6], e[7])}};
            }
        }
    }
    uint32_t exps = 0;
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        int E;
        const uint2 q = encode8(f[r], E);
        exps |= (uint32_t)E << (8 * r);
        if (row0 + r < s.rows && col0 < kp) {
            uint8_t *o = c.codes + (row0 + r) * c.ld_codes + col0;
            if constexpr (kNext) {
                __stcs(reinterpret_cast<uint2 *>(o), q);
            } else {
#pragma unroll
                for (int k = 0; k < 8; ++k) o[16 * k] = (uint8_t)((k < 4 ? q.x : q.y) >> (8 * (k & 3)));
            }
        }
    }
    if (threadIdx.x % 16 == 0 && col0 < kp) {
        uint8_t *e = c.exps + col0 / kQBlock * c.ld_exps + row0;
        if (row0 + kRows <= s.rows) {
            *reinterpret_cast<uint32_t *>(e) = exps;
        } else {
            for (int r = 0; r < kRows && row0 + r < s.rows; ++r) e[r] = (uint8_t)(exps >> (8 * r));
        }
    }
}

template <class T, bool VEC>
__global__ void __launch_bounds__(kThreads) k_ckpt_unpack(Ckpt c, Tiles s, T *__restrict__ out, int64_t ld)
{
    const int64_t row0 = ((int64_t)blockIdx.x * (kThreads / s.tx) + threadIdx.x / s.tx) * kRows;
    const int64_t v = (int64_t)blockIdx.y * s.tx + threadIdx.x % s.tx;
    const int64_t col0 = VEC ? v * 8 : v / 16 * kQBlock + v % 16;
    if (row0 >= s.rows || col0 >= s.cols) return;
    uint2 q[kRows];
    uint32_t exps = 0;
    const uint8_t *e = c.exps + col0 / kQBlock * c.ld_exps + row0;
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        q[r] = make_uint2(0, 0);
        if (row0 + r >= s.rows) continue;
        const uint8_t *p = c.codes + (row0 + r) * c.ld_codes + col0;
        if constexpr (VEC) {
            q[r] = __ldcs(reinterpret_cast<const uint2 *>(p));
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (col0 + 16 * k < s.cols) (k < 4 ? q[r].x : q[r].y) |= (uint32_t)p[16 * k] << (8 * (k & 3));
        }
        exps |= (uint32_t)e[r] << (8 * r);
    }
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        if (row0 + r >= s.rows) continue;
        float f[8];
        values8(q[r], scale_of((exps >> (8 * r)) & 255), f);
        T *p = out + (row0 + r) * ld + col0;
        if constexpr (VEC) {
            store8(p, f);
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (col0 + 16 * k < s.cols) st1(p + 16 * k, f[k]);
        }
    }
}

// The grid over a [rows, cols] matrix: rows on x, so that any row count fits.
int tiles_of(int64_t rows, int64_t cols, const char *call, Tiles *s, dim3 *grid)
{
    const int64_t vecs = round_up(cols, kQBlock) / 8;
    int tx = 16;
    while (tx < kThreads && tx < vecs) tx *= 2;
    const int64_t gx = (rows + (int64_t)kRows * (kThreads / tx) - 1) / (kRows * (kThreads / tx));
    const int64_t gy = (vecs + tx - 1) / tx;
    if (gx > INT32_MAX || gy > 65535) return z1_fail(ZERO1_ERANGE, "%s: size not supported", call);
    *s = Tiles{rows, cols, tx};
    *grid = dim3((unsigned)gx, (unsigned)gy);
    return ZERO1_OK;
}

template <class T>
void launch_pack(const void *x, int64_t ld, const Tiles &s, const Ckpt &c, bool vec, dim3 grid, cudaStream_t st)
{
    if (vec) k_ckpt_pack<T, true><<<grid, kThreads, 0, st>>>(static_cast<const T *>(x), ld, s, c);
    else k_ckpt_pack<T, false><<<grid, kThreads, 0, st>>>(static_cast<const T *>(x), ld, s, c);
}

template <class T>
void launch_unpack(const Ckpt &c, const Tiles &s, void *out, int64_t ld, bool vec, dim3 grid, cudaStream_t st)
{
    if (vec) k_ckpt_unpack<T, true><<<grid, kThreads, 0, st>>>(c, s, static_cast<T *>(out), ld);
    else k_ckpt_unpack<T, false><<<grid, kThreads, 0, st>>>(c, s, static_cast<T *>(out), ld);
}

int check_call(const zero1_checkpoint8_t *ckpt, const void *p, int64_t ld, int32_t dtype, bool out, const char *call,
               Mat *m)
{
    int rc = check_ckpt(ckpt, call, "the checkpoint");
    if (rc != ZERO1_OK) return rc;
    if ((rc = check_dtype(dtype, call, "dtype")) != ZERO1_OK) return rc;
    *m = mat(p, ckpt->rows, ckpt->cols, ld, esize(dtype), out ? "out" : "x");
    if ((rc = check_mat(*m, esize(dtype), out, call)) != ZERO1_OK) return rc;
    const Mat a = codes_mat(ckpt, "codes"), b = exps_mat(ckpt, "exps");
    if (mats_overlap(*m, a) || mats_overlap(*m, b) || mats_overlap(a, b))
        return z1_fail(ZERO1_EINVAL, "%s: buffers overlap", call);
    return ZERO1_OK;
}

}  // namespace

extern "C" int zero1_checkpoint_pack(const void *x, int64_t ld_x, int32_t dtype, const zero1_checkpoint8_t *ckpt,
                                     zero1_stream_t stream)
{
    Z1Trace trace("zero1_checkpoint_pack");
    Mat m;
    int rc = check_call(ckpt, x, ld_x, dtype, false, "checkpoint pack", &m);
    if (rc != ZERO1_OK || ckpt->rows == 0) return rc;
    Tiles s;
    dim3 grid;
    if ((rc = tiles_of(ckpt->rows, ckpt->cols, "checkpoint pack", &s, &grid)) != ZERO1_OK) return rc;
    const bool vec = vec_ok(m) && ckpt->cols % 8 == 0;
    const Ckpt c{ckpt->codes, ckpt->exps, ckpt->ld_codes, ckpt->ld_exps};
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (dtype == ZERO1_DTYPE_F32) launch_pack<float>(x, ld_x, s, c, vec, grid, st);
    else launch_pack<uint16_t>(x, ld_x, s, c, vec, grid, st);
    return launch_status("checkpoint pack launch");
}

extern "C" int zero1_checkpoint_unpack(const zero1_checkpoint8_t *ckpt, void *out, int64_t ld_out, int32_t dtype,
                                       zero1_stream_t stream)
{
    Z1Trace trace("zero1_checkpoint_unpack");
    Mat m;
    int rc = check_call(ckpt, out, ld_out, dtype, true, "checkpoint unpack", &m);
    if (rc != ZERO1_OK || ckpt->rows == 0) return rc;
    Tiles s;
    dim3 grid;
    if ((rc = tiles_of(ckpt->rows, ckpt->cols, "checkpoint unpack", &s, &grid)) != ZERO1_OK) return rc;
    const bool vec = vec_ok(m) && ckpt->cols % 8 == 0;
    const Ckpt c{ckpt->codes, ckpt->exps, ckpt->ld_codes, ckpt->ld_exps};
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (dtype == ZERO1_DTYPE_F32) launch_unpack<float>(c, s, out, ld_out, vec, grid, st);
    else launch_unpack<uint16_t>(c, s, out, ld_out, vec, grid, st);
    return launch_status("checkpoint unpack launch");
}
