// zero1_weight_grad.cu - the weight gradient of a projection, taken straight
// from the 8-bit checkpoint of its input.

#include "zero1_block.cuh"

namespace {

constexpr int kTile = 64, kDeep = 16;

// dw[n, k] = c[k] * sum_t dy[t, n] * x8[t, k]: 64 x 64 outputs per block,
// 4 x 4 per thread, 16 rows of dy and x at a time in shared memory.
template <class TO>
__global__ void __launch_bounds__(256)
k_weight_grad(const uint16_t *__restrict__ dy, int64_t ld_dy, int64_t T, int64_t N, int64_t K, const Ckpt x8,
              const void *scale, int scale_f32, TO *__restrict__ dw, int64_t ld_dw, int accumulate)
{
    __shared__ float a[kDeep][kTile], b[kDeep][kTile];
    const int64_t n0 = (int64_t)blockIdx.x * kTile, k0 = (int64_t)blockIdx.y * kTile;
    const int tn = threadIdx.x / 16 * 4, tk = threadIdx.x % 16 * 4;
    float acc[4][4] = {};
    for (int64_t t0 = 0; t0 < T; t0 += kDeep) {
        for (int q = threadIdx.x; q < kDeep * kTile; q += 256) {
            const int t = q / kTile, c = q % kTile;
            const bool in = t0 + t < T;
            a[t][c] = in && n0 + c < N ? bf_one(dy[(t0 + t) * ld_dy + n0 + c]) : 0.f;
            float v = 0.f;
            if (in && k0 + c < K) {
                const float2 f = value2(x8.codes[(t0 + t) * x8.ld_codes + k0 + c]);
                v = f.x * scale_of(x8.exps[(k0 + c) / kQBlock * x8.ld_exps + t0 + t]);
            }
            b[t][c] = v;
        }
        __syncthreads();
#pragma unroll
        for (int t = 0; t < kDeep; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(a[t][tn + i], b[t][tk + j], acc[i][j]);
        __syncthreads();
    }
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) {
            const int64_t n = n0 + tn + i, k = k0 + tk + j;
            if (n >= N || k >= K) continue;
            TO *o = dw + n * ld_dw + k;
            float v = acc[i][j];
            if (scale) v *= ld_param(scale, scale_f32, k);
            st1(o, accumulate ? ld1(o) + v : v);
        }
}

}  // namespace

extern "C" int zero1_weight_grad_workspace(int64_t rows, int64_t n, int64_t k, const void *dy, int64_t ld_dy,
                                           int64_t *bytes)
{
    if (!bytes) return z1_fail(ZERO1_EINVAL, "weight gradient workspace: bytes is NULL");
    *bytes = 0;
    return ZERO1_OK;
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
    const Mat a = mat(dy, T, n, ld_dy, 2, "dy"), o = mat(dw, n, K, ld_dw, eo, "dw");
    if ((rc = check_mat(a, 2, false, call)) || (rc = check_mat(o, eo, true, call)) ||
        (col_scale && (rc = check_natural(col_scale, es, "col_scale"))))
        return rc;
    const Mat in[] = {a, codes_mat(x8, "the codes of x8"), exps_mat(x8, "the exps of x8"),
                      mat(col_scale, 1, K, 0, es, "col_scale")};
    for (const Mat &m : in)
        if (mats_overlap(o, m)) return z1_fail(ZERO1_EINVAL, "%s: dw and %s overlap", call, m.what);
    const Ckpt c{x8->codes, x8->exps, x8->ld_codes, x8->ld_exps};
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const dim3 grid((unsigned)((n + kTile - 1) / kTile), (unsigned)((K + kTile - 1) / kTile));
    if (out_dtype == ZERO1_DTYPE_F32)
        k_weight_grad<float><<<grid, 256, 0, st>>>(static_cast<const uint16_t *>(dy), ld_dy, T, n, K, c, col_scale,
                                                   scale_dtype, static_cast<float *>(dw), ld_dw, accumulate);
    else
        k_weight_grad<uint16_t><<<grid, 256, 0, st>>>(static_cast<const uint16_t *>(dy), ld_dy, T, n, K, c, col_scale,
                                                      scale_dtype, static_cast<uint16_t *>(dw), ld_dw, accumulate);
    return launch_status("weight gradient launch");
}
