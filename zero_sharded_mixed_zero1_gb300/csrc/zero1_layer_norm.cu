// zero1_layer_norm.cu - layer norm with its residual: the calls, their checks,
// and the joining of the backward pass's column sums.

#include "zero1_layer_norm.cuh"

namespace {

// Adds the blocks' partial column sums in block order: 32 columns per block, 32
// slices of the partials each summed in order and then joined in order.  The
// partials were just written and come from L2; ten loads of a slice are under way
// together (one after the other they took 8 us more at 304 blocks of 4096 columns).
constexpr int kSlices = 32, kAtOnce = 10;

struct LnFinish {
    const float *part;
    int64_t nparts;
    int D, ld, f32, accumulate;
    void *out[2];  // dw, db (NULL: not wanted)
};

__global__ void __launch_bounds__(32 * kSlices) k_layer_norm_finish(const LnFinish f)
{
    wait_prior_grid();
    let_next_grid_start();
    __shared__ float sum[kSlices][32];
    const int s = blockIdx.y;
    if (!f.out[s]) return;
    const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5;
    const int col = blockIdx.x * 32 + lane;
    const float *p = f.part + (int64_t)s * f.nparts * f.ld + col;
    const int per = (int)((f.nparts + kSlices - 1) / kSlices), b = slice * per, e = min(b + per, (int)f.nparts);
    float x = 0.f;
    if (col < f.D) {
        for (int q = b; q < e; q += kAtOnce) {
            float v[kAtOnce];
#pragma unroll
            for (int j = 0; j < kAtOnce; ++j) v[j] = q + j < e ? __ldcg(p + (int64_t)(q + j) * f.ld) : 0.f;
#pragma unroll
            for (int j = 0; j < kAtOnce; ++j) x += v[j];
        }
    }
    sum[slice][lane] = x;
    __syncthreads();
    if (slice || col >= f.D) return;
#pragma unroll
    for (int q = 1; q < kSlices; ++q) x += sum[q][lane];
    if (f.f32) {
        float *o = static_cast<float *>(f.out[s]) + col;
        *o = f.accumulate ? *o + x : x;
    } else {
        uint16_t *o = static_cast<uint16_t *>(f.out[s]) + col;
        *o = to_bf16(f.accumulate ? bf_one(*o) + x : x);
    }
}

int check_ln(const zero1_layer_norm_t *cfg, const char *call)
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
        (rc = check_dtype(cfg->param_dtype, call, "param_dtype")) || (rc = check_dtype(cfg->grad_dtype, call, "grad_dtype")))
        return rc;
    if (cfg->act_dtype == ZERO1_DTYPE_F32 && cfg->res_dtype != ZERO1_DTYPE_F32)
        return z1_fail(ZERO1_EINVAL, "%s: fp32 activations need an fp32 residual stream", call);
    return ZERO1_OK;
}

int check_r8(const zero1_layer_norm_t *cfg, const zero1_checkpoint8_t *k, const char *call)
{
    const int rc = check_ckpt(k, call, "r8");
    if (rc != ZERO1_OK) return rc;
    if (k->rows != cfg->rows || k->cols != cfg->cols)
        return z1_fail(ZERO1_EINVAL, "%s: r8 is %lld x %lld, not %lld x %lld", call, (long long)k->rows, (long long)k->cols,
                       (long long)cfg->rows, (long long)cfg->cols);
    return ZERO1_OK;
}

// Calls f(TA, TR) for the run-time types.
template <class F>
int dispatch_types(const zero1_layer_norm_t *cfg, F &&f)
{
    if (cfg->act_dtype == ZERO1_DTYPE_F32) return f(float{}, float{});
    if (cfg->res_dtype == ZERO1_DTYPE_F32) return f(uint16_t{}, float{});
    return f(uint16_t{}, uint16_t{});
}

}  // namespace

extern "C" int zero1_layer_norm_forward(const zero1_layer_norm_t *cfg, const zero1_layer_norm_forward_t *io, zero1_stream_t stream)
{
    Z1Trace trace("zero1_layer_norm_forward");
    const char *call = "layer norm forward";
    if (!io) return z1_fail(ZERO1_EINVAL, "%s: the buffers are NULL", call);
    int rc = check_ln(cfg, call);
    if (rc != ZERO1_OK) return rc;
    if ((io->y == nullptr) != (io->r == nullptr) && cfg->rows > 0)
        return z1_fail(ZERO1_EINVAL, "%s: %s without %s", call, io->y ? "y" : "r", io->y ? "r" : "y");
    if (cfg->rows == 0) return ZERO1_OK;
    const int64_t T = cfg->rows, D = cfg->cols;
    const int ea = esize(cfg->act_dtype), er = esize(cfg->res_dtype), ep = esize(cfg->param_dtype);
    const Mat in[] = {mat(io->x, T, D, io->ld_x, er, "x"), mat(io->y, T, D, io->ld_y, ea, "y"), mat(io->w, 1, D, 0, ep, "w"),
                      mat(io->b, 1, D, 0, ep, "b")};
    const Mat out[] = {mat(io->r, T, D, io->ld_r, er, "r"), mat(io->h, T, D, io->ld_h, ea, "h"),
                       mat(io->mean, 1, T, 0, 4, "mean"), mat(io->rstd, 1, T, 0, 4, "rstd"),
                       codes_mat(io->r8, "the codes of r8"), exps_mat(io->r8, "the exps of r8")};
    const int in_place[] = {0, -1, -1, -1, -1, -1};
    if ((rc = check_mat(in[0], er, false, call)) || (io->y && ((rc = check_mat(in[1], ea, false, call)) || (rc = check_mat(out[0], er, true, call)))) ||
        (io->w && (rc = check_natural(io->w, ep, "w"))) || (io->b && (rc = check_natural(io->b, ep, "b"))) ||
        (rc = check_mat(out[1], ea, true, call)) || (rc = check_mat(out[2], 4, true, call)) || (rc = check_mat(out[3], 4, true, call)) ||
        (io->r8 && (rc = check_r8(cfg, io->r8, call))) || (rc = check_overlaps(out, in_place, 6, in, 4, call)))
        return rc;
    const int sms = sm_count();
    if (sms == 0) return z1_fail(ZERO1_ECUDA, "%s: no CUDA device", call);
    z1ln::Fwd a{};
    a.rows = T;
    a.D = (int)D;
    a.eps = cfg->eps;
    a.alpha = cfg->residual_scale;
    a.inv_d = (float)(1.0 / (double)D);
    a.inv_d_low = (float)(1.0 / (double)D - (double)a.inv_d);
    a.pf32 = cfg->param_dtype == ZERO1_DTYPE_F32;
    a.x = io->x; a.y = io->y; a.w = io->w; a.b = io->b;
    a.r = io->r; a.h = io->h;
    a.mean = io->mean; a.rstd = io->rstd;
    if (io->r8) a.r8 = Ckpt{io->r8->codes, io->r8->exps, io->r8->ld_codes, io->r8->ld_exps};
    a.ld_x = io->ld_x; a.ld_y = io->ld_y; a.ld_r = io->ld_r; a.ld_h = io->ld_h;
    const bool vec = D % 8 == 0 && vec_ok(in[0]) && vec_ok(in[1]) && vec_ok(out[0]) && vec_ok(out[1]);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    return dispatch_types(cfg, [&](auto ta, auto tr) { return z1ln::run_forward<decltype(ta), decltype(tr)>(a, vec, sms, st); });
}

extern "C" int zero1_layer_norm_workspace(const zero1_layer_norm_t *cfg, int64_t *bytes)
{
    const char *call = "layer norm workspace";
    if (!bytes) return z1_fail(ZERO1_EINVAL, "%s: bytes is NULL", call);
    const int rc = check_ln(cfg, call);
    if (rc != ZERO1_OK) return rc;
    const int sms = sm_count();
    if (sms == 0) return z1_fail(ZERO1_ECUDA, "%s: no CUDA device", call);
    *bytes = 2 * bwd_blocks(cfg->rows, cfg->cols, sms) * round_up(cfg->cols, 8) * 4;
    return ZERO1_OK;
}

extern "C" int zero1_layer_norm_backward(const zero1_layer_norm_t *cfg, const zero1_layer_norm_backward_t *io, void *workspace,
                                         int64_t workspace_bytes, zero1_stream_t stream)
{
    Z1Trace trace("zero1_layer_norm_backward");
    const char *call = "layer norm backward";
    if (!io) return z1_fail(ZERO1_EINVAL, "%s: the buffers are NULL", call);
    int rc = check_ln(cfg, call);
    if (rc != ZERO1_OK) return rc;
    const int64_t T = cfg->rows, D = cfg->cols;
    const int ea = esize(cfg->act_dtype), er = esize(cfg->res_dtype), ep = esize(cfg->param_dtype), eg = esize(cfg->grad_dtype);
    const zero1_checkpoint8_t *r8 = T > 0 ? io->r8 : nullptr;
    const Mat in[] = {mat(io->dr, T, D, io->ld_dr, er, "dr"), mat(io->dh, T, D, io->ld_dh, ea, "dh"),
                      mat(io->r, T, D, io->ld_r, er, "r"), mat(io->w, 1, D, 0, ep, "w"), mat(io->mean, 1, T, 0, 4, "mean"),
                      mat(io->rstd, 1, T, 0, 4, "rstd"), codes_mat(r8, "the codes of r8"), exps_mat(r8, "the exps of r8")};
    const Mat out[] = {mat(io->dx, T, D, io->ld_dx, er, "dx"), mat(io->dy, T, D, io->ld_dy, ea, "dy"),
                       mat(io->dw, 1, D, 0, eg, "dw"), mat(io->db, 1, D, 0, eg, "db"),
                       Mat{workspace, 1, workspace_bytes, workspace_bytes, "the workspace"}};
    const int in_place[] = {0, 1, -1, -1, -1};
    if (T > 0) {
        if ((rc = check_mat(in[1], ea, false, call)) || (io->dr && (rc = check_mat(in[0], er, false, call))) ||
            (io->w && (rc = check_natural(io->w, ep, "w"))) || (rc = check_mat(in[4], 4, false, call)) ||
            (rc = check_mat(in[5], 4, false, call)) || (rc = check_mat(out[0], er, true, call)) ||
            (io->dy && (rc = check_mat(out[1], ea, true, call))))
            return rc;
        if ((io->r != nullptr) == (r8 != nullptr)) return z1_fail(ZERO1_EINVAL, "%s: exactly one of r and r8 is needed", call);
        if (r8 ? (rc = check_r8(cfg, r8, call)) : (rc = check_mat(in[2], er, false, call))) return rc;
    }
    if ((io->dw && (rc = check_natural(io->dw, eg, "dw"))) || (io->db && (rc = check_natural(io->db, eg, "db"))) ||
        (rc = check_overlaps(out, in_place, 5, in, 8, call)))
        return rc;
    const int sms = sm_count();
    if (sms == 0) return z1_fail(ZERO1_ECUDA, "%s: no CUDA device", call);
    const int64_t grid = bwd_blocks(T, D, sms);
    const bool sums = io->dw || io->db;
    const int64_t need = sums ? 2 * grid * round_up(D, 8) * 4 : 0;
    if (need > 0) {
        if (!workspace || workspace_bytes < need)
            return z1_fail(ZERO1_EINVAL, "%s: workspace of %lld bytes, needs %lld", call, (long long)(workspace ? workspace_bytes : 0),
                           (long long)need);
        if ((uintptr_t)workspace & 15) return z1_fail(ZERO1_EALIGN, "%s: the workspace is not 16-byte aligned", call);
        if (in_host_memory(workspace)) return z1_fail(ZERO1_EINVAL, "%s: the workspace must be device memory", call);
    }
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (T > 0) {
        z1ln::Bwd a{};
        a.rows = T;
        a.D = (int)D;
        a.alpha = cfg->residual_scale;
        a.inv_d = (float)(1.0 / (double)D);
        a.pf32 = cfg->param_dtype == ZERO1_DTYPE_F32;
        a.dh = io->dh; a.dr = io->dr; a.r = io->r; a.w = io->w;
        a.mean = io->mean; a.rstd = io->rstd;
        if (r8) a.r8 = Ckpt{r8->codes, r8->exps, r8->ld_codes, r8->ld_exps};
        a.dx = io->dx; a.dy = io->dy;
        a.ld_dh = io->ld_dh; a.ld_dr = io->ld_dr; a.ld_r = io->ld_r; a.ld_dx = io->ld_dx; a.ld_dy = io->ld_dy;
        a.need_w = io->dw != nullptr; a.need_b = io->db != nullptr;
        a.part = static_cast<float *>(workspace);
        a.ld_part = (int)round_up(D, 8);
        const bool vec = D % 8 == 0 && vec_ok(in[0]) && vec_ok(in[1]) && vec_ok(in[2]) && vec_ok(out[0]) && vec_ok(out[1]);
        rc = dispatch_types(cfg, [&](auto ta, auto tr) { return z1ln::run_backward<decltype(ta), decltype(tr)>(a, vec, grid, st); });
        if (rc != ZERO1_OK) return rc;
    }
    if (!sums) return ZERO1_OK;
    LnFinish f{};
    f.part = static_cast<const float *>(workspace);
    f.nparts = grid;
    f.D = (int)D;
    f.ld = (int)round_up(D, 8);
    f.f32 = cfg->grad_dtype == ZERO1_DTYPE_F32;
    f.accumulate = cfg->accumulate != 0;
    f.out[0] = io->dw;
    f.out[1] = io->db;
    const cudaError_t e = launch_after(k_layer_norm_finish, dim3((unsigned)((D + 31) / 32), 2), 32 * kSlices, 0, st, f);
    if (e != cudaSuccess) return pdl_fail(e, "layer norm backward: column sums");
    return ZERO1_OK;
}
