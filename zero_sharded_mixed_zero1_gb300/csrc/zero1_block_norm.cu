// zero1_block_norm.cu - norms before and after a block, fused with the
// block's gate and residual scale: the calls, their checks, and the joining of
// the backward pass's column sums.

#include "zero1_block_norm.cuh"

namespace {

// Adds the blocks' partial column sums in block order: 32 columns per block,
// 8 slices of the partials each summed in order and then joined in order.  The
// partials were just written and come from L2: 3 us for 304 blocks of 4096.
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
    if (s == 2 && f.gate) x *= Logistic<>(ld_param(f.gate, f.gf32, col)).slope;
    if (f.f32) {
        float *o = static_cast<float *>(f.out[s]) + col;
        *o = f.accumulate ? *o + x : x;
    } else {
        uint16_t *o = static_cast<uint16_t *>(f.out[s]) + col;
        *o = to_bf16(f.accumulate ? bf_one(*o) + x : x);
    }
}

int check_cfg(const zero1_block_norm_t *cfg, bool has_gate, const char *call)
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

// Calls f(TA, TR) for the run-time types.
template <class F>
int dispatch_types(const zero1_block_norm_t *cfg, F &&f)
{
    if (cfg->act_dtype == ZERO1_DTYPE_F32) return f(float{}, float{});
    if (cfg->res_dtype == ZERO1_DTYPE_F32) return f(uint16_t{}, float{});
    return f(uint16_t{}, uint16_t{});
}

}  // namespace

extern "C" int zero1_block_norm_forward(const zero1_block_norm_t *cfg, const zero1_block_norm_forward_t *io,
                                        zero1_stream_t stream)
{
    Z1Trace trace("zero1_block_norm_forward");
    const char *call = "block norm forward";
    if (!io) return z1_fail(ZERO1_EINVAL, "%s: the buffers are NULL", call);
    int rc = check_cfg(cfg, io->gate != nullptr, call);
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
    return dispatch_types(cfg, [&](auto ta, auto tr) {
        return z1bn::run_forward<decltype(ta), decltype(tr)>(c, a, vec, sms, st);
    });
}

extern "C" int zero1_block_norm_workspace(const zero1_block_norm_t *cfg, int64_t *bytes)
{
    const char *call = "block norm workspace";
    if (!bytes) return z1_fail(ZERO1_EINVAL, "%s: bytes is NULL", call);
    int rc = check_cfg(cfg, cfg && cfg->gate_kind != ZERO1_GATE_NONE, call);
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
    int rc = check_cfg(cfg, io->gate != nullptr, call);
    if (rc != ZERO1_OK) return rc;
    const int64_t T = cfg->rows, D = cfg->cols;
    const int ea = esize(cfg->act_dtype), er = esize(cfg->res_dtype), ep = esize(cfg->param_dtype),
              eg = esize(cfg->gate_dtype), ew = esize(cfg->grad_dtype);
    const int edg = cfg->gate_kind == ZERO1_GATE_FULL ? eg : ew;
    // What the call does not need is not looked at: neither checked nor read.
    const bool need_y = post || io->dgate;
    const void *y = need_y ? io->y : nullptr;
    const zero1_checkpoint8_t *y8 = need_y && T > 0 ? io->y8 : nullptr, *r8 = T > 0 ? io->r8 : nullptr;
    const Mat in[] = {mat(io->dr, T, D, io->ld_dr, er, "dr"), mat(io->dh, T, D, io->ld_dh, ea, "dh"),
                      mat(y, T, D, io->ld_y, ea, "y"), mat(io->r, T, D, io->ld_r, er, "r"),
                      mat(io->w_post, 1, D, 0, ep, "w_post"), mat(io->w_pre, 1, D, 0, ep, "w_pre"),
                      gate_mat(cfg, io->gate, io->ld_gate, eg, "gate"),
                      mat(io->rstd_post, 1, T, 0, 4, "rstd_post"), mat(io->rstd_pre, 1, T, 0, 4, "rstd_pre"),
                      codes_mat(y8, "the codes of y8"), exps_mat(y8, "the exps of y8"),
                      codes_mat(r8, "the codes of r8"), exps_mat(r8, "the exps of r8")};
    Mat work{workspace, 1, workspace_bytes, workspace_bytes, "the workspace"};
    const Mat out[] = {mat(io->dx, T, D, io->ld_dx, er, "dx"), mat(io->dy, T, D, io->ld_dy, ea, "dy"),
                       mat(io->dw_post, 1, D, 0, ew, "dw_post"), mat(io->dw_pre, 1, D, 0, ew, "dw_pre"),
                       gate_mat(cfg, io->dgate, io->ld_dgate, edg, "dgate"), work};
    const int in_place[] = {0, 1, -1, -1, -1, -1};
    if (!post && (io->dw_post || io->rstd_post)) return z1_fail(ZERO1_EINVAL, "%s: dw_post or rstd_post without w_post", call);
    if (!pre && (io->dw_pre || io->rstd_pre || io->dh || io->r || io->r8))
        return z1_fail(ZERO1_EINVAL, "%s: dw_pre, rstd_pre, dh, r or r8 without w_pre", call);
    if (io->dgate && cfg->gate_kind == ZERO1_GATE_NONE) return z1_fail(ZERO1_EINVAL, "%s: dgate without a gate", call);
    if (T > 0) {
        if ((rc = check_mat(out[0], er, true, call)) || (rc = check_mat(out[1], ea, true, call)) ||
            (io->dr && (rc = check_mat(in[0], er, false, call))) || (io->gate && (rc = check_mat(in[6], eg, false, call))))
            return rc;
        if (pre) {
            if ((rc = check_mat(in[1], ea, false, call)) || (rc = check_natural(io->w_pre, ep, "w_pre")) ||
                (rc = check_mat(in[8], 4, false, call)))
                return rc;
            if ((io->r != nullptr) == (r8 != nullptr))
                return z1_fail(ZERO1_EINVAL, "%s: exactly one of r and r8 is needed", call);
            if (r8 ? (rc = check_saved(cfg, r8, call, "r8")) : (rc = check_mat(in[3], er, false, call))) return rc;
        }
        if (post && ((rc = check_natural(io->w_post, ep, "w_post")) || (rc = check_mat(in[7], 4, false, call)))) return rc;
        if (io->y && io->y8) return z1_fail(ZERO1_EINVAL, "%s: both y and y8", call);
        if (need_y) {
            if (!y && !y8) return z1_fail(ZERO1_EINVAL, "%s: y or y8 is needed", call);
            if (y8 ? (rc = check_saved(cfg, y8, call, "y8")) : (rc = check_mat(in[2], ea, false, call))) return rc;
        }
        if (!pre && !io->dr) return z1_fail(ZERO1_EINVAL, "%s: neither dh nor dr", call);
    }
    if ((io->dw_post && (rc = check_natural(io->dw_post, ew, "dw_post"))) ||
        (io->dw_pre && (rc = check_natural(io->dw_pre, ew, "dw_pre"))) ||
        (io->dgate && (rc = check_mat(out[4], edg, true, call))))
        return rc;
    if ((rc = check_overlaps(out, in_place, 6, in, 13, call)) != ZERO1_OK) return rc;
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
        if (in_host_memory(workspace)) return z1_fail(ZERO1_EINVAL, "%s: the workspace must be device memory", call);
    }

    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (T > 0) {
        const Common c = common_of(cfg, io->w_post, io->w_pre, io->gate, io->ld_gate, y8, r8);
        Bwd a{};
        a.dh = io->dh; a.dr = io->dr; a.y = y; a.r = io->r;
        a.rstd_post = io->rstd_post; a.rstd_pre = io->rstd_pre;
        a.dy = io->dy; a.dx = io->dx; a.dgate = io->dgate;
        a.ld_dh = io->ld_dh; a.ld_dr = io->ld_dr; a.ld_y = io->ld_y; a.ld_r = io->ld_r;
        a.ld_dy = io->ld_dy; a.ld_dx = io->ld_dx; a.ld_dgate = T > 1 ? io->ld_dgate : 0;
        a.need_post = io->dw_post != nullptr; a.need_pre = io->dw_pre != nullptr; a.need_gate = io->dgate != nullptr;
        a.dgvec = vec_ok(out[4]);
        a.part = static_cast<float *>(workspace);
        const bool vec = D % 8 == 0 && vec_ok(in[0]) && vec_ok(in[1]) && vec_ok(in[2]) && vec_ok(in[3]) &&
                         vec_ok(out[0]) && vec_ok(out[1]);
        rc = dispatch_types(cfg, [&](auto ta, auto tr) {
            return z1bn::run_backward<decltype(ta), decltype(tr)>(c, a, vec, grid, st);
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
    // (without rows the gate is not checked, nor does it matter: the sums are +0)
    f.gate = T > 0 && chan && cfg->gate_act == ZERO1_GATE_SIGMOID ? io->gate : nullptr;
    f.gf32 = cfg->gate_dtype == ZERO1_DTYPE_F32;
    const cudaError_t e = launch_after(k_block_norm_finish, dim3((unsigned)((D + 31) / 32), 3), 256, 0, st, f);
    if (e != cudaSuccess) return pdl_fail(e, "block norm backward: column sums");
    return ZERO1_OK;
}
