// C-ABI entry points of the batch-invariant layer norm and of dropout (sm_103a).
#include <cuda_runtime.h>

#include <cmath>

#include "host.cuh"
#include "dropout_kernels.cuh"
#include "layernorm_finalize.cuh"
#include "layernorm_host.cuh"

using namespace rbi;

namespace {

constexpr int64_t kMaxHidden16 = 16384, kMaxHidden32 = 8192, kMaxHiddenDrop = int64_t(1) << 20;

bool bad_align(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }
bool bad_align4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) != 0; }

int ln_check(const rmsnorm_layout_t *L, int64_t H, int64_t max_hidden) {
    if (H < 8 || H % 8 != 0 || H > max_hidden) return RMSNORM_ERR_HIDDEN;
    if (!L) return RMSNORM_ERR_NULL;
    if (L->n_tokens < 0 || L->rows_per_token < 1 || L->reserved0 != 0 || L->n_logical_tokens < 0 ||
        L->plan_items < 0)
        return RMSNORM_ERR_LAYOUT;
    if (L->n_tokens > 0 && !L->tok_id) return RMSNORM_ERR_NULL;
    if (L->token_stride % 8 != 0 || bad_align4(L->tok_id) || bad_align4(L->plan)) return RMSNORM_ERR_ALIGN;
    if (L->token_stride < int64_t(L->rows_per_token) * H) return RMSNORM_ERR_STRIDE;
    const int64_t lim = int64_t(1) << 31;
    if (L->n_tokens >= lim || L->n_logical_tokens >= lim || L->n_tokens * L->rows_per_token >= lim ||
        L->n_logical_tokens * L->rows_per_token >= lim)
        return RMSNORM_ERR_LAYOUT;
    return RMSNORM_OK;
}

int ln_types(int32_t dtype, int32_t param_dtype) {
    if (dtype < LAYERNORM_BF16 || dtype > LAYERNORM_FP32) return RMSNORM_ERR_DTYPE;
    if (param_dtype != dtype && param_dtype != LAYERNORM_FP32) return RMSNORM_ERR_DTYPE;
    return RMSNORM_OK;
}

int64_t ln_max_hidden(int32_t dtype) { return dtype == LAYERNORM_FP32 ? kMaxHidden32 : kMaxHidden16; }

int ln_eps(float eps) { return std::isfinite(eps) && eps >= 0.f ? RMSNORM_OK : RMSNORM_ERR_VALUE; }

// A dropout that drops nothing is still one (its outputs are separate tensors).
int drop_params(const rmsnorm_dropout_t *d, DropParams *out) {
    *out = DropParams{nullptr, 0, 1.f};
    if (!d) return RMSNORM_OK;
    if (!d->state) return RMSNORM_ERR_NULL;
    if ((reinterpret_cast<uintptr_t>(d->state) & 7u) != 0) return RMSNORM_ERR_ALIGN;
    if (!(d->p >= 0.0 && d->p <= 1.0)) return RMSNORM_ERR_VALUE;
    const uint32_t t = uint32_t(std::nearbyint(d->p * 65536.0));
    *out = DropParams{d->state, t, t < 65536u ? float(65536.0 / double(65536u - t)) : 0.f};
    return RMSNORM_OK;
}

LnParams ln_params(const rmsnorm_layout_t *L, int64_t H, float eps, int32_t dtype, int32_t param_dtype) {
    LnParams p = {};
    p.grad_scale = 1.f;
    p.eps = eps;
    p.inv_h = float(1.0 / double(H));
    p.params_f32 = param_dtype == LAYERNORM_FP32 && dtype != LAYERNORM_FP32 ? 1 : 0;
    p.hidden = int32_t(H);
    p.rpt = L->rows_per_token;
    p.tok_id = L->tok_id;
    p.n_rows = L->n_tokens * L->rows_per_token;
    p.token_stride = L->token_stride;
    p.items = static_cast<const PlanItem *>(L->plan);
    p.n_items = L->plan ? L->plan_items : 0;
    return p;
}

int run(const LnParams &p, int32_t dtype, bool bwd, bool grads, rmsnorm_stream_t stream) {
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    switch (dtype) {
        case LAYERNORM_BF16: return ln_run_rows<__nv_bfloat16>(p, bwd, grads, s);
        case LAYERNORM_FP16: return ln_run_rows<__half>(p, bwd, grads, s);
        default: return ln_run_rows<float>(p, bwd, grads, s);
    }
}

int ln_ws_check(const void *ws, int64_t N, int64_t H) {
    if (!ws) return RMSNORM_ERR_NULL;
    if ((reinterpret_cast<uintptr_t>(ws) & 255u) != 0) return RMSNORM_ERR_ALIGN;
    if (N < 0 || N >= (int64_t(1) << 31)) return RMSNORM_ERR_LAYOUT;
    if (H < 8 || H % 8 != 0 || H > kMaxHidden16) return RMSNORM_ERR_HIDDEN;
    return RMSNORM_OK;
}

}  // namespace

extern "C" int layernorm_fwd(const void *x, const void *weight, const void *bias, int64_t hidden, float eps,
                             int32_t dtype, int32_t param_dtype, const rmsnorm_layout_t *layout, void *y,
                             float *mean, float *rstd, rmsnorm_stream_t stream) {
    int rc = ln_types(dtype, param_dtype);
    if (rc || (rc = ln_check(layout, hidden, ln_max_hidden(dtype))) || (rc = ln_eps(eps))) return rc;
    if (layout->n_tokens == 0) return RMSNORM_OK;
    if (!x || !y) return RMSNORM_ERR_NULL;
    if (bad_align(x) || bad_align(weight) || bad_align(bias) || bad_align(y) || bad_align4(mean) || bad_align4(rstd))
        return RMSNORM_ERR_ALIGN;
    LnParams p = ln_params(layout, hidden, eps, dtype, param_dtype);
    p.x = x;
    p.w = weight;
    p.b = bias;
    p.out = y;
    p.mean = mean;
    p.rstd = rstd;
    return run(p, dtype, false, false, stream);
}

extern "C" int layernorm_add_fwd(const void *x, const void *residual, const void *weight, const void *bias,
                                 int64_t hidden, float eps, int32_t dtype, int32_t param_dtype,
                                 const rmsnorm_layout_t *layout, const rmsnorm_dropout_t *dropout, void *h_out,
                                 void *y, float *mean, float *rstd, rmsnorm_stream_t stream) {
    int rc = ln_types(dtype, param_dtype);
    if (rc || (rc = ln_check(layout, hidden, ln_max_hidden(dtype))) || (rc = ln_eps(eps))) return rc;
    DropParams drop;
    if ((rc = drop_params(dropout, &drop))) return rc;
    if (layout->n_tokens == 0) return RMSNORM_OK;
    if (!x || !residual || !h_out || !y) return RMSNORM_ERR_NULL;
    if (h_out == y) return RMSNORM_ERR_LAYOUT;
    if (bad_align(x) || bad_align(residual) || bad_align(weight) || bad_align(bias) || bad_align(h_out) || bad_align(y) ||
        bad_align4(mean) || bad_align4(rstd))
        return RMSNORM_ERR_ALIGN;
    LnParams p = ln_params(layout, hidden, eps, dtype, param_dtype);
    p.x = x;
    p.res = residual;
    p.w = weight;
    p.b = bias;
    p.out = y;
    p.out2 = h_out;
    p.mean = mean;
    p.rstd = rstd;
    p.drop = drop;
    return run(p, dtype, false, false, stream);
}

extern "C" int layernorm_add_bwd(const void *h, const void *weight, const void *dy, const void *dres, int64_t hidden,
                                 float eps, float grad_scale, int32_t dtype, int32_t param_dtype,
                                 const rmsnorm_layout_t *layout, const rmsnorm_dropout_t *dropout, void *dh, void *dx,
                                 void *workspace, rmsnorm_stream_t stream) {
    int rc = ln_types(dtype, param_dtype);
    if (rc || (rc = ln_check(layout, hidden, ln_max_hidden(dtype))) || (rc = ln_eps(eps))) return rc;
    if (!std::isfinite(grad_scale)) return RMSNORM_ERR_VALUE;
    DropParams drop;
    if ((rc = drop_params(dropout, &drop))) return rc;
    if (!dh && (!workspace || dres || dropout) && layout->n_tokens > 0) return RMSNORM_ERR_NULL;
    if (dropout && !dx && layout->n_tokens > 0) return RMSNORM_ERR_NULL;
    if (dropout && dh == dx && layout->n_tokens > 0) return RMSNORM_ERR_LAYOUT;
    if (workspace && !layout->plan && layout->n_tokens > 0) return RMSNORM_ERR_PLAN;
    const int64_t N = layout->n_logical_tokens * layout->rows_per_token;
    if (workspace && (rc = ln_ws_check(workspace, N, hidden))) return rc;
    if (layout->n_tokens == 0) return RMSNORM_OK;
    if (!h || !dy) return RMSNORM_ERR_NULL;
    if (bad_align(h) || bad_align(weight) || bad_align(dy) || bad_align(dres) || bad_align(dh) ||
        (dropout && bad_align(dx)))
        return RMSNORM_ERR_ALIGN;
    LnParams p = ln_params(layout, hidden, eps, dtype, param_dtype);
    p.x = h;
    p.w = weight;
    p.dy = dy;
    p.res = dres;
    p.out = dh;
    p.out2 = dropout ? dx : nullptr;
    p.drop = drop;
    p.grad_scale = grad_scale;
    if (workspace) p.ws = ln_ws(workspace, N, hidden);
    return run(p, dtype, true, workspace != nullptr, stream);
}

extern "C" int layernorm_bwd(const void *x, const void *weight, const void *dy, int64_t hidden, float eps,
                             int32_t dtype, int32_t param_dtype, const rmsnorm_layout_t *layout, void *dx,
                             void *workspace, rmsnorm_stream_t stream) {
    return layernorm_add_bwd(x, weight, dy, nullptr, hidden, eps, 1.f, dtype, param_dtype, layout, nullptr, dx,
                             nullptr, workspace, stream);
}

extern "C" size_t layernorm_workspace_bytes(int64_t n_logical_rows, int64_t hidden) {
    if (n_logical_rows < 0 || n_logical_rows >= (int64_t(1) << 31) || hidden < 8 || hidden % 8 != 0 ||
        hidden > kMaxHidden16)
        return 0;
    return size_t(LnWsLayout(n_logical_rows, hidden).total);
}

extern "C" int layernorm_begin(void *workspace, size_t bytes, int64_t n_logical_rows, int64_t hidden,
                               rmsnorm_stream_t stream) {
    int rc = ln_ws_check(workspace, n_logical_rows, hidden);
    if (rc) return rc;
    if (bytes < layernorm_workspace_bytes(n_logical_rows, hidden)) return RMSNORM_ERR_WORKSPACE;
    DeviceInfo *d = nullptr;
    if ((rc = device_info(&d))) return rc;
    const LnWs ws = ln_ws(workspace, n_logical_rows, hidden);
    const int64_t n16 = (reinterpret_cast<uint8_t *>(ws.partial) - ws.state) / 16;
    int64_t blocks = (n16 + 255) / 256;
    if (blocks > int64_t(d->sms) * 4) blocks = int64_t(d->sms) * 4;
    if (blocks < 1) blocks = 1;
    ln_begin_kernel<<<unsigned(blocks), 256, 0, reinterpret_cast<cudaStream_t>(stream)>>>(ws);
    if (cudaGetLastError() != cudaSuccess) return RMSNORM_ERR_CUDA;
    count_launch();
    return RMSNORM_OK;
}

extern "C" int layernorm_finalize(void *workspace, int64_t n_logical_rows, int64_t hidden, float grad_scale,
                                  float *dweight, float *dbias, rmsnorm_stream_t stream) {
    if (!std::isfinite(grad_scale)) return RMSNORM_ERR_VALUE;
    int rc = ln_ws_check(workspace, n_logical_rows, hidden);
    if (rc) return rc;
    if (!dweight && !dbias) return RMSNORM_ERR_NULL;
    if (bad_align(dweight) || bad_align(dbias)) return RMSNORM_ERR_ALIGN;
    DeviceInfo *d = nullptr;
    if ((rc = device_info(&d))) return rc;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const LnWs ws = ln_ws(workspace, n_logical_rows, hidden);
    if (ws.n_blocks == 0) {
        if (dweight && cudaMemsetAsync(dweight, 0, size_t(hidden) * 4, s) != cudaSuccess) return RMSNORM_ERR_CUDA;
        if (dbias && cudaMemsetAsync(dbias, 0, size_t(hidden) * 4, s) != cudaSuccess) return RMSNORM_ERR_CUDA;
        return RMSNORM_OK;
    }
    const unsigned gy = unsigned((2 * hidden + kLnTreeCols - 1) / kLnTreeCols);
    const float *in = nullptr;
    float *scratch[2] = {ws.scratch_a, ws.scratch_b};
    int flip = 0;
    for (int64_t n = ws.n_blocks;;) {
        const int64_t per = in ? kLnTreeNodes : kLnTreeBlocks, groups = (n + per - 1) / per;
        const bool last = groups == 1;
        float *dst = scratch[flip];
        auto kern = in ? ln_tree_kernel<false> : ln_tree_kernel<true>;
        kern<<<dim3(unsigned(groups), gy), 256, 0, s>>>(
            ws, in, last ? dweight : dst, last ? dbias : dst + hidden, last ? 0 : 2 * hidden, n,
            last ? grad_scale : 1.f);
        if (cudaGetLastError() != cudaSuccess) return RMSNORM_ERR_CUDA;
        count_launch();
        if (last) return RMSNORM_OK;
        in = dst;
        n = groups;
        flip ^= 1;
    }
}

extern "C" int layernorm_status(const void *workspace, rmsnorm_stream_t stream, int32_t *status) {
    return rmsnorm_dweight_status(workspace, stream, status);
}

extern "C" int dropout_fwd(const void *x, int64_t hidden, int32_t dtype, const rmsnorm_layout_t *layout,
                           const rmsnorm_dropout_t *dropout, void *y, rmsnorm_stream_t stream) {
    int rc = ln_types(dtype, dtype);
    if (rc || (rc = ln_check(layout, hidden, kMaxHiddenDrop))) return rc;
    if (!dropout) return RMSNORM_ERR_NULL;
    DropParams drop;
    if ((rc = drop_params(dropout, &drop))) return rc;
    if (layout->n_tokens == 0) return RMSNORM_OK;
    if (!x || !y) return RMSNORM_ERR_NULL;
    if (bad_align(x) || bad_align(y)) return RMSNORM_ERR_ALIGN;
    DeviceInfo *d = nullptr;
    if ((rc = device_info(&d))) return rc;
    const DropoutParams p = {x, y, drop, layout->tok_id, layout->n_tokens * layout->rows_per_token, layout->token_stride,
                             layout->rows_per_token, int32_t(hidden)};
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    switch (dtype) {
        case LAYERNORM_BF16: return dropout_launch<__nv_bfloat16>(p, s);
        case LAYERNORM_FP16: return dropout_launch<__half>(p, s);
        default: return dropout_launch<float>(p, s);
    }
}

extern "C" int dropout_bwd(const void *dy, int64_t hidden, int32_t dtype, const rmsnorm_layout_t *layout,
                           const rmsnorm_dropout_t *dropout, void *dx, rmsnorm_stream_t stream) {
    return dropout_fwd(dy, hidden, dtype, layout, dropout, dx, stream);
}
