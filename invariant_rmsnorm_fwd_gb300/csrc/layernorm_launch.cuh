// Launcher of the layer-norm row kernels, instantiated per element type.
#pragma once
#include "host.cuh"
#include "layernorm_host.cuh"

namespace rbi {

template <class E, int NV>
int ln_launch(const LnParams &p, bool bwd, bool grads, cudaStream_t stream) {
    const int V = p.hidden / 8, per = (V + NV - 1) / NV, threads = (per + 31) / 32 * 32;
    const int64_t grid = grads ? p.n_items * kGroups : p.n_rows;
    if (grid == 0) return RMSNORM_OK;
    if (grid >= (int64_t(1) << 31)) return RMSNORM_ERR_LAYOUT;
    if (grads) ln_rows_kernel<E, NV, true, true><<<unsigned(grid), threads, 0, stream>>>(p);
    else if (bwd) ln_rows_kernel<E, NV, true, false><<<unsigned(grid), threads, 0, stream>>>(p);
    else ln_rows_kernel<E, NV, false, false><<<unsigned(grid), threads, 0, stream>>>(p);
    if (cudaGetLastError() != cudaSuccess) return RMSNORM_ERR_CUDA;
    count_launch();
    return RMSNORM_OK;
}

template <class E>
int ln_run_rows(const LnParams &p, bool bwd, bool grads, cudaStream_t stream) {
    DeviceInfo *d = nullptr;
    if (int rc = device_info(&d)) return rc;
    const int V = p.hidden / 8;
    if (V <= 512) return ln_launch<E, 1>(p, bwd, grads, stream);
    if (V <= 1024) return ln_launch<E, 2>(p, bwd, grads, stream);
    if constexpr (sizeof(E) == 2) return ln_launch<E, 4>(p, bwd, grads, stream);
    return RMSNORM_ERR_HIDDEN;
}

}  // namespace rbi
