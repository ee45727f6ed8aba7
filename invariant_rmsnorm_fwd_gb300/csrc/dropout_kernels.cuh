// Dropout alone (sm_103a): an elementwise pass over the active token slots.
#pragma once
#include <cuda_runtime.h>

#include "layernorm_kernels.cuh"
#include "rmsnorm_bi.h"

namespace rbi {

struct DropoutParams {
    const void *x;
    void *y;
    DropParams drop;
    const int32_t *tok_id;
    int64_t n_tokens, token_stride;
    int32_t rpt, hidden;
};

// One CTA per token slot at a time; thread i takes vectors i, i + blockDim, ...
// of the slot's rows.
template <class E>
__global__ void __launch_bounds__(256) dropout_kernel(const __grid_constant__ DropoutParams p) {
    const DropKey key = drop_key(p.drop);
    const int V = p.hidden >> 3;
    const int64_t n = int64_t(p.rpt) * V;
    for (int64_t t = blockIdx.x; t < p.n_tokens; t += gridDim.x) {
        const int32_t id = p.tok_id[t];
        if (id < 0) continue;
        for (int64_t i = threadIdx.x; i < n; i += blockDim.x) {
            const int64_t r = i / V;
            const uint32_t v = uint32_t(i - r * V);
            const int64_t off = t * p.token_stride + i * 8;
            float f[8];
            unpack(vload<E>(p.x, off), f);
            const uint32_t keep = keep_bits(v, uint32_t(int64_t(id) * p.rpt + r), key, p.drop.t);
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = (keep >> e) & 1 ? __fmul_rn(f[e], p.drop.scale) : 0.f;
            Vec<E> o;
            pack(f, o);
            vstore<E>(p.y, off, o);
        }
    }
}

template <class E>
int dropout_launch(const DropoutParams &p, int sms, cudaStream_t stream) {
    const int64_t cap = int64_t(sms) * 8, grid = p.n_tokens < cap ? p.n_tokens : cap;
    dropout_kernel<E><<<unsigned(grid), 256, 0, stream>>>(p);
    return cudaGetLastError() == cudaSuccess ? RMSNORM_OK : RMSNORM_ERR_CUDA;
}

}  // namespace rbi
