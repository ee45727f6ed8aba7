// Launcher of the rotary kernels, instantiated per element type.
#pragma once
#include "rotary_kernels.cuh"

namespace rbi {

inline int lanes_pow2(int lanes) {
    int p = 1;
    while (p < lanes) p <<= 1;
    return p;
}

template <class E, bool INTER, bool WIDE>
static int rotary_launch(RotaryParams &p, int mode, cudaStream_t stream) {
    const int lanes = (p.D + 15) / 16;
    if (mode <= 1) {
        p.team = mode == 0 ? (p.in_place ? (p.rot + 15) / 16 : lanes) : lanes_pow2(lanes);
        p.by_team = Divisor(uint32_t(p.team));
        const uint32_t teams = uint32_t(kRotaryThreads / p.team);
        p.units = uint32_t(p.n_tokens * p.chunks);
        const unsigned grid = (p.units + teams - 1) / teams;
        if (mode == 0) rotary_kernel<E, INTER, WIDE, false><<<grid, kRotaryThreads, 0, stream>>>(p);
        else rotary_kernel<E, INTER, WIDE, true><<<grid, kRotaryThreads, 0, stream>>>(p);
    } else {
        p.team = lanes_pow2(lanes);
        p.units = uint32_t((p.n_tokens + kQkGroup - 1) / kQkGroup * p.chunks);
        const unsigned grid = (p.units + kQkWarps - 1) / kQkWarps;
        if (mode == 2) {
            qk_bwd_kernel<E, INTER, WIDE, false><<<grid, kQkWarps * 32, 0, stream>>>(p);
        } else {
            auto kern = qk_bwd_kernel<E, INTER, WIDE, true>;
            static KernelInfo info;
            DeviceInfo *d = nullptr;
            int regs = 0;
            if (int rc = device_info(&d)) return rc;
            if (int rc = info.get(reinterpret_cast<const void *>(kern), d->max_smem, &regs)) return rc;
            kern<<<grid, kQkWarps * 32, size_t(kQkWarps) * kQkGroup * p.D * 4, stream>>>(p);
        }
    }
    if (cudaGetLastError() != cudaSuccess) return RMSNORM_ERR_CUDA;
    count_launch();
    return RMSNORM_OK;
}

template <class E>
int rotary_run(RotaryParams p, int mode, bool interleaved, cudaStream_t stream) {
    // Vectors of 8 columns where the rotation is made of whole ones, else pieces of two.
    const bool wide = p.first % 8 == 0 && p.rot % (interleaved ? 8 : 16) == 0;
    if (interleaved) return wide ? rotary_launch<E, true, true>(p, mode, stream) : rotary_launch<E, true, false>(p, mode, stream);
    return wide ? rotary_launch<E, false, true>(p, mode, stream) : rotary_launch<E, false, false>(p, mode, stream);
}

}  // namespace rbi
