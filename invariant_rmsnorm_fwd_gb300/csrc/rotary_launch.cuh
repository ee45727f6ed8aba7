// Launcher of the rotary kernels, instantiated per element type.
#pragma once
#include "rotary_kernels.cuh"

namespace rbi {

inline int lanes_pow2(int lanes) {
    int p = 1;
    while (p < lanes) p <<= 1;
    return p;
}

template <class E, int PAIRS, bool NORM>
static int rotary_launch_fwd(RotaryParams &p, cudaStream_t stream) {
    constexpr int U = sizeof(E) == 4 ? 2 : 4;
    p.team = NORM || PAIRS == kSplit ? lanes_pow2(p.lanes) : PAIRS == kHalf && p.in_place ? p.rot / 16 : p.lanes;
    p.by_team = Divisor(uint32_t(p.team));
    const uint32_t teams = uint32_t(kRotaryThreads / p.team);
    p.units = uint32_t(p.n_tokens * p.chunks);
    const int smem = (NORM ? 16 * p.D : 0) + (PAIRS == kSplit ? int(teams) * p.D * 4 : 0);
    rotary_kernel<E, PAIRS, NORM, U><<<(p.units + teams - 1) / teams, kRotaryThreads, smem, stream>>>(p);
    if (cudaGetLastError() != cudaSuccess) return RMSNORM_ERR_CUDA;
    count_launch();
    return RMSNORM_OK;
}

template <class E, int PAIRS, bool GRADS>
static int rotary_launch_bwd(RotaryParams &p, cudaStream_t stream) {
    auto kern = qk_bwd_kernel<E, PAIRS, GRADS>;
    static KernelInfo info;
    DeviceInfo *d = nullptr;
    int regs = 0;
    if (int rc = device_info(&d)) return rc;
    if (int rc = info.get(reinterpret_cast<const void *>(kern), d->max_smem, &regs)) return rc;
    p.team = lanes_pow2(p.lanes);
    p.units = uint32_t((p.n_tokens + kQkGroup - 1) / kQkGroup * p.chunks);
    const bool straddles = p.hq % p.per != 0 && p.heads > p.hq;
    kern<<<(p.units + kQkWarps - 1) / kQkWarps, kQkWarps * 32,
           qk_bwd_smem(Ring<E>::kBytes, p.D, PAIRS == kSplit, GRADS, straddles), stream>>>(p, straddles);
    if (cudaGetLastError() != cudaSuccess) return RMSNORM_ERR_CUDA;
    count_launch();
    return RMSNORM_OK;
}

template <class E, int PAIRS>
static int rotary_launch(RotaryParams &p, int mode, cudaStream_t stream) {
    switch (mode) {
        case 0: return rotary_launch_fwd<E, PAIRS, false>(p, stream);
        case 1: return rotary_launch_fwd<E, PAIRS, true>(p, stream);
        case 2: return rotary_launch_bwd<E, PAIRS, false>(p, stream);
        default: return rotary_launch_bwd<E, PAIRS, true>(p, stream);
    }
}

template <class E>
int rotary_run(RotaryParams p, int mode, bool interleaved, cudaStream_t stream) {
    p.lanes = (p.D + 15) / 16;
    const QkChunks cut(p.hq, p.heads - p.hq);
    p.chunks = cut.chunks;
    p.per = cut.per;
    p.by_chunks = Divisor(uint32_t(p.chunks));
    if (interleaved) return rotary_launch<E, kNear>(p, mode, stream);
    return p.first % 8 == 0 && p.rot % 16 == 0 ? rotary_launch<E, kHalf>(p, mode, stream) : rotary_launch<E, kSplit>(p, mode, stream);
}

}  // namespace rbi
