// Launcher of the rotary kernels, instantiated per element type and kind of pairs.
#pragma once
#include "rotary_kernels.cuh"

namespace rbi {

template <class E, int PAIRS>
static int rotary_launch_alone(RotaryParams &p, cudaStream_t stream) {
    // No team of a power of two but where it exchanges columns.
    p.team = PAIRS == kSplit ? qk_team(p.D) : PAIRS == kHalf && p.in_place ? p.rot / 16 : p.lanes;
    p.by_team = Divisor(uint32_t(p.team));
    const uint32_t teams = uint32_t(kRotaryThreads / p.team);
    p.units = uint32_t(p.n_tokens * p.chunks);
    rotary_kernel<E, PAIRS><<<(p.units + teams - 1) / teams, kRotaryThreads, PAIRS == kSplit ? int(teams) * p.D * 4 : 0, stream>>>(p);
    if (cudaGetLastError() != cudaSuccess) return RMSNORM_ERR_CUDA;
    count_launch();
    return RMSNORM_OK;
}

template <class E, int PAIRS, int TEAM>
static int rotary_launch_fwd(RotaryParams &p, cudaStream_t stream) {
    auto kern = qk_fwd_kernel<E, PAIRS, TEAM>;
    static KernelInfo info;
    DeviceInfo *d = nullptr;
    int regs = 0;
    if (int rc = device_info(&d)) return rc;
    if (int rc = info.get(reinterpret_cast<const void *>(kern), d->max_smem, &regs)) return rc;
    // Steps of a warp: up to 4 while that leaves every SM 32 warps' work.
    const int teams = 32 / p.team;
    int slots = teams;
    while (slots < 32 && slots < 4 * teams && p.n_tokens * p.chunks >= int64_t(2) * slots * 32 * d->sms) slots *= 2;
    p.units = uint32_t((p.n_tokens + slots - 1) / slots * p.chunks);
    kern<<<(p.units + kQkWarps - 1) / kQkWarps, kQkWarps * 32,
           16 * p.D + kQkWarps * (Ring<E, 1>::kBytes + (PAIRS == kSplit ? 2048 : 0)), stream>>>(p, slots);
    if (cudaGetLastError() != cudaSuccess) return RMSNORM_ERR_CUDA;
    count_launch();
    return RMSNORM_OK;
}

template <class E, int PAIRS, int TEAM>
static int rotary_launch_bwd(RotaryParams &p, cudaStream_t stream) {
    auto kern = qk_bwd_kernel<E, PAIRS, TEAM>;
    static KernelInfo info;
    DeviceInfo *d = nullptr;
    int regs = 0;
    if (int rc = device_info(&d)) return rc;
    if (int rc = info.get(reinterpret_cast<const void *>(kern), d->max_smem, &regs)) return rc;
    p.units = uint32_t((p.n_tokens + kQkGroup - 1) / kQkGroup * p.chunks);
    const bool straddles = p.hq % p.per != 0 && p.heads > p.hq;
    kern<<<(p.units + kQkWarps - 1) / kQkWarps, kQkWarps * 32,
           qk_bwd_smem(Ring<E, 2>::kBytes, p.D, PAIRS == kSplit, p.ws.hdr != nullptr, straddles), stream>>>(p, straddles);
    if (cudaGetLastError() != cudaSuccess) return RMSNORM_ERR_CUDA;
    count_launch();
    return RMSNORM_OK;
}

template <class E, int PAIRS, int TEAM>
static int rotary_launch_norm(RotaryParams &p, int mode, cudaStream_t stream) {
    return mode == 1 ? rotary_launch_fwd<E, PAIRS, TEAM>(p, stream) : rotary_launch_bwd<E, PAIRS, TEAM>(p, stream);
}

template <class E, int PAIRS>
static int rotary_launch(RotaryParams &p, int mode, cudaStream_t stream) {
    if (mode == 0) return rotary_launch_alone<E, PAIRS>(p, stream);
    p.team = qk_team(p.D);
    if constexpr (PAIRS != kSplit) {
        if (p.team == 4) return rotary_launch_norm<E, PAIRS, 4>(p, mode, stream);
        if (p.team == 8) return rotary_launch_norm<E, PAIRS, 8>(p, mode, stream);
        if (p.team == 16) return rotary_launch_norm<E, PAIRS, 16>(p, mode, stream);
    }
    return rotary_launch_norm<E, PAIRS, 0>(p, mode, stream);
}

// One translation unit per element type and kind of pairs (rotary_*.cu).
template <class E, int PAIRS>
int rotary_run_pairs(RotaryParams p, int mode, cudaStream_t stream) {
    p.lanes = (p.D + 15) / 16;
    const QkChunks cut(p.hq, p.heads - p.hq);
    p.chunks = cut.chunks;
    p.per = cut.per;
    p.by_chunks = Divisor(uint32_t(p.chunks));
    return rotary_launch<E, PAIRS>(p, mode, stream);
}

}  // namespace rbi
