// Launcher of the streaming layer-norm kernel, instantiated per element type.
#pragma once
#include "host.cuh"
#include "layernorm_host.cuh"
#include "layernorm_stream.cuh"

namespace rbi {

template <class E, int NV, int MODE, bool DROP, bool GRADS, int MAXT, int MINB>
static int ln_launch_stream_t(const LnParams &p, int threads, const DeviceInfo &d, cudaStream_t stream) {
    auto kern = ln_stream_kernel<E, NV, MODE, DROP, GRADS, MAXT, MINB>;
    static KernelInfo info;
    int regs = 0;
    if (int rc = info.get(reinterpret_cast<const void *>(kern), d.max_smem, &regs)) return rc;
    // Resident CTAs by registers and threads, then as many stages as their share of
    // the shared memory holds; fewer CTAs where that leaves less than `want`.
    // Backward, row i + 1 arrives while row i is in use and the stage of row i - 1
    // is being refilled: three stages at least, and more of them are not worth
    // warps (residual-add backward of 64 M bf16 elements, three staged tensors,
    // 3 / 4 stages wanted: hidden 5120 165 / 218 us, 1024 169 / 176; 6 wanted:
    // hidden 4096 225 against 171).  Forward has more warps than it needs: 5 wanted
    // against 3 take the FP32 forward of 1024 columns from 60 to 53 us, the
    // residual-add one in bf16 from 130 to 101, and change nothing else by 2 %;
    // 7 wanted cost 40 % at hidden 5120.
    const int row = NV * threads * 16;                   // a staged row, padded to whole vectors of the CTA
    const int least = MODE == kLnBwd ? 3 : 2, want = MODE == kLnBwd ? 3 : 5;
    int nt = MODE == kLnFwd ? 1 : MODE == kLnAdd ? 2 : p.res ? 3 : 2;
    if (MODE == kLnBwd && nt == 3 && kFixedBytes + least * nt * row > d.max_smem) nt = 2;
    // tensor memory of a CTA: the sums and the fold of its warps, four side by side
    int cols = 0;
    if (GRADS) {
        cols = 32;
        while (cols < (threads + 127) / 128 * 4 * NV * Lane<E>::kE) cols *= 2;
    }
    int ctas = resident_ctas(regs, threads);
    if (GRADS && ctas > 512 / cols) ctas = 512 / cols;
    if (ctas < 1) return RMSNORM_ERR_HIDDEN;
    int S = 0;
    for (; ctas >= 1; --ctas) {
        int room = kSmemPerSm / ctas - kSmemPerCta;
        if (room > d.max_smem) room = d.max_smem;
        S = (room - kFixedBytes) / (nt * row);
        if (S >= want || (ctas == 1 && S >= least)) break;
    }
    if (ctas < 1) return RMSNORM_ERR_HIDDEN;
    if (S > kMaxStages) S = kMaxStages;
    const int smem = kFixedBytes + S * nt * row;
    int64_t grid = int64_t(ctas) * d.sms;
    const int64_t units = GRADS ? p.n_items * kGroups : p.n_rows;
    if (units == 0) return RMSNORM_OK;
    if (grid > units) grid = units;
    LnParams q = p;
    q.share = int32_t(units / grid);
    q.share_rest = int32_t(units % grid);
    kern<<<unsigned(grid), threads, smem, stream>>>(q, S, nt, cols);
    if (cudaGetLastError() != cudaSuccess) return RMSNORM_ERR_CUDA;
    count_launch();
    return RMSNORM_OK;
}

template <class E, int NV, int MODE, bool DROP, bool GRADS>
int ln_launch_stream(const LnParams &p, const DeviceInfo &d, cudaStream_t stream) {
    const int V = p.hidden / Lane<E>::kE, per = (V + NV - 1) / NV, threads = (per + 31) / 32 * 32;
    // Two CTAs of up to 320 threads fit an SM at 96 registers a thread; FP32's
    // residual add with dropout needs 119 and is faster alone than spilled (hidden
    // 5120, 32 M elements: 92 against 112 us).
    constexpr bool kPair320 = NV * Lane<E>::kE == 16 && !(sizeof(E) == 4 && MODE == kLnAdd && DROP);
    if constexpr (NV * Lane<E>::kE <= 16) {              // wider threads: rows of more than 8192 columns only
        if (threads <= 256) return ln_launch_stream_t<E, NV, MODE, DROP, GRADS, 256, 2>(p, threads, d, stream);
        if constexpr (kPair320) {
            if (threads <= 320) return ln_launch_stream_t<E, NV, MODE, DROP, GRADS, 320, 2>(p, threads, d, stream);
        }
    }
    return ln_launch_stream_t<E, NV, MODE, DROP, GRADS, 512, 1>(p, threads, d, stream);
}

template <class E, int NV>
int ln_launch_mode(const LnParams &p, bool bwd, bool grads, const DeviceInfo &d, cudaStream_t s) {
    const bool drop = p.drop.state != nullptr;
    if (!bwd) {
        if (!p.res) return ln_launch_stream<E, NV, kLnFwd, false, false>(p, d, s);
        return drop ? ln_launch_stream<E, NV, kLnAdd, true, false>(p, d, s)
                    : ln_launch_stream<E, NV, kLnAdd, false, false>(p, d, s);
    }
    if (grads) return drop ? ln_launch_stream<E, NV, kLnBwd, true, true>(p, d, s)
                           : ln_launch_stream<E, NV, kLnBwd, false, true>(p, d, s);
    return drop ? ln_launch_stream<E, NV, kLnBwd, true, false>(p, d, s)
                : ln_launch_stream<E, NV, kLnBwd, false, false>(p, d, s);
}

template <class E>
int ln_run_rows(const LnParams &p, bool bwd, bool grads, cudaStream_t stream) {
    DeviceInfo *d = nullptr;
    if (int rc = device_info(&d)) return rc;
    if (p.hidden <= 512) return ln_run_narrow<E>(p, bwd, grads, stream);
    // Vectors per thread: two of 8 elements (FP32: four of 4), in the widest rows twice
    // that.  Rows of up to 512 columns are teams of lanes: a CTA of one or two warps
    // pays its barrier for too few columns (64 M bf16 elements, this kernel against
    // teams: hidden 512 forward 64 / 50 us, backward 138 / 98; hidden 264 118 / 73
    // and 235 / 147).  The rule looks at hidden size and type alone, so every call
    // sums a row in the same order.
    if constexpr (sizeof(E) == 4) {
        return ln_launch_mode<E, 4>(p, bwd, grads, *d, stream);
    } else {
        if (p.hidden <= 8192) return ln_launch_mode<E, 2>(p, bwd, grads, *d, stream);
        return ln_launch_mode<E, 4>(p, bwd, grads, *d, stream);
    }
}

}  // namespace rbi
