// Host-side pieces of the layer norm shared by its translation units.
#pragma once
#include <cuda_runtime.h>

#include <mutex>

#include "layernorm_kernels.cuh"
#include "layernorm_bi.h"

namespace rbi {

constexpr int kSmemPerSm = 228 * 1024, kSmemPerCta = 1024;   // an SM's shared memory; what the system takes per CTA

// CTAs that an SM's registers and warps hold: a quarter of an SM has 16,384
// registers, of which a warp takes whole multiples of 256.
inline int resident_ctas(int regs, int threads) {
    const int per_warp = (regs * 32 + 255) / 256 * 256, warps = 16384 / per_warp * 4;
    return (warps < 64 ? warps : 64) / (threads / 32);
}

// What a launcher needs of its kernel, asked for once per device: the registers
// per thread; the kernel's shared-memory limit is raised on the way.  The launchers
// that keep one have internal linkage: a static of a function template with external
// linkage is one object for the whole process, so a second copy of the library in it
// would take the first one's kernels for its own.
struct KernelInfo {
    std::mutex mu;
    uint64_t ready = 0;
    int regs = 0;
    int get(const void *kern, int max_smem, int *out) {
        int dev = 0;
        if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return RMSNORM_ERR_CUDA;
        std::lock_guard<std::mutex> lk(mu);
        if (!((ready >> dev) & 1)) {
            cudaFuncAttributes a;
            if (cudaFuncGetAttributes(&a, kern) != cudaSuccess) return RMSNORM_ERR_CUDA;
            if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, max_smem) != cudaSuccess)
                return RMSNORM_ERR_CUDA;
            regs = a.numRegs;
            ready |= uint64_t(1) << dev;
        }
        *out = regs;
        return RMSNORM_OK;
    }
};

// Launches the rows of one call for element type E (ln_rows_*.cu instantiate it).
// Rows of at most 512 columns take ln_run_narrow (ln_narrow_*.cu).
template <class E>
int ln_run_narrow(const LnParams &p, bool bwd, bool grads, cudaStream_t stream);
template <class E>
int ln_run_rows(const LnParams &p, bool bwd, bool grads, cudaStream_t stream);

}  // namespace rbi
