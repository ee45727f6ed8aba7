// Host-side pieces of the layer norm shared by its translation units.
#pragma once
#include <cuda_runtime.h>

#include "layernorm_kernels.cuh"
#include "layernorm_bi.h"

namespace rbi {

// Launches the rows of one call for element type E (ln_rows_*.cu instantiate it).
// Rows of at most 256 columns take ln_run_narrow (ln_narrow_*.cu).
template <class E>
int ln_run_narrow(const LnParams &p, bool bwd, bool grads, cudaStream_t stream);
template <class E>
int ln_run_rows(const LnParams &p, bool bwd, bool grads, cudaStream_t stream);

}  // namespace rbi
