// Layer-norm row kernels of at most 512 columns for bf16 rows.
#include "layernorm_narrow.cuh"

template int rbi::ln_run_narrow<__nv_bfloat16>(const rbi::LnParams &, bool, bool, cudaStream_t);
