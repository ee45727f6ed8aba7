// Layer-norm row kernels of more than 512 columns for bf16 rows.
#include "layernorm_launch.cuh"

template int rbi::ln_run_rows<__nv_bfloat16>(const rbi::LnParams &, bool, bool, cudaStream_t);
