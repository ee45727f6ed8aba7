// Layer-norm row kernels of more than 512 columns for fp16 rows.
#include "layernorm_launch.cuh"

template int rbi::ln_run_rows<__half>(const rbi::LnParams &, bool, bool, cudaStream_t);
