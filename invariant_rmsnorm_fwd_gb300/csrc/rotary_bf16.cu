// Rotary kernels for bf16 heads.
#include "rotary_launch.cuh"

template int rbi::rotary_run<__nv_bfloat16>(rbi::RotaryParams, int, bool, cudaStream_t);
