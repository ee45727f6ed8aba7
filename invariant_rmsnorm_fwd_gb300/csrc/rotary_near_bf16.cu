// Rotary kernels for bf16 heads, neighbouring pairs.
#include "rotary_launch.cuh"

template int rbi::rotary_run_pairs<__nv_bfloat16, rbi::kNear>(rbi::RotaryParams, int, cudaStream_t);
