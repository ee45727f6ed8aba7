// Rotary kernels for bf16 heads, halves of whole vectors.
#include "rotary_launch.cuh"

template int rbi::rotary_run_pairs<__nv_bfloat16, rbi::kHalf>(rbi::RotaryParams, int, cudaStream_t);
