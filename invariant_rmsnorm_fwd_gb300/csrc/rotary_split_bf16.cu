// Rotary kernels for bf16 heads, halves of other sizes.
#include "rotary_launch.cuh"

template int rbi::rotary_run_pairs<__nv_bfloat16, rbi::kSplit>(rbi::RotaryParams, int, cudaStream_t);
