// Rotary kernels for bf16 heads, halves of whole pieces of 4 columns.
#include "rotary_launch.cuh"

template int rbi::rotary_run_pairs<__nv_bfloat16, rbi::kQuad>(rbi::RotaryParams, int, cudaStream_t);
