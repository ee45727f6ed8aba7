// Rotary kernels for fp16 heads, halves of whole pieces of 4 columns.
#include "rotary_launch.cuh"

template int rbi::rotary_run_pairs<__half, rbi::kQuad>(rbi::RotaryParams, int, cudaStream_t);
