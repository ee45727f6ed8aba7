// Rotary kernels for fp16 heads, halves of whole vectors.
#include "rotary_launch.cuh"

template int rbi::rotary_run_pairs<__half, rbi::kHalf>(rbi::RotaryParams, int, cudaStream_t);
