// Rotary kernels for FP32 heads, halves of whole vectors.
#include "rotary_launch.cuh"

template int rbi::rotary_run_pairs<float, rbi::kHalf>(rbi::RotaryParams, int, cudaStream_t);
