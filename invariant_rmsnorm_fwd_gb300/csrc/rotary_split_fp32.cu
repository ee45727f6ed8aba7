// Rotary kernels for FP32 heads, halves of other sizes.
#include "rotary_launch.cuh"

template int rbi::rotary_run_pairs<float, rbi::kSplit>(rbi::RotaryParams, int, cudaStream_t);
