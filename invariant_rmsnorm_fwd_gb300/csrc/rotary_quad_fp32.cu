// Rotary kernels for FP32 heads, halves of whole pieces of 4 columns.
#include "rotary_launch.cuh"

template int rbi::rotary_run_pairs<float, rbi::kQuad>(rbi::RotaryParams, int, cudaStream_t);
