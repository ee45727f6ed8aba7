// Rotary kernels for FP32 heads, neighbouring pairs.
#include "rotary_launch.cuh"

template int rbi::rotary_run_pairs<float, rbi::kNear>(rbi::RotaryParams, int, cudaStream_t);
