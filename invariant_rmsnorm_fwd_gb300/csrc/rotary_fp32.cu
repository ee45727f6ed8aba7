// Rotary kernels for FP32 heads.
#include "rotary_launch.cuh"

template int rbi::rotary_run<float>(rbi::RotaryParams, int, bool, cudaStream_t);
