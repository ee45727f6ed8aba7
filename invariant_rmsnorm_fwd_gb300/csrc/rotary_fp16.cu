// Rotary kernels for fp16 heads.
#include "rotary_launch.cuh"

template int rbi::rotary_run<__half>(rbi::RotaryParams, int, bool, cudaStream_t);
