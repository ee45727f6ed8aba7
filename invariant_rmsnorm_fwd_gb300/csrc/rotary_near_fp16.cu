// Rotary kernels for fp16 heads, neighbouring pairs.
#include "rotary_launch.cuh"

template int rbi::rotary_run_pairs<__half, rbi::kNear>(rbi::RotaryParams, int, cudaStream_t);
