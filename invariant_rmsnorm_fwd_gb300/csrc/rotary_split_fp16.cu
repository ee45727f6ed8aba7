// Rotary kernels for fp16 heads, halves of other sizes.
#include "rotary_launch.cuh"

template int rbi::rotary_run_pairs<__half, rbi::kSplit>(rbi::RotaryParams, int, cudaStream_t);
