// zero1_block_norm_fwd_f32.cu - block norms, forward: fp32 throughout.

#include "zero1_block_norm_fwd.cuh"

template int z1bn::run_forward<float, float>(const Common &, const Fwd &, bool, int, cudaStream_t);
