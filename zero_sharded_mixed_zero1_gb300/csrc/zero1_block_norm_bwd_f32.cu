// zero1_block_norm_bwd_f32.cu - block norms, backward: fp32 throughout.

#include "zero1_block_norm_bwd.cuh"

template int z1bn::run_backward<float, float>(const Common &, const Bwd &, bool, int64_t, cudaStream_t);
