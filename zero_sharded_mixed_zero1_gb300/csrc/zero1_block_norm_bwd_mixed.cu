// zero1_block_norm_bwd_mixed.cu - block norms, backward: bf16 activations, fp32 residual stream.

#include "zero1_block_norm_bwd.cuh"

template int z1bn::run_backward<uint16_t, float>(const Common &, const Bwd &, bool, int64_t, cudaStream_t);
