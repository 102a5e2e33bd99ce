// zero1_block_norm_bwd_bf16.cu - block norms, backward: bf16 activations and residual stream.

#include "zero1_block_norm_bwd.cuh"

template int z1bn::run_backward<uint16_t, uint16_t>(const Common &, const Bwd &, bool, int64_t, cudaStream_t);
