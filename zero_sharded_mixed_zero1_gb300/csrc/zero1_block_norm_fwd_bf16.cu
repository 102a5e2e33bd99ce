// zero1_block_norm_fwd_bf16.cu - block norms, forward: bf16 activations and residual stream.

#include "zero1_block_norm_fwd.cuh"

template int z1bn::run_forward<uint16_t, uint16_t>(const Common &, const Fwd &, bool, int, cudaStream_t);
