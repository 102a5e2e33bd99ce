// zero1_block_norm_fwd_mixed.cu - block norms, forward: bf16 activations, fp32 residual stream.

#include "zero1_block_norm_fwd.cuh"

template int z1bn::run_forward<uint16_t, float>(const Common &, const Fwd &, bool, int, cudaStream_t);
