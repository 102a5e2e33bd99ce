// zero1_layer_norm_bf16.cu - layer norm, bf16 activations, bf16 residual stream.
#include "zero1_layer_norm.cuh"

template int z1ln::run_forward<uint16_t, uint16_t>(const Fwd &, bool, int, cudaStream_t);
template int z1ln::run_backward<uint16_t, uint16_t>(const Bwd &, bool, int64_t, cudaStream_t);
