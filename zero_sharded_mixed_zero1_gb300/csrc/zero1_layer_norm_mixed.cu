// zero1_layer_norm_mixed.cu - layer norm, bf16 activations, fp32 residual stream.
#include "zero1_layer_norm.cuh"

template int z1ln::run_forward<uint16_t, float>(const Fwd &, bool, int, cudaStream_t);
template int z1ln::run_backward<uint16_t, float>(const Bwd &, bool, int64_t, cudaStream_t);
