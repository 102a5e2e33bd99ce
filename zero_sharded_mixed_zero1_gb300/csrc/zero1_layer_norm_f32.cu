// zero1_layer_norm_f32.cu - layer norm, fp32 activations, fp32 residual stream.
#include "zero1_layer_norm.cuh"

template int z1ln::run_forward<float, float>(const Fwd &, bool, int, cudaStream_t);
template int z1ln::run_backward<float, float>(const Bwd &, bool, int64_t, cudaStream_t);
