// Short causal convolution of bf16 sequences.
#include "conv.cuh"

namespace gbfft {

cudaError_t conv_forward_bf16(ConvArgs a, cudaStream_t s) { return conv_run<__nv_bfloat16, 4>(a, false, s); }
cudaError_t conv_backward_bf16(ConvArgs a, cudaStream_t s) { return conv_run<__nv_bfloat16, 4>(a, true, s); }

}  // namespace gbfft
