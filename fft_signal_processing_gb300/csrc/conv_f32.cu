// Short causal convolution of f32 sequences.
#include "conv.cuh"

namespace gbfft {

cudaError_t conv_forward_f32(ConvArgs a, cudaStream_t s) { return conv_run<float, 2>(a, false, s); }
cudaError_t conv_backward_f32(ConvArgs a, cudaStream_t s) { return conv_run<float, 2>(a, true, s); }

}  // namespace gbfft
