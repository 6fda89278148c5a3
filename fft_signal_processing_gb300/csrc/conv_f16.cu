// Short causal convolution of f16 sequences.
#include "conv.cuh"

namespace gbfft {

cudaError_t conv_forward_f16(ConvArgs a, cudaStream_t s) { return conv_run<__half, 4>(a, false, s); }
cudaError_t conv_backward_f16(ConvArgs a, cudaStream_t s) { return conv_run<__half, 4>(a, true, s); }

}  // namespace gbfft
