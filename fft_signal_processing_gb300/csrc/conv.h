// Short causal convolution: arguments of the kernels and the per-type launchers (conv.cuh).
#pragma once

#include "seq_common.cuh"

namespace gbfft {

struct ConvArgs {
    fft_conv_desc d;
    fft_seq out;        // forward: out; backward: dx (data may be null)
    fft_seq dout;       // backward
    void* final_state;  // forward: final state; backward: its gradient (read), or null
    void* dinitial;     // backward, or null
    float* parts;       // backward: partial sums [token tiles][(width + 1) * channels], or null
    int64_t ctiles, ttiles;  // channel tiles; token tiles per row
};

// Tokens of one block of the backward pass.
constexpr int kConvBwdTokens = 512;

cudaError_t conv_forward_f32(ConvArgs a, cudaStream_t s);
cudaError_t conv_forward_bf16(ConvArgs a, cudaStream_t s);
cudaError_t conv_forward_f16(ConvArgs a, cudaStream_t s);
cudaError_t conv_backward_f32(ConvArgs a, cudaStream_t s);
cudaError_t conv_backward_bf16(ConvArgs a, cudaStream_t s);
cudaError_t conv_backward_f16(ConvArgs a, cudaStream_t s);

}  // namespace gbfft
