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

// A block has 32 lanes along the channels and 8 runs of tokens; the runs of a block are its token
// tile (one partial row of the parameter gradients).
constexpr int kConvLanes = 32, kConvRuns = 8, kConvRun = 64;
constexpr int kConvTile = kConvRuns * kConvRun;

cudaError_t conv_forward_f32(ConvArgs a, cudaStream_t s);
cudaError_t conv_forward_bf16(ConvArgs a, cudaStream_t s);
cudaError_t conv_forward_f16(ConvArgs a, cudaStream_t s);
cudaError_t conv_backward_f32(ConvArgs a, cudaStream_t s);
cudaError_t conv_backward_bf16(ConvArgs a, cudaStream_t s);
cudaError_t conv_backward_f16(ConvArgs a, cudaStream_t s);

}  // namespace gbfft
