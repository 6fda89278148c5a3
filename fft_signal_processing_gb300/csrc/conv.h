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
    int run;                 // tokens of a run
};

// A block has 32 lanes along the channels and 8 runs of tokens; the runs of a block are its token
// tile (one partial row of the parameter gradients).
constexpr int kConvLanes = 32, kConvRuns = 8;
constexpr int kConvMaxRun = 64;

// Tokens of a run: of 64 and less, the number whose rounds of resident blocks (three to an SM
// forward, two backward) take the fewest tokens' time, with the halo and about 8 tokens to start.
// 16001 tokens of 2000 channels, backward: 56.  Three and two are what width 4 in 16 bits has; by
// their registers other widths hold two to five and one to three, float32 three to six and two to
// four, and the rule is used for them as it is.
inline int conv_run_tokens(const fft_conv_desc& d, bool backward) {
    const int64_t lanes = d.dtype == FFT_F32 ? 2 : 4;  // channels of a lane
    const int64_t ctiles = (d.channels + kConvLanes * lanes - 1) / (kConvLanes * lanes);
    const int64_t rows = d.offsets ? 1 : d.nseq, resident = (int64_t)num_sms() * (backward ? 2 : 3);
    int64_t best = INT64_MAX;
    int run = kConvMaxRun;
    // forward, many rounds of full runs: shorter ones only read more halo
    if (!backward && ctiles * rows * (d.length / (kConvRuns * run)) >= 2 * resident) return run;
    for (int r = kConvMaxRun; r >= 16; r -= 4) {
        const int64_t blocks = ctiles * rows * ((d.length + kConvRuns * r - 1) / (kConvRuns * r));
        const int64_t cost = (blocks + resident - 1) / resident * (r + 2 * (d.width - 1) + 8);
        if (cost < best) {
            best = cost;
            run = r;
        }
    }
    return run;
}

cudaError_t conv_forward_f32(ConvArgs a, cudaStream_t s);
cudaError_t conv_forward_bf16(ConvArgs a, cudaStream_t s);
cudaError_t conv_forward_f16(ConvArgs a, cudaStream_t s);
cudaError_t conv_backward_f32(ConvArgs a, cudaStream_t s);
cudaError_t conv_backward_bf16(ConvArgs a, cudaStream_t s);
cudaError_t conv_backward_f16(ConvArgs a, cudaStream_t s);

}  // namespace gbfft
