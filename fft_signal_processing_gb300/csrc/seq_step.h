// Single-token forms of the sequence operators: arguments and launchers (seq_step.cu).
#pragma once

#include "seq_common.cuh"

namespace gbfft {

struct ConvStepArgs {
    fft_conv_desc d;
    fft_seq out;
    void* state;
    const int64_t* slots;      // or null: sequence q has slot q
    const int64_t* slots_out;  // or null: in place
    int64_t pool;
};
struct ScanStepArgs {
    fft_scan_desc d;
    fft_seq out;
    float* state;
    const int64_t* slots;
    const int64_t* slots_out;
    int64_t pool, ctiles;
    bool vec;  // 16-byte accesses to states
};
cudaError_t conv_step_any(const ConvStepArgs& a, cudaStream_t s);
cudaError_t scan_step_any(const ScanStepArgs& a, cudaStream_t s);

}  // namespace gbfft
