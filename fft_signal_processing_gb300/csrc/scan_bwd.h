// Selective state-space scan, backward: arguments, workspace layout and per-type launchers
// (scan_bwd.cuh).
#pragma once

#include "scan.h"

namespace gbfft {

struct ScanBwdArgs {
    fft_scan_desc d;
    fft_scan_grads g;
    ScanArgs f;        // the forward passes (carry, dsum, reset, tiles)
    float* carry;      // gradient that enters every chunk from behind [rows][chunks][channels][np]
    float* bc;         // partial dB, dC [channel tiles][rows][length][groups][2][states]
    float* pA;         // partial dA [rows * chunks][channels * states]
    float* pD;         // partial dD [rows * chunks][channels]
    float* pbias;      // partial ddelta_bias [rows * chunks][channels]
    int64_t ctiles;    // channel tiles per group of the main kernel
    int64_t back_ctiles;  // and of the pass that finds what the chunks send back
};

// Lanes that share a channel and warps per block of the main kernel: a thread holds 4 channels x
// 4 states.
inline int bwd_sl(int64_t n) {
    int sl = 1;
    while (sl * 4 < n) sl *= 2;
    return sl;
}
inline int bwd_warps(int sl) { return sl < 4 ? sl : 4; }
inline int bwd_channels(int sl) { return bwd_warps(sl) * 128 / sl; }

// Fills `a` (unless null) from a workspace at w and returns the bytes it takes.
int64_t scan_bwd_layout(const fft_scan_desc& d, ScanBwdArgs* a, char* w);

cudaError_t scan_backward_f32(const ScanBwdArgs& a, cudaStream_t s);
cudaError_t scan_backward_bf16(const ScanBwdArgs& a, cudaStream_t s);
cudaError_t scan_backward_f16(const ScanBwdArgs& a, cudaStream_t s);

}  // namespace gbfft
