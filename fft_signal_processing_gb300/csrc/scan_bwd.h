// Selective state-space scan, backward: arguments, workspace layout and per-type launchers
// (scan_bwd.cuh).
#pragma once

#include "scan.h"

namespace gbfft {

// Tokens whose dA, dD and ddelta_bias one float32 accumulator adds up.  A sum of T terms one after
// another is off by some sqrt(T) / 4 units of 2^-24, and chunks may be as long as the row.
constexpr int kScanPart = 256;

struct ScanBwdArgs {
    fft_scan_desc d;
    fft_scan_grads g;
    ScanArgs f;        // the forward passes (carry, dsum, reset, tiles)
    float* carry;      // gradient that enters every chunk from behind [rows][chunks][channels][np]
    float* bc;         // partial dB, dC [channel tiles][rows][length][groups][2][states]
    float* pA;         // partial dA [rows * parts][channels * states]
    float* pD;         // partial dD [rows * parts][channels]
    float* pbias;      // partial ddelta_bias [rows * parts][channels]
    int64_t cuts, parts;  // partial rows of a chunk, kScanPart tokens each, and of a row
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
