// Selective state-space scan: arguments of the kernels, the plan of a call and the per-type
// launchers (scan.cuh, scan_bwd.cuh).
#pragma once

#include "seq_common.cuh"

namespace gbfft {

// States of a channel, padded: what the rows of a workspace hold.
inline int scan_np(int64_t n) {
    int np = 4;
    while (np < n) np *= 2;
    return np;
}
// The same in the forward call, whose kernel also comes for twelve states.
inline int scan_out_np(int64_t n) { return n > 8 && n <= 12 ? 12 : scan_np(n); }
constexpr int kScanThreads = 128;
constexpr int kScanTile = 16;  // the backward pass restarts at these tiles
// Channels of a block of 64 threads: two per thread (sl 0), or sl lanes per channel.
inline int scan_channels(int sl) { return sl ? 64 / sl : 128; }
// Lanes per channel of the kernels that cut time: 16 states per thread.
inline int scan_lanes(int np) { return np <= 16 ? 0 : np / 16; }

struct ScanArgs {
    fft_scan_desc d;
    fft_seq out;
    float* final_state;  // or null
    // chunked: the state before every chunk [rows][chunks][channels][np], the sum of d over it
    // [rows][chunks][channels], and whether a sequence starts in it [rows][chunks]
    float* carry;
    float* dsum;
    int* reset;
    float* tiles;  // the state before every tile [rows][tiles][channels][np]
    int64_t rows, chunk, nchunks, ctiles;  // tokens per chunk; channel tiles per group
    int sl;    // 0: k_scan, else the lanes per channel of k_scan_lanes
    int vec;   // bytes that rows of u, delta and z start on: 16, 4 or 0
    int wide;  // the states of B and C are whole 16-byte accesses
    int pair;  // two channels of out are one access
};

// Passes of the forward kernel: the effect of a chunk on the state; outputs and final states;
// the states that the backward pass restarts from.
enum { SCAN_SUMMARY = 0, SCAN_OUTPUT = 1, SCAN_TILES = 2 };

// Kernel and chunks of a forward call: fills sl, rows, chunk, nchunks and ctiles.
void scan_plan(ScanArgs* a);

cudaError_t scan_forward_f32(const ScanArgs& a, cudaStream_t s);
cudaError_t scan_forward_bf16(const ScanArgs& a, cudaStream_t s);
cudaError_t scan_forward_f16(const ScanArgs& a, cudaStream_t s);

}  // namespace gbfft
