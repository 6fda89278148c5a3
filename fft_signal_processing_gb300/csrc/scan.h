// Selective state-space scan: arguments of the kernels, the plan of a call and the per-type
// launchers (scan.cuh, scan_bwd.cuh).
#pragma once

#include "seq_common.cuh"

namespace gbfft {

// States per thread and lanes per channel of the forward kernels: n <= spt * sl.
struct ScanShape {
    int spt, sl;
    int np() const { return spt * sl; }
};
inline ScanShape scan_shape(int64_t n) {
    if (n <= 4) return {4, 1};
    if (n <= 8) return {8, 1};
    if (n <= 16) return {16, 1};
    if (n <= 32) return {16, 2};
    if (n <= 64) return {16, 4};
    return {16, 8};
}
constexpr int kScanThreads = 128;
constexpr int kScanTile = 8;  // tokens of one tile

struct ScanArgs {
    fft_scan_desc d;
    fft_seq out;
    float* final_state;  // or null
    // chunked: the state before every chunk [rows][chunks][channels][np], the sum of d over it
    // [rows][chunks][channels], and whether a sequence starts in it [rows][chunks]
    float* carry;
    float* dsum;
    int* reset;
    float* tiles;  // the state before every kScanStateTile-th token [rows][tiles][channels][np]
    int64_t rows, chunk, nchunks, ctiles;  // tokens per chunk; channel tiles per group
};

// Passes of the forward kernel: the effect of a chunk on the state; outputs and final states;
// the states that the backward pass restarts from.
enum { SCAN_SUMMARY = 0, SCAN_OUTPUT = 1, SCAN_TILES = 2 };
constexpr int kScanStateTile = 16;

struct ScanChunks {
    int64_t rows, chunk, nchunks, ctiles;
};
inline ScanChunks scan_chunks(const fft_scan_desc& d) {
    const ScanShape sh = scan_shape(d.states);
    const int64_t ct = kScanThreads / sh.sl, dg = d.channels / d.groups;
    ScanChunks p;
    p.rows = d.offsets ? 1 : d.nseq;
    p.ctiles = (dg + ct - 1) / ct;
    const int64_t blocks = p.rows * p.ctiles * d.groups;
    const int64_t want = (int64_t)num_sms() * 6;  // resident blocks
    p.chunk = d.length;
    if (blocks * 2 < want) {
        const int64_t n = (want + blocks - 1) / blocks;
        p.chunk = (d.length + n - 1) / n;
        p.chunk = (p.chunk + 63) / 64 * 64;
    }
    if (p.chunk < 64) p.chunk = 64;
    p.nchunks = (d.length + p.chunk - 1) / p.chunk;
    return p;
}

cudaError_t scan_forward_f32(const ScanArgs& a, cudaStream_t s);
cudaError_t scan_forward_bf16(const ScanArgs& a, cudaStream_t s);
cudaError_t scan_forward_f16(const ScanArgs& a, cudaStream_t s);

}  // namespace gbfft
