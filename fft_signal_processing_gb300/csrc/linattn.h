// Linear attention with a decay for each head and token: arguments of the kernels, the plan of a
// call and the launchers (linattn.cuh, one file per type and direction).
//
// One kernel serves the forward pass and the three passes of the gradients.  It is given "queries"
// x, "keys" y (rows of dx values) and "values" z (rows of dz values) and computes, over the tokens
// of a sequence in either direction,
//   out[r] = sum_{c before r} decay(c, r) p (x[r] y[c]) z[c] + decay(start, r) i x[r] S
// and the state S (dx by dz) behind the last token.
#pragma once

#include "seq_common.cuh"

namespace gbfft {

constexpr int kAttnChunk = 64;     // tokens that one step of the kernel takes
constexpr int kTcChunk = 128;      // and of the tcgen05 kernel; the decay's gradient takes sums by them
constexpr int kAttnMaxDim = 256;   // dk and dv

// Rows of one head at data + (q * seq + t * tok + (h / share) * head) elements.
struct AttnRows {
    const void* data;
    int64_t seq, tok, head;
    int share;  // heads that read the same rows
    int vec;    // bytes that all rows start on: 16, 4 or 0
};

struct AttnArgs {
    AttnRows x, y, z;
    AttnRows partner;  // rows of dz values whose products with the outputs are wanted, or none
    void* out;
    int64_t out_seq, out_tok, out_head;
    int out_f32;   // outputs in float32 whatever the type (partial sums over heads)
    int out_pair;  // two neighbouring outputs are one store
    fft_seq decay;
    const int64_t* offsets;
    int64_t nseq, length, rows;  // rows: 1 if packed, else nseq
    int64_t heads, dx, dz;
    float scale_pair, scale_inter, scale_update;
    int reverse, summary;
    // states [sequence][head][dk][dv]: element (x, z) at x * state_x + z * state_z
    const float* initial;
    float* final_state;
    const float* final_dot;  // states whose products with the final ones are wanted
    float* final_dots;       // [ztile][sequence][head]
    int64_t state_x, state_z;
    // cut time: `segment` tokens each; the state that a segment begins with, as the threads hold
    // it, its decay (log2) and whether that state's sequence begins within the segment before
    int64_t segment, nsegments, ztiles;
    float* carry;
    float* carry_decay;  // [row][segment][head]
    int* carry_reset;    // [row][segment][head]
    float* dots_inter;   // [ztile][head][row * length + t]
    float* dots_all;
    uint32_t wait_ns;  // limit of a device-side wait; 0: none is begun
};

// A number in two floats, 48 bits.
struct Two {
    float hi, lo;
};
__device__ __forceinline__ Two add(Two a, Two b) {
    const float s = a.hi + b.hi, t = s - a.hi;
    const float e = (a.hi - (s - t)) + (b.hi - t) + (a.lo + b.lo);
    const float hi = s + e;
    return {hi, e - (hi - s)};
}
// A log decay in units of log2: at most 0 (a NaN stays), and at least -288, where every float32
// number has become 0.
__device__ __forceinline__ Two log2_decay(float g) {
    const float c = g > 0.f ? 0.f : (g < -200.f ? -200.f : g), hi = c * kLog2e;
    return {hi, fmaf(c, 1.9259630e-8f, fmaf(c, kLog2e, -hi))};  // log2(e) beyond 24 bits
}

// Padded sizes of the kernel's variants.
inline int attn_pad(int64_t d) { return d <= 64 ? 64 : (d <= 128 ? 128 : 256); }
inline int attn_warps(int dtype, int64_t dx, int64_t dz) {
    return dz <= 64 || (dtype == FFT_F32 && dx > 128) ? 4 : 8;
}
inline int64_t attn_ztile(int dtype, int64_t dx, int64_t dz) { return 16 * attn_warps(dtype, dx, dz); }
// Values of a carried state: what the threads of a block hold, zeros beyond dx and dz among them
// (the tcgen05 kernel's always have 128 columns of z).
inline int64_t attn_carry(int dtype, int64_t dx, int64_t dz) {
    return attn_pad(dx) * (dtype == FFT_BF16 && dx <= 128 ? 128 : attn_ztile(dtype, dx, dz));
}

cudaError_t attn_f32_fwd(const AttnArgs& a, cudaStream_t s);
cudaError_t attn_f32_bwd(const AttnArgs& a, cudaStream_t s);
cudaError_t attn_bf16_fwd(const AttnArgs& a, cudaStream_t s);
cudaError_t attn_bf16_bwd(const AttnArgs& a, cudaStream_t s);
cudaError_t attn_f16_fwd(const AttnArgs& a, cudaStream_t s);
cudaError_t attn_f16_bwd(const AttnArgs& a, cudaStream_t s);

// The same on tcgen05: rows on 16-byte boundaries, dx at most 128; err: the device's error word.
cudaError_t attn_tc_fwd(const AttnArgs& a, int* err, cudaStream_t s);
cudaError_t attn_tc_bwd(const AttnArgs& a, int* err, cudaStream_t s);

// Turns what every segment adds into the state that it begins with; quads: float4 of a head's.
cudaError_t attn_carry_pass(const AttnArgs& a, int64_t quads, cudaStream_t s);

}  // namespace gbfft
