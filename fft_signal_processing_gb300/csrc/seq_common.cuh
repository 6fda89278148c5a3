// Shared by the sequence operators (short causal convolution, selective scan, residual norm):
// type conversions, rows addressed by strides, sequences found from packed offsets, and the
// column sums that close every parameter gradient.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/gbfft.h"

namespace gbfft {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f(__half v) { return __half2float(v); }
template <class T> __device__ __forceinline__ T from_f(float v);
template <> __device__ __forceinline__ float from_f<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) {
    return __float2bfloat16_rn(v);
}
template <> __device__ __forceinline__ __half from_f<__half>(float v) { return __float2half_rn(v); }

// A run of V contiguous values of T, moved in accesses of up to 16 bytes.
template <class T, int V>
struct alignas(sizeof(T) * V > 16 ? 16 : sizeof(T) * V) Pack {
    T v[V];
};
template <int V, class T>
__device__ __forceinline__ Pack<T, V> ld_pack(const T* p) {
    return *reinterpret_cast<const Pack<T, V>*>(p);
}
template <int V, class T>
__device__ __forceinline__ void st_pack(T* p, const Pack<T, V>& x) {
    *reinterpret_cast<Pack<T, V>*>(p) = x;
}

// Two values rounded at once.
template <class T> __device__ __forceinline__ Pack<T, 2> from_f2(float2 v);
template <> __device__ __forceinline__ Pack<float, 2> from_f2<float>(float2 v) {
    return {v.x, v.y};
}
template <> __device__ __forceinline__ Pack<__nv_bfloat16, 2> from_f2<__nv_bfloat16>(float2 v) {
    const __nv_bfloat162 r = __floats2bfloat162_rn(v.x, v.y);
    return {r.x, r.y};
}
template <> __device__ __forceinline__ Pack<__half, 2> from_f2<__half>(float2 v) {
    const __half2 r = __floats2half2_rn(v.x, v.y);
    return {r.x, r.y};
}

// A parameter of type float or T (f32 != 0: float).
template <class T>
__device__ __forceinline__ float ld_param(const void* p, int64_t i, int f32) {
    return f32 ? static_cast<const float*>(p)[i] : to_f(static_cast<const T*>(p)[i]);
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// 1 / (1 + exp(-x)): exp(-x) overflows to infinity for x < -88 and the quotient is 0.
__device__ __forceinline__ float sigmoid(float x) { return rcp(1.0f + ex2(-kLog2e * x)); }

// Two float32 values in one 64-bit register pair: sm_103a multiplies and adds both at once.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 d;
    asm("mul.rn.f32x2 %0, %1, %2;"
        : "=l"(reinterpret_cast<unsigned long long&>(d))
        : "l"(reinterpret_cast<unsigned long long&>(a)),
          "l"(reinterpret_cast<unsigned long long&>(b)));
    return d;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(reinterpret_cast<unsigned long long&>(d))
        : "l"(reinterpret_cast<unsigned long long&>(a)),
          "l"(reinterpret_cast<unsigned long long&>(b)),
          "l"(reinterpret_cast<unsigned long long&>(c)));
    return d;
}

__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("add.rn.f32x2 %0, %1, %2;"
        : "=l"(reinterpret_cast<unsigned long long&>(d))
        : "l"(reinterpret_cast<unsigned long long&>(a)),
          "l"(reinterpret_cast<unsigned long long&>(b)));
    return d;
}
__device__ __forceinline__ float2 splat(float v) { return make_float2(v, v); }
// exp(d A) of two states, A2 = A log2(e).  ex2.approx lies low: for d A between -1e-6 and -4 its
// results are on average 0.1 to 0.5 units of 2^-24 below the exponential, and a state that is kept
// for a thousand tokens collects that a thousand times.  The shift of the argument costs no
// instruction and takes the average to within 0.28 units (0.2 above -0.5).  Gradients of A, 4 x 2048
// tokens of 2048 bfloat16 channels: off by 1.7e-6 without it, 0.8e-6 with it; at 2.5e-8 sequences of
// 6000 tokens, whose slow states are kept longest, come out worse again (0.74e-6 against 0.96e-6).
constexpr float kEx2Shift = 2e-8f;
__device__ __forceinline__ float2 decay2(float2 d, float2 A2) {
    const float2 e = fma2(d, A2, splat(kEx2Shift));
    return make_float2(ex2(e.x), ex2(e.y));
}
__device__ __forceinline__ float max_nan(float a, float b) {  // a NaN stays
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}

__device__ __forceinline__ float2 sigmoid2(float2 x) {
    const float2 e = mul2(x, splat(-kLog2e));
    const float2 d = add2(make_float2(ex2(e.x), ex2(e.y)), splat(1.f));
    return make_float2(rcp(d.x), rcp(d.y));
}

// log(1 + exp(x)) = max(x, 0) + log1p(t), t = exp(-|x|) in (0, 1], and log1p(t) = 2 atanh(w) with
// w = t / (2 + t) <= 1/3: w times a polynomial in w^2, interpolated at Chebyshev nodes of
// [0, 1/9] (relative error 8e-9).  The exponent's rounding error is put back, since t is the
// result itself where x << 0; below -87, where t leaves the normal range, the result stays there.
__device__ __forceinline__ float2 softplus2(float2 x) {
    const float2 y = make_float2(max_nan(-fabsf(x.x), -87.f), max_nan(-fabsf(x.y), -87.f));
    const float2 hi = mul2(y, splat(kLog2e));
    float2 lo = fma2(y, splat(kLog2e), make_float2(-hi.x, -hi.y));
    lo = fma2(y, splat(1.9259630e-8f), lo);  // log2(e) beyond 24 bits
    float2 t = make_float2(ex2(hi.x), ex2(hi.y));
    t = fma2(mul2(lo, splat(kLn2)), t, t);
    const float2 den = add2(t, splat(2.f));
    const float2 w = mul2(t, make_float2(rcp(den.x), rcp(den.y))), q = mul2(w, w);
    float2 p = fma2(q, splat(0.28157779574394226f), splat(0.27965158224105835f));
    p = fma2(q, p, splat(0.4002459645271301f));
    p = fma2(q, p, splat(0.6666632294654846f));
    p = fma2(q, p, splat(2.f));
    return fma2(w, p, make_float2(max_nan(x.x, 0.f), max_nan(x.y, 0.f)));
}
__device__ __forceinline__ float softplus(float x) { return softplus2(splat(x)).x; }

// Sum of V values over lanes that differ in the bits of `mask` steps (from W down to 1, times
// STEP): while a lane carries more than one value it keeps half of them.
template <int V, int W, int STEP>
__device__ __forceinline__ void hand_out(float (&v)[V], int id) {
    int cnt = V;
#pragma unroll
    for (int w = W; w; w /= 2) {
        if (cnt > 1) {
            cnt /= 2;
            const bool up = id & w;
#pragma unroll
            for (int j = 0; j < V / 2; ++j) {
                if (j < cnt) {
                    const float send = up ? v[j] : v[j + cnt], keep = up ? v[j + cnt] : v[j];
                    v[j] = keep + __shfl_xor_sync(0xffffffffu, send, w * STEP);
                }
            }
        } else {
            v[0] += __shfl_xor_sync(0xffffffffu, v[0], w * STEP);
        }
    }
}

// Asynchronous copies of 16, 8 and 4 bytes into shared memory; zeros where `in` is false (nothing is
// read).
__device__ __forceinline__ void copy16(void* dst, const void* src, bool in) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                     (unsigned)__cvta_generic_to_shared(dst)),
                 "l"(src), "r"(in ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void copy8(void* dst, const void* src, bool in) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(
                     (unsigned)__cvta_generic_to_shared(dst)),
                 "l"(src), "r"(in ? 8 : 0)
                 : "memory");
}
__device__ __forceinline__ void copy4(void* dst, const void* src, bool in) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(
                     (unsigned)__cvta_generic_to_shared(dst)),
                 "l"(src), "r"(in ? 4 : 0)
                 : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {  // all but the last N groups have landed
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Number of ascending offsets[0 .. n-1] that are <= t, found by a whole warp: 32 probes a step
// instead of one, since each step costs a trip to L2.
__device__ __forceinline__ int64_t warp_count_le(const int64_t* offsets, int64_t n, int64_t t) {
    const int lane = (int)(threadIdx.y * blockDim.x + threadIdx.x) & 31;
    int64_t lo = 0, hi = n;  // the count lies in [lo, hi]
    while (hi > lo) {
        const int64_t step = (hi - lo + 31) / 32;
        const int64_t i = lo + (int64_t)(lane + 1) * step - 1;
        const unsigned le = __ballot_sync(0xffffffffu, i < hi && __ldg(offsets + i) <= t);
        const int k = __popc(le);  // the first k probes are <= t
        const int64_t nlo = lo + (int64_t)k * step;
        const int64_t nhi = lo + (int64_t)(k + 1) * step - 1;
        hi = nhi < hi ? nhi : hi;
        lo = nlo < hi ? nlo : hi;
    }
    return lo;
}

// The sequence that token t of a row belongs to: [begin, end) are its tokens.  Offsets lie on the
// device and no host check sees them: q is a sequence that there is, begin and end may be anything.
struct SeqAt {
    int64_t q, begin, end;
};
__host__ __device__ __forceinline__ SeqAt seq_span(const int64_t* offsets, int64_t nseq, int64_t q) {
    q = q < 0 ? 0 : (q >= nseq ? nseq - 1 : q);
    const int64_t begin = offsets[q];
    return {q, begin < 0 ? 0 : begin, offsets[q + 1]};
}
// Dense rows: sequence q is the row itself.  Packed: found by the whole warp.
__device__ __forceinline__ SeqAt seq_at(const int64_t* offsets, int64_t nseq, int64_t length,
                                        int64_t row, int64_t t) {
    if (!offsets) return {row, 0, length};
    return seq_span(offsets, nseq, warp_count_le(offsets, nseq + 1, t) - 1);
}
// The sequence that begins where s ends (token t = s.end), empty ones skipped.
__host__ __device__ __forceinline__ void seq_next(const int64_t* offsets, int64_t nseq, int64_t t,
                                                  SeqAt* s) {
    while (s->q + 1 < nseq && s->end <= t) {
        s->q += 1;
        s->begin = s->end < 0 ? 0 : s->end;
        s->end = offsets[s->q + 1];
    }
}
// The end of s counted from token t0 of a run of len tokens: len + 1 where s goes on behind the run.
// A tile [t, t + n) with t + n < seq_stop lies within the run, whatever the offsets say, and s does
// not end in it.
__host__ __device__ __forceinline__ int seq_stop(const SeqAt& s, int64_t t0, int len) {
    const int64_t end = s.end - t0;
    return end > len ? len + 1 : (end < 0 ? 0 : (int)end);
}

// Whether the state of a scan starts anew at token t of its row: at a sequence's first token and,
// where offsets leave the first tokens to no sequence, at the row's.  (A chunk's own start state
// exists only where time is cut.)
__host__ __device__ __forceinline__ bool starts_at(const SeqAt& s, int64_t t) {
    return t == 0 || s.begin == t;
}

// Sums over parts, the last step of a parameter gradient, in an order that does not depend on the
// launch: column k * chan + c of parts[p * stride + column] (cols of them) goes to
// out[c * (cols / chan) + k].  No parts: zeros.
cudaError_t run_sum_parts(const float* parts, int64_t nparts, int64_t stride, int64_t cols,
                          float* out, int64_t chan, int64_t wide, cudaStream_t s);

inline bool aligned_to(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }
inline size_t dtype_size(int t) { return t == FFT_F32 ? 4 : (t == FFT_E4M3 ? 1 : 2); }
inline int num_sms() {
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1)
        return 152;
    return n;
}

}  // namespace gbfft
