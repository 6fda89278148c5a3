// Single tokens of the sequence operators (fft_conv_step, fft_scan_step): every sequence reads
// its state from a slot of a pool, takes one token and writes the new state to a slot.  Both are
// bound by the state's bytes for many sequences and by latency for one.
#include "seq_step.h"

namespace gbfft {
namespace {

constexpr int kThreads = 128;

// The slots of a sequence; false where one lies outside the pool (a padding row).
__device__ __forceinline__ bool step_slots(const int64_t* slots, const int64_t* slots_out,
                                           int64_t pool, int64_t q, int64_t* in, int64_t* out) {
    *in = slots ? slots[q] : q;
    *out = slots_out ? slots_out[q] : *in;
    return *in >= 0 && *in < pool && *out >= 0 && *out < pool;
}

// A thread holds VEC channels of one sequence; the taps come straight from the state's rows.
template <class T, int VEC>
__global__ void __launch_bounds__(kThreads) k_conv_step(const ConvStepArgs a) {
    const int64_t vecs = a.d.channels / VEC;
    const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (i >= vecs * a.d.nseq) return;
    const int64_t q = i / vecs, c = (i - q * vecs) * VEC;
    const int w = a.d.width, f32 = a.d.param_dtype == FFT_F32;
    int64_t in, to;
    const bool live = step_slots(a.slots, a.slots_out, a.pool, q, &in, &to);
    T* out = static_cast<T*>(a.out.data) + q * a.out.seq_stride + c;
    Pack<T, VEC> y;
    if (!live) {
#pragma unroll
        for (int k = 0; k < VEC; ++k) y.v[k] = from_f<T>(0.f);
        st_pack<VEC>(out, y);
        return;
    }
    const int64_t per = (w - 1) * a.d.channels;
    const T* src = static_cast<const T*>(a.state) + in * per + c;
    T* dst = static_cast<T*>(a.state) + to * per + c;
    const Pack<T, VEC> x =
        ld_pack<VEC>(static_cast<const T*>(a.d.x.data) + q * a.d.x.seq_stride + c);
    Pack<T, VEC> s[FFT_CONV_MAX_WIDTH - 1];
#pragma unroll
    for (int r = 0; r < FFT_CONV_MAX_WIDTH - 1; ++r)
        if (r < w - 1) s[r] = ld_pack<VEC>(src + r * a.d.channels);
    float p[VEC];
#pragma unroll
    for (int k = 0; k < VEC; ++k) {
        p[k] = a.d.bias ? ld_param<T>(a.d.bias, c + k, f32) : 0.f;
#pragma unroll
        for (int r = 0; r < FFT_CONV_MAX_WIDTH - 1; ++r)
            if (r < w - 1) p[k] += ld_param<T>(a.d.weight, (c + k) * w + r, f32) * to_f(s[r].v[k]);
        p[k] += ld_param<T>(a.d.weight, (c + k) * w + w - 1, f32) * to_f(x.v[k]);
        if (a.d.silu) p[k] *= sigmoid(p[k]);
        y.v[k] = from_f<T>(p[k]);
    }
    st_pack<VEC>(out, y);
#pragma unroll
    for (int r = 1; r < FFT_CONV_MAX_WIDTH - 1; ++r)
        if (r < w - 1) st_pack<VEC>(dst + (r - 1) * a.d.channels, s[r]);
    if (w > 1) st_pack<VEC>(dst + (w - 2) * a.d.channels, x);
}

// L lanes share a channel, four states each: a warp moves 32 * 16 contiguous bytes of states.
template <class T, int L>
__global__ void __launch_bounds__(kThreads) k_scan_step(const ScanStepArgs a) {
    constexpr int CT = kThreads / L;
    const int64_t q = blockIdx.x / a.ctiles;
    const int64_t c = (blockIdx.x - q * a.ctiles) * CT + threadIdx.x / L;
    const int n = (int)a.d.states, s0 = (int)(threadIdx.x % L) * 4;
    const bool in = c < a.d.channels;
    int64_t from, to;
    const bool live = step_slots(a.slots, a.slots_out, a.pool, q, &from, &to);
    float y = 0.f, uu = 0.f, gate = 1.f;
    if (in && live) {
        const int64_t g = c / (a.d.channels / a.d.groups);
        const T* B = static_cast<const T*>(a.d.B.data) + q * a.d.B.seq_stride + g * n;
        const T* C = static_cast<const T*>(a.d.C.data) + q * a.d.C.seq_stride + g * n;
        const float* src = a.state + (from * a.d.channels + c) * n;
        float* dst = a.state + (to * a.d.channels + c) * n;
        float h[4], A[4], b[4], cc[4];
        if (a.vec) {
            if (s0 < n) {
                const float4 hv = *reinterpret_cast<const float4*>(src + s0);
                const float4 av = *reinterpret_cast<const float4*>(a.d.A + c * n + s0);
                h[0] = hv.x; h[1] = hv.y; h[2] = hv.z; h[3] = hv.w;
                A[0] = av.x; A[1] = av.y; A[2] = av.z; A[3] = av.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (s0 + i < n) {
                    h[i] = src[s0 + i];
                    A[i] = a.d.A[c * n + s0 + i];
                }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (s0 + i < n) {
                b[i] = to_f(B[s0 + i]);
                cc[i] = to_f(C[s0 + i]);
            }
        uu = to_f(static_cast<const T*>(a.d.u.data)[q * a.d.u.seq_stride + c]);
        float d = to_f(static_cast<const T*>(a.d.delta.data)[q * a.d.delta.seq_stride + c]);
        if (a.d.z.data) {
            const float z = to_f(static_cast<const T*>(a.d.z.data)[q * a.d.z.seq_stride + c]);
            gate = z * sigmoid(z);
        }
        if (a.d.delta_bias) d += a.d.delta_bias[c];
        if (a.d.softplus) d = softplus(d);
        const float du = d * uu;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (s0 + i < n) {
                h[i] = fmaf(ex2(d * (A[i] * kLog2e)), h[i], du * b[i]);
                y = fmaf(cc[i], h[i], y);
            }
        if (a.vec) {
            if (s0 < n) *reinterpret_cast<float4*>(dst + s0) = make_float4(h[0], h[1], h[2], h[3]);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (s0 + i < n) dst[s0 + i] = h[i];
        }
    }
#pragma unroll
    for (int o = L / 2; o; o >>= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
    if (in && threadIdx.x % L == 0) {
        if (live && a.d.D) y = fmaf(a.d.D[c], uu, y);
        if (live && a.d.z.data) y *= gate;
        static_cast<T*>(a.out.data)[q * a.out.seq_stride + c] = from_f<T>(y);
    }
}

template <class T>
cudaError_t conv_step(const ConvStepArgs& a, cudaStream_t s) {
    constexpr int V = 16 / sizeof(T);
    auto rows_ok = [&](const fft_seq& q) {
        return aligned_to(q.data, 16) && (a.d.nseq == 1 || q.seq_stride % V == 0);
    };
    const bool vec = a.d.channels % V == 0 && rows_ok(a.d.x) && rows_ok(a.out) &&
                     aligned_to(a.state, 16);
    const int64_t blocks = (a.d.channels / (vec ? V : 1) * a.d.nseq + kThreads - 1) / kThreads;
    if (blocks > INT32_MAX) return cudaErrorInvalidValue;
    if (vec)
        k_conv_step<T, V><<<(unsigned)blocks, kThreads, 0, s>>>(a);
    else
        k_conv_step<T, 1><<<(unsigned)blocks, kThreads, 0, s>>>(a);
    return cudaGetLastError();
}

template <class T, int L>
cudaError_t scan_step_lanes(ScanStepArgs a, cudaStream_t s) {
    a.ctiles = (a.d.channels + kThreads / L - 1) / (kThreads / L);
    if (a.ctiles * a.d.nseq > INT32_MAX) return cudaErrorInvalidValue;
    k_scan_step<T, L><<<(unsigned)(a.ctiles * a.d.nseq), kThreads, 0, s>>>(a);
    return cudaGetLastError();
}
template <class T>
cudaError_t scan_step(ScanStepArgs a, cudaStream_t s) {
    a.vec = a.d.states % 4 == 0 && aligned_to(a.state, 16) && aligned_to(a.d.A, 16);
    if (a.d.states <= 4) return scan_step_lanes<T, 1>(a, s);
    if (a.d.states <= 8) return scan_step_lanes<T, 2>(a, s);
    if (a.d.states <= 16) return scan_step_lanes<T, 4>(a, s);
    if (a.d.states <= 32) return scan_step_lanes<T, 8>(a, s);
    if (a.d.states <= 64) return scan_step_lanes<T, 16>(a, s);
    return scan_step_lanes<T, 32>(a, s);
}

}  // namespace

cudaError_t conv_step_any(const ConvStepArgs& a, cudaStream_t s) {
    if (a.d.dtype == FFT_F32) return conv_step<float>(a, s);
    return a.d.dtype == FFT_BF16 ? conv_step<__nv_bfloat16>(a, s) : conv_step<__half>(a, s);
}
cudaError_t scan_step_any(const ScanStepArgs& a, cudaStream_t s) {
    if (a.d.dtype == FFT_F32) return scan_step<float>(a, s);
    return a.d.dtype == FFT_BF16 ? scan_step<__nv_bfloat16>(a, s) : scan_step<__half>(a, s);
}

}  // namespace gbfft
