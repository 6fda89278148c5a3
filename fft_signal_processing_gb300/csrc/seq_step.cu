// Single tokens of the sequence operators (fft_conv_step, fft_scan_step): every sequence reads
// its state from a slot of a pool, takes one token and writes the new state to a slot.  Both are
// bound by the state's bytes for many sequences and by latency for one.  Measured: scan of 256
// sequences of 4096 channels and 16 states 39 us, 3.7 TB/s (54% of the copy rate: two dependent
// trips, slot then state); one sequence of 2048 channels 4.8 us on the GPU, 17 us with the host
// side of the call; convolution of one sequence of 4096 channels 5.4 and 18 us.
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

// L lanes share a channel, four states each, and a thread has four channels, 32 / L apart, so that
// a warp's accesses to the states are 512 contiguous bytes each.  What is needed once per channel
// (softplus, the gate, the output) is done by the lane that owns it: the step is then bound by
// the states' bytes and not by instructions.
template <class T, int L>
__global__ void __launch_bounds__(kThreads) k_scan_step(const ScanStepArgs a) {
    constexpr int G = 32 / L, OWN = L >= 4 ? 1 : 4 / L;  // groups of lanes; channels a lane owns
    const int64_t q = blockIdx.x / a.ctiles;
    const int lane = (int)threadIdx.x & 31, sl = lane % L, s0 = sl * 4;
    // channel k of the thread: cw + k * G
    const int64_t cw = ((blockIdx.x - q * a.ctiles) * (kThreads / 32) + threadIdx.x / 32) * (4 * G) + lane / L;
    const int n = (int)a.d.states, own0 = (sl & 3) * OWN % 4;  // the first channel that it owns
    const bool owner = sl < 4;
    int64_t from, to;
    const bool live = step_slots(a.slots, a.slots_out, a.pool, q, &from, &to);
    const float* src = a.state + (live ? from * a.d.channels * n : 0);
    float* dst = a.state + (live ? to * a.d.channels * n : 0);
    float2 h[4][2], A[4][2];
    auto states = [&](const float* p, bool in, float2 (&v)[2]) {
        if (a.vec) {
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            if (in && s0 < n) x = *reinterpret_cast<const float4*>(p + s0);
            v[0] = make_float2(x.x, x.y);
            v[1] = make_float2(x.z, x.w);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                (i & 1 ? v[i / 2].y : v[i / 2].x) = in && s0 + i < n ? p[s0 + i] : 0.f;
        }
    };
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int64_t c = cw + k * G;
        states(src + c * n, live && c < a.d.channels, h[k]);
        states(a.d.A + c * n, live && c < a.d.channels, A[k]);
    }
    // B and C of the thread's states; with one group they serve all four channels
    const T* B = static_cast<const T*>(a.d.B.data) + q * a.d.B.seq_stride;
    const T* C = static_cast<const T*>(a.d.C.data) + q * a.d.C.seq_stride;
    float2 b[2], cc[2];
    auto inputs = [&](int64_t g) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const bool in = s0 + i < n;
            (i & 1 ? b[i / 2].y : b[i / 2].x) = in ? to_f(B[g * n + s0 + i]) : 0.f;
            (i & 1 ? cc[i / 2].y : cc[i / 2].x) = in ? to_f(C[g * n + s0 + i]) : 0.f;
        }
    };
    inputs(0);
    float d[OWN], du[OWN], uu[OWN], z[OWN], D[OWN];
#pragma unroll
    for (int j = 0; j < OWN; ++j) {
        const int64_t c = cw + (own0 + j) * G;
        const bool in = live && c < a.d.channels;
        uu[j] = in ? to_f(static_cast<const T*>(a.d.u.data)[q * a.d.u.seq_stride + c]) : 0.f;
        d[j] = in ? to_f(static_cast<const T*>(a.d.delta.data)[q * a.d.delta.seq_stride + c]) : 0.f;
        z[j] = in && a.d.z.data ? to_f(static_cast<const T*>(a.d.z.data)[q * a.d.z.seq_stride + c]) : 0.f;
        D[j] = in && a.d.D ? a.d.D[c] : 0.f;
        if (in && a.d.delta_bias) d[j] += a.d.delta_bias[c];
    }
#pragma unroll
    for (int j = 0; j < OWN; ++j) {
        if (a.d.softplus) d[j] = softplus(d[j]);
        du[j] = d[j] * uu[j];
    }
    float y[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int64_t c = cw + k * G;
        const int from_lane = lane - sl + k / OWN;
        const float dk = L > 1 ? __shfl_sync(0xffffffffu, d[k % OWN], from_lane) : d[k % OWN];
        const float uk = L > 1 ? __shfl_sync(0xffffffffu, du[k % OWN], from_lane) : du[k % OWN];
        if (a.d.groups > 1 && c < a.d.channels) inputs(c / (a.d.channels / a.d.groups));
        float2 acc = splat(0.f);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            h[k][i] = fma2(decay2(splat(dk), mul2(A[k][i], splat(kLog2e))), h[k][i], mul2(splat(uk), b[i]));
            if (!a.vec) {  // a state beyond n stays out of y where d u is infinite
                if (s0 + 2 * i >= n) h[k][i].x = 0.f;
                if (s0 + 2 * i + 1 >= n) h[k][i].y = 0.f;
            } else if (s0 >= n) {
                h[k][i] = splat(0.f);
            }
            acc = fma2(cc[i], h[k][i], acc);
        }
        y[k] = acc.x + acc.y;
        if (live && c < a.d.channels) {
            float* p = dst + c * n;
            if (a.vec) {
                if (s0 < n)
                    *reinterpret_cast<float4*>(p + s0) =
                        make_float4(h[k][0].x, h[k][0].y, h[k][1].x, h[k][1].y);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (s0 + i < n) p[s0 + i] = i & 1 ? h[k][i / 2].y : h[k][i / 2].x;
            }
        }
    }
    if constexpr (L >= 4) {
        hand_out<4, 2, 1>(y, sl);
#pragma unroll
        for (int w = 4; w < L; w *= 2) y[0] += __shfl_xor_sync(0xffffffffu, y[0], w);
    } else if constexpr (L == 2) {
        hand_out<4, 1, 1>(y, sl);
    }
#pragma unroll
    for (int j = 0; j < OWN; ++j) {
        const int64_t c = cw + (own0 + j) * G;
        float v = live ? fmaf(D[j], uu[j], y[j]) : 0.f;
        if (live && a.d.z.data) v *= z[j] * sigmoid(z[j]);
        if (owner && c < a.d.channels)
            static_cast<T*>(a.out.data)[q * a.out.seq_stride + c] = from_f<T>(v);
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
    constexpr int CT = kThreads / L * 4;
    a.ctiles = (a.d.channels + CT - 1) / CT;
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
