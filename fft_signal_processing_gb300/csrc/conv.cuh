// Short causal convolution along the tokens (fft_conv_forward, fft_conv_backward).
//
//   p[t] = bias + sum_k weight[k] x[t-(W-1)+k],  out = p or p * sigmoid(p)
//   dp = dout * act'(p);  dx[t] = sum_k weight[k] dp[t+(W-1)-k]
//   dweight[k] = sum_t dp[t] x[t-(W-1)+k];  dbias = sum_t dp[t]
//
// A thread holds VEC neighbouring channels (16 bytes) and walks a run of tokens with the last
// W-1 inputs in registers, so every input is read once and a run pays W-1 rows of halo.  Bound by
// HBM: 2 (backward 3) values moved per 2W (6W) operations.
#pragma once

#include "conv.h"

namespace gbfft {

constexpr int kConvRun = 16;     // tokens per thread, forward
constexpr int kConvBatch = 4;    // rows loaded ahead of their use
constexpr int kConvThreads = 128;

template <class T, int VEC>
struct Row {  // VEC channels of one token
    Pack<T, VEC> p;
};

// Channels of a block and token runs of a block: blockDim.x lanes of VEC channels,
// blockDim.y runs.
struct ConvShape {
    unsigned x, y;
};
inline ConvShape conv_shape(int64_t channels, int vec, int threads) {
    unsigned x = 1;
    while (x < (unsigned)threads && (int64_t)x * vec < channels) x *= 2;
    return {x, (unsigned)threads / x};
}

template <class T, int VEC>
__device__ __forceinline__ void load_f(const T* p, float (&v)[VEC]) {
    const Pack<T, VEC> x = ld_pack<VEC>(p);
#pragma unroll
    for (int k = 0; k < VEC; ++k) v[k] = to_f(x.v[k]);
}

// x at position t of sequence s (t < s.begin: its initial state, or zero; older: zero).
template <class T, int VEC, int W>
__device__ __forceinline__ void load_before(const ConvArgs& a, const T* x, const SeqAt& s,
                                            int64_t t, int64_t c, float (&v)[VEC]) {
    if (t >= s.begin) {
        load_f<T, VEC>(x + t * a.d.x.tok_stride + c, v);
    } else {
        const int64_t row = (W - 1) + (t - s.begin);
        if (a.d.initial_state && row >= 0) {
            load_f<T, VEC>(static_cast<const T*>(a.d.initial_state) +
                               (s.q * (W - 1) + row) * a.d.channels + c, v);
        } else {
#pragma unroll
            for (int k = 0; k < VEC; ++k) v[k] = 0.f;
        }
    }
}

template <class T, int VEC, int W>
__device__ __forceinline__ void load_weights(const ConvArgs& a, int64_t c, float (&w)[W][VEC],
                                             float (&bias)[VEC]) {
    const int f32 = a.d.param_dtype == FFT_F32;
#pragma unroll
    for (int k = 0; k < VEC; ++k) {
#pragma unroll
        for (int i = 0; i < W; ++i) w[i][k] = ld_param<T>(a.d.weight, (c + k) * W + i, f32);
        bias[k] = a.d.bias ? ld_param<T>(a.d.bias, c + k, f32) : 0.f;
    }
}

// The last W-1 inputs of every sequence: one block per sequence and channel tile.
template <class T, int VEC, int W>
__device__ void conv_final(const ConvArgs& a, int64_t q, int64_t c) {
    const SeqAt s = a.d.offsets ? SeqAt{q, a.d.offsets[q], a.d.offsets[q + 1]}
                                : SeqAt{q, 0, a.d.length};
    if (s.begin < 0 || s.end < s.begin || s.end > a.d.length || c >= a.d.channels) return;
    const T* x = static_cast<const T*>(a.d.x.data) + (a.d.offsets ? 0 : q * a.d.x.seq_stride);
    for (int r = 0; r < W - 1; ++r) {
        float v[VEC];
        load_before<T, VEC, W>(a, x, s, s.end - (W - 1) + r, c, v);
        Pack<T, VEC> p;
#pragma unroll
        for (int k = 0; k < VEC; ++k) p.v[k] = from_f<T>(v[k]);
        st_pack<VEC>(static_cast<T*>(a.final_state) + (q * (W - 1) + r) * a.d.channels + c, p);
    }
}

template <class T, int VEC, int W>
__global__ void __launch_bounds__(kConvThreads) k_conv_fwd(const ConvArgs a) {
    const int64_t ct = blockIdx.x % a.ctiles, tile = blockIdx.x / a.ctiles;
    const int64_t c = (ct * blockDim.x + threadIdx.x) * VEC;
    const int64_t rows = a.d.offsets ? 1 : a.d.nseq;
    if (tile >= rows * a.ttiles) {  // the blocks behind the outputs: final states
        const int64_t q = tile - rows * a.ttiles;
        if (threadIdx.y == 0) conv_final<T, VEC, W>(a, q, c);
        return;
    }
    const int64_t row = tile / a.ttiles;
    const int64_t t0 = ((tile - row * a.ttiles) * blockDim.y) * kConvRun;
    const int64_t b = t0 + (int64_t)threadIdx.y * kConvRun;
    const int64_t e = b + kConvRun < a.d.length ? b + kConvRun : a.d.length;
    // packed rows: the whole warp looks for the block's first token, then each run walks on
    SeqAt s = seq_at(a.d.offsets, a.d.nseq, a.d.length, row, t0);
    if (c >= a.d.channels || b >= e) return;
    seq_next(a.d.offsets, a.d.nseq, b, &s);
    const T* x = static_cast<const T*>(a.d.x.data) + (a.d.offsets ? 0 : row * a.d.x.seq_stride);
    T* out = static_cast<T*>(a.out.data) + (a.d.offsets ? 0 : row * a.out.seq_stride);
    float w[W][VEC], bias[VEC], win[W][VEC];
    load_weights<T, VEC, W>(a, c, w, bias);
#pragma unroll
    for (int i = 0; i < W - 1; ++i)
        load_before<T, VEC, W>(a, x, s, b - (W - 1) + i, c, win[i]);
    for (int64_t t = b; t < e; t += kConvBatch) {
        Pack<T, VEC> next[kConvBatch];
#pragma unroll
        for (int j = 0; j < kConvBatch; ++j)
            if (t + j < e) next[j] = ld_pack<VEC>(x + (t + j) * a.d.x.tok_stride + c);
#pragma unroll
        for (int j = 0; j < kConvBatch; ++j) {
            if (t + j >= e) break;
            if (t + j >= s.end) {  // packed: the next sequence begins here
                seq_next(a.d.offsets, a.d.nseq, t + j, &s);
#pragma unroll
                for (int i = 0; i < W - 1; ++i)
                    load_before<T, VEC, W>(a, x, s, t + j - (W - 1) + i, c, win[i]);
            }
            Pack<T, VEC> y;
#pragma unroll
            for (int k = 0; k < VEC; ++k) {
                win[W - 1][k] = to_f(next[j].v[k]);
                float p = bias[k];
#pragma unroll
                for (int i = 0; i < W; ++i) p += w[i][k] * win[i][k];
                if (a.d.silu) p *= sigmoid(p);
                y.v[k] = from_f<T>(p);
#pragma unroll
                for (int i = 0; i < W - 1; ++i) win[i][k] = win[i + 1][k];
            }
            st_pack<VEC>(out + (t + j) * a.out.tok_stride + c, y);
        }
    }
}

__device__ __forceinline__ float act_grad(float p, float dout, int silu) {
    if (!silu) return dout;
    const float g = sigmoid(p);
    return dout * (g * (1.f + p * (1.f - g)));
}

// Gradient of every sequence's initial state: row r of the state reaches the outputs of tokens
// r - k, k <= r, and (in a sequence shorter than the state) the final state's row r - length.
template <class T, int VEC, int W>
__device__ void conv_dinitial(const ConvArgs& a, int64_t q, int64_t c) {
    const SeqAt s = a.d.offsets ? SeqAt{q, a.d.offsets[q], a.d.offsets[q + 1]}
                                : SeqAt{q, 0, a.d.length};
    if (s.begin < 0 || s.end < s.begin || s.end > a.d.length || c >= a.d.channels) return;
    const int64_t base = a.d.offsets ? 0 : q;
    const T* x = static_cast<const T*>(a.d.x.data) + base * a.d.x.seq_stride;
    const T* dout = static_cast<const T*>(a.dout.data) + base * a.dout.seq_stride;
    const int64_t len = s.end - s.begin;
    float w[W][VEC], bias[VEC], acc[W][VEC] = {};
    load_weights<T, VEC, W>(a, c, w, bias);
    for (int64_t t = 0; t < W - 1 && t < len; ++t) {
        float p[VEC], g[VEC];
#pragma unroll
        for (int k = 0; k < VEC; ++k) p[k] = bias[k];
#pragma unroll
        for (int i = 0; i < W; ++i) {
            float v[VEC];
            load_before<T, VEC, W>(a, x, s, s.begin + t - (W - 1) + i, c, v);
#pragma unroll
            for (int k = 0; k < VEC; ++k) p[k] += w[i][k] * v[k];
        }
        load_f<T, VEC>(dout + (s.begin + t) * a.dout.tok_stride + c, g);
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
            const float dp = act_grad(p[k], g[k], a.d.silu);
#pragma unroll
            for (int r = 0; r < W - 1; ++r)  // tap i = r - t of the state's row r
#pragma unroll
                for (int i = 0; i < W; ++i)
                    if (r - t == i) acc[r][k] += w[i][k] * dp;
        }
    }
#pragma unroll
    for (int r = 0; r < W - 1; ++r) {
        Pack<T, VEC> p;
        float f[VEC] = {};
        if (a.final_state && r >= len)
            load_f<T, VEC>(static_cast<const T*>(a.final_state) +
                               (q * (W - 1) + (r - len)) * a.d.channels + c, f);
#pragma unroll
        for (int k = 0; k < VEC; ++k) p.v[k] = from_f<T>(acc[r][k] + f[k]);
        st_pack<VEC>(static_cast<T*>(a.dinitial) + (q * (W - 1) + r) * a.d.channels + c, p);
    }
}

// Backward.  A run walks its tokens [b, e) and W-1 more: dp of the tokens up to e-1+(W-1) gives
// dx of [b, e); only dp of its own tokens enters dweight and dbias.  The runs of a block are
// summed in shared memory, one partial row per token tile.
template <class T, int VEC, int W>
__global__ void __launch_bounds__(kConvThreads) k_conv_bwd(const ConvArgs a) {
    extern __shared__ float red[];  // [blockDim.y][blockDim.x * VEC], used once per tap
    const int64_t ct = blockIdx.x % a.ctiles, tile = blockIdx.x / a.ctiles;
    const int64_t c = (ct * blockDim.x + threadIdx.x) * VEC;
    const int64_t rows = a.d.offsets ? 1 : a.d.nseq;
    if (tile >= rows * a.ttiles) {
        if (threadIdx.y == 0) conv_dinitial<T, VEC, W>(a, tile - rows * a.ttiles, c);
        return;
    }
    const int64_t row = tile / a.ttiles, run = kConvBwdTokens / blockDim.y;
    const int64_t t0 = (tile - row * a.ttiles) * kConvBwdTokens;
    const int64_t b = t0 + (int64_t)threadIdx.y * run;
    const int64_t e = b + run < a.d.length ? b + run : a.d.length;
    SeqAt s = seq_at(a.d.offsets, a.d.nseq, a.d.length, row, t0);
    float dw[W][VEC] = {}, db[VEC] = {};
    if (c < a.d.channels && b < e) {
        seq_next(a.d.offsets, a.d.nseq, b, &s);
        const int64_t base = a.d.offsets ? 0 : row;
        const T* x = static_cast<const T*>(a.d.x.data) + base * a.d.x.seq_stride;
        const T* dout = static_cast<const T*>(a.dout.data) + base * a.dout.seq_stride;
        T* dx = static_cast<T*>(a.out.data) + base * a.out.seq_stride;
        const T* dfin = static_cast<const T*>(a.final_state);
        float w[W][VEC], bias[VEC], win[W][VEC], dps[W][VEC] = {};
        load_weights<T, VEC, W>(a, c, w, bias);
#pragma unroll
        for (int i = 0; i < W - 1; ++i)
            load_before<T, VEC, W>(a, x, s, b - (W - 1) + i, c, win[i]);
        // dps[j] is dp of token t - (W-1) + j; past a sequence's end it is 0, and dfinal joins
        SeqAt cur = s;  // the sequence of token t - (W-1), whose dx leaves at step t
        int64_t dp_end = s.end < a.d.length ? s.end : a.d.length;
        for (int64_t t = b; t < e + (W - 1); ++t) {
            float xv[VEC] = {}, g[VEC] = {};
            const bool in = t < a.d.length;
            if (in) {
                load_f<T, VEC>(x + t * a.d.x.tok_stride + c, xv);
                load_f<T, VEC>(dout + t * a.dout.tok_stride + c, g);
                if (t >= s.end) {
                    seq_next(a.d.offsets, a.d.nseq, t, &s);
#pragma unroll
                    for (int i = 0; i < W - 1; ++i)
                        load_before<T, VEC, W>(a, x, s, t - (W - 1) + i, c, win[i]);
                }
            }
#pragma unroll
            for (int k = 0; k < VEC; ++k) {
                win[W - 1][k] = xv[k];
                float p = bias[k];
#pragma unroll
                for (int i = 0; i < W; ++i) p += w[i][k] * win[i][k];
                const float dp = in ? act_grad(p, g[k], a.d.silu) : 0.f;
                dps[W - 1][k] = dp;
                if (t < e) {
                    db[k] += dp;
#pragma unroll
                    for (int i = 0; i < W; ++i) dw[i][k] += dp * win[i][k];
                }
#pragma unroll
                for (int i = 0; i < W - 1; ++i) win[i][k] = win[i + 1][k];
            }
            const int64_t td = t - (W - 1);  // dx[td] = sum_j weight[W-1-j] dp[td + j]
            if (td >= b && a.out.data) {
                if (td >= cur.end) {
                    seq_next(a.d.offsets, a.d.nseq, td, &cur);
                    dp_end = cur.end < a.d.length ? cur.end : a.d.length;
                }
                float f[VEC] = {};
                const int64_t fr = td + (W - 1) - dp_end;  // row of the final state that td is
                if (dfin && fr >= 0 && fr < W - 1)
                    load_f<T, VEC>(dfin + (cur.q * (W - 1) + fr) * a.d.channels + c, f);
                Pack<T, VEC> y;
#pragma unroll
                for (int k = 0; k < VEC; ++k) {
                    float d = f[k];
#pragma unroll
                    for (int j = 0; j < W; ++j)
                        if (td + j < dp_end) d += w[W - 1 - j][k] * dps[j][k];
                    y.v[k] = from_f<T>(d);
                }
                st_pack<VEC>(dx + td * a.out.tok_stride + c, y);
            }
#pragma unroll
            for (int k = 0; k < VEC; ++k)
#pragma unroll
                for (int i = 0; i < W - 1; ++i) dps[i][k] = dps[i + 1][k];
        }
    }
    if (!a.parts) return;
    const int lanes = (int)blockDim.x * VEC;
#pragma unroll
    for (int i = 0; i <= W; ++i) {
        __syncthreads();
#pragma unroll
        for (int k = 0; k < VEC; ++k)
            red[threadIdx.y * lanes + threadIdx.x * VEC + k] = i < W ? dw[i < W ? i : 0][k] : db[k];
        __syncthreads();
        const int tid = (int)(threadIdx.y * blockDim.x + threadIdx.x);
        for (int l = tid; l < lanes; l += kConvThreads) {
            const int64_t ch = ct * lanes + l;
            if (ch < a.d.channels) {
                float v = 0.f;
                for (int y = 0; y < (int)blockDim.y; ++y) v += red[y * lanes + l];
                a.parts[(tile * (W + 1) + i) * a.d.channels + ch] = v;
            }
        }
    }
}

template <class T, int VEC, int W>
cudaError_t conv_launch(ConvArgs a, bool backward, cudaStream_t s) {
    const ConvShape sh = conv_shape(a.d.channels, VEC, kConvThreads);
    const int64_t rows = a.d.offsets ? 1 : a.d.nseq;
    a.ctiles = (a.d.channels + (int64_t)sh.x * VEC - 1) / ((int64_t)sh.x * VEC);
    const int64_t per = backward ? kConvBwdTokens : (int64_t)sh.y * kConvRun;
    a.ttiles = (a.d.length + per - 1) / per;
    const bool states = W > 1 && (backward ? a.dinitial : a.final_state) != nullptr;
    const int64_t blocks = a.ctiles * (rows * a.ttiles + (states ? a.d.nseq : 0));
    if (blocks < 1) return cudaSuccess;
    if (blocks > INT32_MAX) return cudaErrorInvalidValue;
    if (backward)
        k_conv_bwd<T, VEC, W><<<(unsigned)blocks, dim3(sh.x, sh.y),
                                sizeof(float) * kConvThreads * VEC, s>>>(a);
    else
        k_conv_fwd<T, VEC, W><<<(unsigned)blocks, dim3(sh.x, sh.y), 0, s>>>(a);
    return cudaGetLastError();
}

template <class T, int VEC>
cudaError_t conv_width(const ConvArgs& a, bool backward, cudaStream_t s) {
    switch (a.d.width) {
        case 1: return conv_launch<T, VEC, 1>(a, backward, s);
        case 2: return conv_launch<T, VEC, 2>(a, backward, s);
        case 3: return conv_launch<T, VEC, 3>(a, backward, s);
        case 4: return conv_launch<T, VEC, 4>(a, backward, s);
        case 5: return conv_launch<T, VEC, 5>(a, backward, s);
        case 6: return conv_launch<T, VEC, 6>(a, backward, s);
        case 7: return conv_launch<T, VEC, 7>(a, backward, s);
        case 8: return conv_launch<T, VEC, 8>(a, backward, s);
        default: return cudaErrorInvalidValue;
    }
}

// VEC values per access where every row starts on such a boundary, else single values.
template <class T, int VEC>
cudaError_t conv_run(const ConvArgs& a, bool backward, cudaStream_t s) {
    const bool packed = a.d.offsets != nullptr;
    const int64_t bytes = VEC * sizeof(T);
    auto rows_ok = [&](const fft_seq& q) {
        return !q.data || (aligned_to(q.data, bytes) && q.tok_stride % VEC == 0 &&
                           (packed || q.seq_stride % VEC == 0));
    };
    const bool vec = a.d.channels % VEC == 0 && rows_ok(a.d.x) && rows_ok(a.out) &&
                     (!backward || rows_ok(a.dout)) && aligned_to(a.d.initial_state, bytes) &&
                     aligned_to(a.final_state, bytes) && aligned_to(a.dinitial, bytes);
    return vec ? conv_width<T, VEC>(a, backward, s) : conv_width<T, 1>(a, backward, s);
}

}  // namespace gbfft
