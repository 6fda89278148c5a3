// Short causal convolution along the tokens (fft_conv_forward, fft_conv_backward).
//
//   p[t] = bias + sum_k weight[k] x[t-(W-1)+k],  out = p or p * sigmoid(p)
//   dp = dout * act'(p);  dx[t] = sum_k weight[k] dp[t+(W-1)-k]
//   dweight[k] = sum_t dp[t] x[t-(W-1)+k];  dbias = sum_t dp[t]
//
// A thread holds VEC neighbouring channels (8 bytes) and walks a run of up to 64 tokens with the last W-1
// inputs (and, backward, the last W-1 dp) in registers, so a run reads its rows once and W-1
// (backward 2(W-1)) rows of halo.  Channels go in pairs, two float32 operations to an
// instruction.  Tokens go by fours: their rows come by asynchronous copies into the thread's own
// places in shared memory, three fours ahead, which keeps more loads in flight than the registers
// would; inside a sequence the window slides by renaming, at sequence ends and in the halo tokens
// go one by one.  2 (backward 3) values are moved per 2W (6W) operations: forward is bound by HBM
// (4 x 4096 tokens of 4096 bfloat16 channels, W = 4: 51 us, 5.2 TB/s), backward by the
// 16 warps of an SM that 126 registers leave (16001 packed tokens of 2000 channels:
// 78 us, 2.5 TB/s, 2.0 of 4 instructions a cycle).  16 bytes a thread took so many registers that it
// was slower (78 and 107 us at the time, against 72 and 89), 4 bytes too many instructions (83,
// 107).
#pragma once

#include "conv.h"
#include "launch_cache.cuh"

namespace gbfft {

constexpr int kConvBatch = 4;
constexpr int kConvAhead = 3;  // fours of rows on their way
constexpr int kConvThreads = kConvLanes * kConvRuns;

// The rows of a run, in fours, R tensors side by side.  VEC 1: no ring, rows are loaded when they
// are needed.
template <class T, int VEC, int R>
struct ConvRing {
    static constexpr bool kOn = VEC * sizeof(T) == 8;
    static constexpr int kFours = kConvAhead + 1;
    static constexpr int kBytes = kOn ? kFours * kConvBatch * R * kConvThreads * 8 : 0;
    // [four][row][tensor][thread]; `four` counts from the run's start
    char* mine;  // the thread's place
    __device__ __forceinline__ explicit ConvRing(void* memory)
        : mine(static_cast<char*>(memory) + (threadIdx.y * kConvLanes + threadIdx.x) * 8) {}
    __device__ __forceinline__ char* at(int four, int row, int r) const {
        return mine + (four % kFours) * (kConvBatch * R * kConvThreads * 8) +
               (row * R + r) * (kConvThreads * 8);
    }
    __device__ __forceinline__ Pack<T, VEC> get(int four, int row, int r) const {
        return *reinterpret_cast<const Pack<T, VEC>*>(at(four, row, r));
    }
    // row 4 * four + j of a tensor at p + j * stride, rows from `left` on do not exist
    __device__ __forceinline__ void copy(int four, int r, const T* p, int64_t stride, int left) const {
        if (left >= kConvBatch) {
#pragma unroll
            for (int j = 0; j < kConvBatch; ++j, p += stride) copy8(at(four, j, r), p, true);
        } else {
#pragma unroll
            for (int j = 0; j < kConvBatch; ++j)
                if (j < left) copy8(at(four, j, r), p + j * stride, true);
        }
    }
};
template <int VEC>
struct Pairs {  // VEC channels; one channel leaves the second half idle
    static constexpr int P = (VEC + 1) / 2;
    float2 v[P];
};
template <class T, int VEC>
__device__ __forceinline__ Pairs<VEC> widen(const Pack<T, VEC>& x) {
    Pairs<VEC> r;
#pragma unroll
    for (int p = 0; p < Pairs<VEC>::P; ++p)
        r.v[p] = make_float2(to_f(x.v[2 * p]), VEC > 1 ? to_f(x.v[VEC > 1 ? 2 * p + 1 : 0]) : 0.f);
    return r;
}
template <class T, int VEC>
__device__ __forceinline__ Pack<T, VEC> narrow(const Pairs<VEC>& x) {
    Pack<T, VEC> r;
    if constexpr (VEC == 1) {
        r.v[0] = from_f<T>(x.v[0].x);
    } else {
#pragma unroll
        for (int p = 0; p < VEC / 2; ++p) {
            const Pack<T, 2> y = from_f2<T>(x.v[p]);
            r.v[2 * p] = y.v[0];
            r.v[2 * p + 1] = y.v[1];
        }
    }
    return r;
}
template <int VEC>
__device__ __forceinline__ Pairs<VEC> zeros() {
    Pairs<VEC> r;
#pragma unroll
    for (int p = 0; p < Pairs<VEC>::P; ++p) r.v[p] = make_float2(0.f, 0.f);
    return r;
}

// x at position t of sequence s (t < s.begin: its initial state, or zero; older: zero); x points
// at channel c.
template <class T, int VEC, int W>
__device__ __forceinline__ Pairs<VEC> load_before(const ConvArgs& a, const T* x, const SeqAt& s,
                                                  int64_t t, int64_t c) {
    if (t >= s.begin) return widen<T, VEC>(ld_pack<VEC>(x + t * a.d.x.tok_stride));
    const int64_t row = (W - 1) + (t - s.begin);
    if (a.d.initial_state && row >= 0)
        return widen<T, VEC>(ld_pack<VEC>(static_cast<const T*>(a.d.initial_state) +
                                          (s.q * (W - 1) + row) * a.d.channels + c));
    return zeros<VEC>();
}

template <class T, int VEC, int W>
__device__ __forceinline__ void load_weights(const ConvArgs& a, int64_t c, Pairs<VEC> (&w)[W],
                                             Pairs<VEC>& bias) {
    const int f32 = a.d.param_dtype == FFT_F32;
    bias = zeros<VEC>();
#pragma unroll
    for (int i = 0; i < W; ++i) w[i] = zeros<VEC>();
#pragma unroll
    for (int k = 0; k < VEC; ++k) {
#pragma unroll
        for (int i = 0; i < W; ++i)
            (k & 1 ? w[i].v[k / 2].y : w[i].v[k / 2].x) = ld_param<T>(a.d.weight, (c + k) * W + i, f32);
        if (a.d.bias) (k & 1 ? bias.v[k / 2].y : bias.v[k / 2].x) = ld_param<T>(a.d.bias, c + k, f32);
    }
}

__device__ __forceinline__ SeqAt conv_seq(const ConvArgs& a, int64_t q) {
    return a.d.offsets ? SeqAt{q, a.d.offsets[q], a.d.offsets[q + 1]} : SeqAt{q, 0, a.d.length};
}

// The last W-1 inputs of every sequence: the blocks behind the outputs.
template <class T, int VEC, int W>
__device__ void conv_final(const ConvArgs& a, int64_t q, int64_t c) {
    const SeqAt s = conv_seq(a, q);
    if (s.begin < 0 || s.end < s.begin || s.end > a.d.length || c >= a.d.channels) return;
    const T* x = static_cast<const T*>(a.d.x.data) + (a.d.offsets ? 0 : q * a.d.x.seq_stride) + c;
    for (int r = 0; r < W - 1; ++r)
        st_pack<VEC>(static_cast<T*>(a.final_state) + (q * (W - 1) + r) * a.d.channels + c,
                     narrow<T, VEC>(load_before<T, VEC, W>(a, x, s, s.end - (W - 1) + r, c)));
}

template <class T, int VEC, int W>
__global__ void __launch_bounds__(kConvThreads) k_conv_fwd(const ConvArgs a) {
    constexpr int P = Pairs<VEC>::P, N = kConvBatch;
    using Ring = ConvRing<T, VEC, 1>;
    extern __shared__ uint2 ring_memory[];
    const Ring ring(ring_memory);
    const int64_t ct = blockIdx.x % a.ctiles, tile = blockIdx.x / a.ctiles;
    const int64_t c = (ct * kConvLanes + threadIdx.x) * VEC;
    const int64_t rows = a.d.offsets ? 1 : a.d.nseq;
    if (tile >= rows * a.ttiles) {
        if (threadIdx.y == 0) conv_final<T, VEC, W>(a, tile - rows * a.ttiles, c);
        return;
    }
    const int64_t row = tile / a.ttiles;
    const int64_t b = ((tile - row * a.ttiles) * kConvRuns + threadIdx.y) * a.run;
    const int64_t e = b + a.run < a.d.length ? b + a.run : a.d.length;
    if (b >= e) return;  // a warp is one run
    SeqAt s = seq_at(a.d.offsets, a.d.nseq, a.d.length, row, b);
    if (c >= a.d.channels) return;
    const int64_t xs = a.d.x.tok_stride, os = a.out.tok_stride;
    const T* x0 = static_cast<const T*>(a.d.x.data) + (a.d.offsets ? 0 : row * a.d.x.seq_stride) + c;
    T* out = static_cast<T*>(a.out.data) + (a.d.offsets ? 0 : row * a.out.seq_stride);
    Pairs<VEC> w[W], bias, win[W - 1 + N];  // win[W-1] is the token at hand
    load_weights<T, VEC, W>(a, c, w, bias);
    auto refill = [&](int64_t t) {
#pragma unroll
        for (int i = 0; i < W - 1; ++i) win[i] = load_before<T, VEC, W>(a, x0, s, t - (W - 1) + i, c);
    };
    auto emit = [&](int j, T* o) {  // the output of token j of the window
        Pairs<VEC> y;
#pragma unroll
        for (int p = 0; p < P; ++p) {
            float2 v = bias.v[p];
#pragma unroll
            for (int i = 0; i < W; ++i) v = fma2(w[i].v[p], win[j + i].v[p], v);
            if (a.d.silu) v = mul2(v, sigmoid2(v));
            y.v[p] = v;
        }
        st_pack<VEC>(o, narrow<T, VEC>(y));
    };
    auto slide = [&](int by) {
#pragma unroll
        for (int i = 0; i < W - 1; ++i) win[i] = win[by + i];
    };
    const int len = (int)(e - b);
    const T* x = x0 + b * xs;  // rows count from the run's start
    const T* next = x;
    auto ahead = [&](int four) {
        ring.copy(four, 0, next, xs, len - four * N);
        next += N * xs;
        copy_commit();
    };
    if constexpr (Ring::kOn) {
#pragma unroll
        for (int k = 0; k < kConvAhead; ++k) ahead(k);
    }
    refill(b);
    T* op = out + b * os + c;
    for (int i = 0, four = 0; i < len; i += N, ++four, op += N * os) {
        if constexpr (Ring::kOn) {
            ahead(four + kConvAhead);
            copy_wait<kConvAhead>();
        }
        auto row_at = [&](int j) {
            if constexpr (Ring::kOn) return ring.get(four, j, 0);
            return ld_pack<VEC>(x + (i + j) * xs);
        };
        if (i + N <= len && b + i + N <= s.end) {
            Pack<T, VEC> rows_[N];
#pragma unroll
            for (int j = 0; j < N; ++j) rows_[j] = row_at(j);
#pragma unroll
            for (int j = 0; j < N; ++j) win[W - 1 + j] = widen<T, VEC>(rows_[j]);
#pragma unroll
            for (int j = 0; j < N; ++j) emit(j, op + j * os);
            slide(N);
        } else {
            for (int j = 0; j < N && i + j < len; ++j) {
                if (b + i + j >= s.end) {  // packed: the next sequence begins here
                    const int64_t q = s.q;
                    seq_next(a.d.offsets, a.d.nseq, b + i + j, &s);
                    if (s.q != q) refill(b + i + j);
                }
                win[W - 1] = widen<T, VEC>(row_at(j));
                emit(0, op + j * os);
                slide(1);
            }
        }
    }
    if constexpr (Ring::kOn) copy_wait<0>();
}

// dout * act'(p), act = silu: g (1 + p (1 - g)) with g = sigmoid(p)
__device__ __forceinline__ float2 act_grad(float2 p, float2 dout, int silu) {
    if (!silu) return dout;
    const float2 g = sigmoid2(p);
    const float2 r = fma2(p, fma2(g, splat(-1.f), splat(1.f)), splat(1.f));
    return mul2(dout, mul2(g, r));
}

// Gradient of every sequence's initial state: row r of the state reaches the outputs of tokens
// r - k, k <= r, and (in a sequence shorter than the state) the final state's row r - length.
template <class T, int VEC, int W>
__device__ void conv_dinitial(const ConvArgs& a, int64_t q, int64_t c) {
    constexpr int P = Pairs<VEC>::P;
    const SeqAt s = conv_seq(a, q);
    if (s.begin < 0 || s.end < s.begin || s.end > a.d.length || c >= a.d.channels) return;
    const int64_t base = a.d.offsets ? 0 : q;
    const T* x = static_cast<const T*>(a.d.x.data) + base * a.d.x.seq_stride + c;
    const T* dout = static_cast<const T*>(a.dout.data) + base * a.dout.seq_stride;
    const int64_t len = s.end - s.begin;
    Pairs<VEC> w[W], bias, acc[W];
    load_weights<T, VEC, W>(a, c, w, bias);
#pragma unroll
    for (int r = 0; r < W; ++r) acc[r] = zeros<VEC>();
    for (int64_t t = 0; t < W - 1 && t < len; ++t) {
        Pairs<VEC> p = bias;
#pragma unroll
        for (int i = 0; i < W; ++i) {
            const Pairs<VEC> v = load_before<T, VEC, W>(a, x, s, s.begin + t - (W - 1) + i, c);
#pragma unroll
            for (int k = 0; k < P; ++k) p.v[k] = fma2(w[i].v[k], v.v[k], p.v[k]);
        }
        const Pairs<VEC> g = widen<T, VEC>(ld_pack<VEC>(dout + (s.begin + t) * a.dout.tok_stride + c));
#pragma unroll
        for (int k = 0; k < P; ++k) {
            const float2 dp = act_grad(p.v[k], g.v[k], a.d.silu);
#pragma unroll
            for (int r = 0; r < W - 1; ++r)  // tap i = r - t of the state's row r
#pragma unroll
                for (int i = 0; i < W; ++i)
                    if (r - t == i) acc[r].v[k] = fma2(w[i].v[k], dp, acc[r].v[k]);
        }
    }
#pragma unroll
    for (int r = 0; r < W - 1; ++r) {
        if (a.final_state && r >= len) {
            const Pairs<VEC> f = widen<T, VEC>(ld_pack<VEC>(
                static_cast<const T*>(a.final_state) + (q * (W - 1) + (r - len)) * a.d.channels + c));
#pragma unroll
            for (int k = 0; k < P; ++k) acc[r].v[k] = add2(acc[r].v[k], f.v[k]);
        }
        st_pack<VEC>(static_cast<T*>(a.dinitial) + (q * (W - 1) + r) * a.d.channels + c,
                     narrow<T, VEC>(acc[r]));
    }
}

// Backward.  A run walks its tokens [b, e) and W-1 more: dp of the tokens up to e-1+(W-1) gives
// dx of [b, e); only dp of its own tokens enters dweight and dbias.  The runs of a block are
// summed in shared memory, one partial row per token tile.
template <class T, int VEC, int W>
__global__ void __launch_bounds__(kConvThreads) k_conv_bwd(const ConvArgs a) {
    constexpr int P = Pairs<VEC>::P, N = kConvBatch, LANES = kConvLanes * VEC;
    using Ring = ConvRing<T, VEC, 2>;
    extern __shared__ uint2 ring_memory[];
    const Ring ring(ring_memory);
    __shared__ float red[kConvRuns][LANES];
    const int64_t ct = blockIdx.x % a.ctiles, tile = blockIdx.x / a.ctiles;
    const int64_t c = (ct * kConvLanes + threadIdx.x) * VEC;
    const int64_t rows = a.d.offsets ? 1 : a.d.nseq;
    if (tile >= rows * a.ttiles) {
        if (threadIdx.y == 0) conv_dinitial<T, VEC, W>(a, tile - rows * a.ttiles, c);
        return;
    }
    const int64_t row = tile / a.ttiles;
    const int64_t b = ((tile - row * a.ttiles) * kConvRuns + threadIdx.y) * a.run;
    const int64_t e = b + a.run < a.d.length ? b + a.run : a.d.length;
    Pairs<VEC> dw[W], db = zeros<VEC>();
#pragma unroll
    for (int i = 0; i < W; ++i) dw[i] = zeros<VEC>();
    SeqAt s = {0, 0, 0};
    if (b < e) s = seq_at(a.d.offsets, a.d.nseq, a.d.length, row, b);  // a warp is one run
    if (c < a.d.channels && b < e) {
        const int64_t base = a.d.offsets ? 0 : row;
        const int64_t xs = a.d.x.tok_stride, gs = a.dout.tok_stride, os = a.out.tok_stride;
        const T* x0 = static_cast<const T*>(a.d.x.data) + base * a.d.x.seq_stride + c;
        const T* x = x0 + b * xs;  // rows count from the run's start
        const T* dout = static_cast<const T*>(a.dout.data) + base * a.dout.seq_stride + b * gs + c;
        const int len = (int)(e - b), all = len + W - 1;  // own tokens, and with the halo
        const int fours = (all + N - 1) / N * N;
        const int there = a.d.length - b < fours ? (int)(a.d.length - b) : fours;  // that exist
        const T* nextx = x;
        const T* nextg = dout;
        auto ahead = [&](int four) {
            ring.copy(four, 0, nextx, xs, there - four * N);
            ring.copy(four, 1, nextg, gs, there - four * N);
            nextx += N * xs;
            nextg += N * gs;
            copy_commit();
        };
        if constexpr (Ring::kOn) {
#pragma unroll
            for (int k = 0; k < kConvAhead; ++k) ahead(k);
        }
        T* dx = a.out.data ? static_cast<T*>(a.out.data) + base * a.out.seq_stride + c : nullptr;
        const T* dfin = static_cast<const T*>(a.final_state);
        Pairs<VEC> w[W], bias, win[W - 1 + N], dps[W - 1 + N];
        load_weights<T, VEC, W>(a, c, w, bias);
        auto refill = [&](int64_t t) {
#pragma unroll
            for (int i = 0; i < W - 1; ++i)
                win[i] = load_before<T, VEC, W>(a, x0, s, t - (W - 1) + i, c);
        };
        // dp of token j of the window from its dout
        auto grad = [&](int j, const Pairs<VEC>& g) {
#pragma unroll
            for (int p = 0; p < P; ++p) {
                float2 v = bias.v[p];
#pragma unroll
                for (int i = 0; i < W; ++i) v = fma2(w[i].v[p], win[j + i].v[p], v);
                dps[W - 1 + j].v[p] = act_grad(v, g.v[p], a.d.silu);
            }
        };
        auto params = [&](int j, bool own) {
            if (!own) return;
#pragma unroll
            for (int p = 0; p < P; ++p) {
                db.v[p] = add2(db.v[p], dps[W - 1 + j].v[p]);
#pragma unroll
                for (int i = 0; i < W; ++i)
                    dw[i].v[p] = fma2(dps[W - 1 + j].v[p], win[j + i].v[p], dw[i].v[p]);
            }
        };
        auto slide = [&](int by) {
#pragma unroll
            for (int i = 0; i < W - 1; ++i) {
                win[i] = win[by + i];
                dps[i] = dps[by + i];
            }
        };
#pragma unroll
        for (int i = 0; i < W - 1; ++i) dps[i] = zeros<VEC>();
        refill(b);
        SeqAt cur = s;  // the sequence of token t - (W-1), whose dx leaves at step t
        for (int i = 0, four = 0; i < all; i += N, ++four) {
            if constexpr (Ring::kOn) {
                ahead(four + kConvAhead);
                copy_wait<kConvAhead>();
            }
            auto x_at = [&](int j) {
                if constexpr (Ring::kOn) return ring.get(four, j, 0);
                return ld_pack<VEC>(x + (i + j) * xs);
            };
            auto g_at = [&](int j) {
                if constexpr (Ring::kOn) return ring.get(four, j, 1);
                return ld_pack<VEC>(dout + (i + j) * gs);
            };
            const int64_t t0 = b + i;
            if ((i == 0 || t0 - (W - 1) >= s.begin) && i + N <= there && t0 + N <= s.end) {
                // inside one sequence, and so are the tokens whose dx leaves (those of the run)
                Pack<T, VEC> nx[N], ng[N];
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    nx[j] = x_at(j);
                    ng[j] = g_at(j);
                }
#pragma unroll
                for (int j = 0; j < N; ++j) win[W - 1 + j] = widen<T, VEC>(nx[j]);
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    grad(j, widen<T, VEC>(ng[j]));
                    params(j, i + j < len);
                }
                if (dx) {
                    T* o = dx + (t0 - (W - 1)) * os;
#pragma unroll
                    for (int j = 0; j < N; ++j) {
                        Pairs<VEC> y = zeros<VEC>();
#pragma unroll
                        for (int p = 0; p < P; ++p)
#pragma unroll
                            for (int k = 0; k < W; ++k)
                                y.v[p] = fma2(w[W - 1 - k].v[p], dps[j + k].v[p], y.v[p]);
                        if (i + j >= W - 1 && i + j < all) st_pack<VEC>(o + j * os, narrow<T, VEC>(y));
                    }
                }
                slide(N);
                cur = s;
                continue;
            }
            for (int j = 0; j < N && i + j < all; ++j) {
                const int64_t t = t0 + j;
                win[W - 1] = dps[W - 1] = zeros<VEC>();
                if (i + j < there) {
                    if (t >= s.end) {  // packed: the next sequence begins here
                        const int64_t q = s.q;
                        seq_next(a.d.offsets, a.d.nseq, t, &s);
                        if (s.q != q) refill(t);
                    }
                    win[W - 1] = widen<T, VEC>(x_at(j));
                    grad(0, widen<T, VEC>(g_at(j)));
                    params(0, t < e);
                }
                const int64_t td = t - (W - 1);  // dx[td] = sum_k weight[W-1-k] dp[td + k]
                if (td >= b && dx) {
                    if (td >= cur.end) seq_next(a.d.offsets, a.d.nseq, td, &cur);
                    const int64_t end = cur.end < a.d.length ? cur.end : a.d.length;
                    Pairs<VEC> y = zeros<VEC>();
                    const int64_t fr = td + (W - 1) - end;  // row of the final state that td is
                    if (dfin && fr >= 0 && fr < W - 1)
                        y = widen<T, VEC>(
                            ld_pack<VEC>(dfin + (cur.q * (W - 1) + fr) * a.d.channels + c));
#pragma unroll
                    for (int p = 0; p < P; ++p)
#pragma unroll
                        for (int k = 0; k < W; ++k)
                            if (td + k < end) y.v[p] = fma2(w[W - 1 - k].v[p], dps[k].v[p], y.v[p]);
                    st_pack<VEC>(dx + td * os, narrow<T, VEC>(y));
                }
                slide(1);
            }
        }
        if constexpr (Ring::kOn) copy_wait<0>();
    }
    if (!a.parts) return;
    const int tid = (int)(threadIdx.y * kConvLanes + threadIdx.x);
#pragma unroll
    for (int i = 0; i <= W; ++i) {
        __syncthreads();
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
            const float2 v = i < W ? dw[i < W ? i : 0].v[k / 2] : db.v[k / 2];
            red[threadIdx.y][threadIdx.x * VEC + k] = k & 1 ? v.y : v.x;
        }
        __syncthreads();
        for (int l = tid; l < LANES; l += kConvThreads) {
            const int64_t chan = ct * LANES + l;
            if (chan < a.d.channels) {
                float v = 0.f;
#pragma unroll
                for (int y = 0; y < kConvRuns; ++y) v += red[y][l];
                a.parts[(tile * (W + 1) + i) * a.d.channels + chan] = v;
            }
        }
    }
}

template <class T, int VEC, int W>
cudaError_t conv_launch(ConvArgs a, bool backward, cudaStream_t s) {
    const int64_t rows = a.d.offsets ? 1 : a.d.nseq;
    a.ctiles = (a.d.channels + kConvLanes * VEC - 1) / (kConvLanes * VEC);
    a.run = conv_run_tokens(a.d, backward);
    a.ttiles = (a.d.length + kConvRuns * a.run - 1) / (kConvRuns * a.run);
    const bool states = W > 1 && (backward ? a.dinitial : a.final_state) != nullptr;
    const int64_t blocks = a.ctiles * (rows * a.ttiles + (states ? a.d.nseq : 0));
    if (blocks < 1) return cudaSuccess;
    if (blocks > INT32_MAX) return cudaErrorInvalidValue;
    const dim3 threads(kConvLanes, kConvRuns);
    if (backward) {
        constexpr int bytes = ConvRing<T, VEC, 2>::kBytes;
        static LaunchCache cache;
        LaunchGeom geo;
        const cudaError_t e = cache.get([](int dev, LaunchGeom* g) {
            return setup_persistent(k_conv_bwd<T, VEC, W>, kConvThreads, bytes, dev, g);
        }, &geo);
        if (e != cudaSuccess) return e;
        k_conv_bwd<T, VEC, W><<<(unsigned)blocks, threads, bytes, s>>>(a);
    } else {
        constexpr int bytes = ConvRing<T, VEC, 1>::kBytes;
        k_conv_fwd<T, VEC, W><<<(unsigned)blocks, threads, bytes, s>>>(a);
    }
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
