// Selective state-space scan, backward (fft_scan_backward).
//
// With y[t] = C[t] h[t] + D u[t], out = y silu(z) and dy = dout silu(z), the gradient at the state
//   q[t] = dy[t] C[t] + a[t+1] q[t+1],  a[t] = exp(d[t] A)
// runs from the last token to the first, and
//   dC = sum_c dy h      dB = sum_c q d u      du = d sum_s q B + dy D      dz = dout y silu'(z)
//   dd = u sum_s q B + sum_s q a h[t-1] A      dA = sum_t q a h[t-1] d      dD = sum_t dy u
//
// The states are not kept by the forward call: the forward passes run again and write the state
// before every 16th token.  Time is cut into chunks as in the forward scan; the gradient that a
// chunk sends back, m = a[t0] q[t0], is m_local + exp(A sum d) m_in, so one pass computes m_local,
// one runs along the chunks, and the main kernel walks each chunk from behind, 16 tokens at a
// time: what a token needs once per channel is prepared for the tile (the next tile's copies are
// then on their way), then forward over the tile (start states of its 4-token pieces to shared
// memory), then piece by piece backwards with the piece's states in registers.
//
// Main kernel: a thread holds 4 channels x 4 states, so the sums over states (for du, dd and y)
// and over channels (for dB and dC) are mostly within the thread; what crosses lanes is summed
// with the values handed out to the lanes (each step halves what a lane carries).  Channel tiles
// leave partial dB and dC, and chunks partial dA, dD, ddelta_bias, added up in a fixed order.
//
// Measured, 4 sequences of 2048 tokens, 2048 bfloat16 channels, 16 states, gated: 666 us, of which
// the main kernel 390 (1.9 instructions a cycle at the 8 warps of an SM that 250 registers and 92
// KB of shared memory allow; about 415 instructions per token and 32 channels), the pass from
// behind 90, the forward passes 59 and 70, the rest sums and carries.  Keeping questions about
// sequence ends out of whole tiles took the main kernel from 614 to 385 us.
#pragma once

#include "scan.cuh"
#include "scan_bwd.h"

namespace gbfft {

// The gradient that a chunk sends back, with nothing entering from behind: the tokens in reverse,
//   m <- a[t] (dy[t] C[t] + m).
// Up to 16 states: two channels per thread, built like the forward kernel k_scan.
template <class T, int SPT, bool FAST>
__global__ void __launch_bounds__(kPairThreads) k_scan_back_pair(const ScanBwdArgs a) {
    constexpr int NT = kPairThreads, CT = kPairChannels, TK = kPairTile, ST = 3, RAW = TK * CT;
    extern __shared__ float4 smem4[];
    T* raw = reinterpret_cast<T*>(smem4);  // [stage][delta, dout, z][token][channel]
    float* sc = reinterpret_cast<float*>(raw + ST * 3 * RAW);  // [buffer][token][state]
    const int n = (int)a.d.states, tid = (int)threadIdx.x;
    const bool packed = a.d.offsets != nullptr, gate = a.d.z.data != nullptr;
    // chunk 0 sends nothing on: blocks are the chunks 1 ...
    ScanBlock blk = scan_block(a.f, blockIdx.x, a.f.nchunks - 1, CT);
    blk.chunk += 1;
    blk.t0 += a.f.chunk;
    blk.t1 = blk.t0 + a.f.chunk < a.d.length ? blk.t0 + a.f.chunk : a.d.length;
    const int width = (int)(blk.cend - blk.c0 < CT ? blk.cend - blk.c0 : CT);
    const int lc = 2 * tid, len = (int)(blk.t1 - blk.t0);
    const int64_t c = blk.c0 + lc;
    const bool live[2] = {lc < width, lc + 1 < width};
    // tokens count from t0; tiles lie at multiples of TK, the last one may be short
    const T* src[3] = {row_of<T>(a.d.delta, packed, blk.row) + blk.t0 * a.d.delta.tok_stride + blk.c0,
                       row_of<T>(a.g.dout, packed, blk.row) + blk.t0 * a.g.dout.tok_stride + blk.c0,
                       gate ? row_of<T>(a.d.z, packed, blk.row) + blk.t0 * a.d.z.tok_stride + blk.c0
                            : nullptr};
    const int64_t str[3] = {a.d.delta.tok_stride, a.g.dout.tok_stride, a.d.z.tok_stride};
    const T* Cp = row_of<T>(a.d.C, packed, blk.row) + blk.t0 * a.d.C.tok_stride + blk.g * n;
    auto copy = [&](int t, int stage) {
        if (t >= 0) {
#pragma unroll
            for (int k = 0; k < 3; ++k) {
                if (k == 2 && !gate) break;
                copy_tile<T, TK, CT, NT, FAST>(raw + (stage * 3 + k) * RAW, src[k], str[k], t, len, width,
                                         a.f.vec);
            }
        }
        copy_commit();
    };
    RowsAhead<T, TK, SPT, NT, false, FAST> rows;
    auto fetch = [&](int t) { rows.fetch(Cp, a.d.C.tok_stride, Cp, 0, t, len, n); };
    auto stage_c = [&](int buf) { rows.stage(sc + buf * TK * SPT); };
    const int first = (len - 1) / TK * TK;
#pragma unroll
    for (int i = 0; i < ST - 1; ++i) copy(first - i * TK, i);
    fetch(first);
    float2 A2[2][SPT / 2], m[2][SPT / 2], bias = splat(0.f);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        load_states<SPT>(live[k] ? a.d.A + (c + k) * n : nullptr, 0, n, A2[k]);
        load_states<SPT>(nullptr, 0, n, m[k]);
#pragma unroll
        for (int i = 0; i < SPT / 2; ++i) A2[k][i] = mul2(A2[k][i], splat(kLog2e));
        if (live[k] && a.d.delta_bias) (k ? bias.y : bias.x) = a.d.delta_bias[c + k];
    }
    stage_c(0);
    fetch(first - TK);
    SeqAt sq = seq_at(a.d.offsets, a.d.nseq, a.d.length, blk.row, blk.t1 - 1);
    int stage = 0, buf = 0;
    for (int t = first; t >= 0; t -= TK) {
        copy_wait<ST - 2>();
        __syncthreads();  // this tile has landed; the last one's buffers are free
        copy(t - (ST - 1) * TK, stage >= 1 ? stage - 1 : ST - 1);
        stage_c(buf ^ 1);
        fetch(t - 2 * TK);
        const T* rd = raw + stage * 3 * RAW + lc;
        const T* ro = rd + RAW;
        const T* rz = ro + RAW;
        const float* sC = sc + buf * TK * SPT;
        const int tl = len - t < TK ? len - t : TK;
        // d and dy of all tokens, then the recurrence
        float2 d[TK], dy[TK];
#pragma unroll
        for (int j = 0; j < TK; ++j) {
            const Pack<T, 2> pd = ld_pack<2>(rd + j * CT), po = ld_pack<2>(ro + j * CT);
            d[j] = add2(make_float2(to_f(pd.v[0]), to_f(pd.v[1])), bias);
            dy[j] = make_float2(to_f(po.v[0]), to_f(po.v[1]));
            if (a.d.softplus) d[j] = softplus2(d[j]);
            if (gate) {
                const Pack<T, 2> pz = ld_pack<2>(rz + j * CT);
                const float2 z = make_float2(to_f(pz.v[0]), to_f(pz.v[1]));
                dy[j] = mul2(dy[j], mul2(z, sigmoid2(z)));
            }
        }
        const int64_t at = blk.t0 + t;
        const bool inside = at > sq.begin && at + tl < sq.end && tl == TK;
#pragma unroll
        for (int j = TK - 1; j >= 0; --j) {
            bool start = false;
            if (!inside) {
                if (j >= tl) continue;
                while (packed && sq.q > 0 && at + j < sq.begin) {
                    sq.q -= 1;
                    sq.end = sq.begin;
                    sq.begin = a.d.offsets[sq.q];
                }
                start = at + j == sq.begin;
                if (at + j + 1 == sq.end) {
#pragma unroll
                    for (int k = 0; k < 2; ++k)
                        load_states<SPT>(live[k] && a.g.dfinal_state
                                             ? a.g.dfinal_state + (sq.q * a.d.channels + c + k) * n
                                             : nullptr, 0, n, m[k]);
                }
            }
            const float2 dd[2] = {splat(d[j].x), splat(d[j].y)};
            const float2 yy[2] = {splat(dy[j].x), splat(dy[j].y)};
#pragma unroll
            for (int i = 0; i < SPT / 4; ++i) {
                const float4 c4 = *reinterpret_cast<const float4*>(sC + j * SPT + 4 * i);
#pragma unroll
                for (int p = 0; p < 2; ++p)
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        float2& mm = m[k][2 * i + p];
                        const float2 q = fma2(yy[k], p ? make_float2(c4.z, c4.w) : make_float2(c4.x, c4.y), mm);
                        mm = mul2(decay2(dd[k], A2[k][2 * i + p]), q);
                    }
            }
            if (start) {
#pragma unroll
                for (int k = 0; k < 2; ++k) load_states<SPT>(nullptr, 0, n, m[k]);
            }
        }
        stage = stage + 1 < ST ? stage + 1 : 0;
        buf ^= 1;
    }
    copy_wait<0>();
#pragma unroll
    for (int k = 0; k < 2; ++k)
        if (live[k])
            store_row<SPT>(a.carry + ((blk.row * a.f.nchunks + blk.chunk) * a.d.channels + c + k) * SPT, m[k]);
}

// More states: several lanes per channel, 16 states each.
template <class T, int SPT, int SL>
__global__ void __launch_bounds__(kScanThreads) k_scan_back(const ScanBwdArgs a) {
    constexpr int NP = SPT * SL, CT = kScanThreads / SL, TK = 8, OWN = TK / SL;
    constexpr int CL = 32 / SL;
    constexpr int CN = (TK * NP + kScanThreads - 1) / kScanThreads;
    __shared__ alignas(16) float sC[TK][NP];
    const int n = (int)a.d.states, tid = (int)threadIdx.x, lane = tid & 31;
    const bool packed = a.d.offsets != nullptr, gate = a.d.z.data != nullptr;
    // chunk 0 sends nothing on: blocks are the chunks 1 ...
    ScanArgs f = a.f;
    f.ctiles = a.back_ctiles;
    ScanBlock blk = scan_block(f, blockIdx.x, a.f.nchunks - 1, CT);
    blk.chunk += 1;
    blk.t0 += a.f.chunk;
    blk.t1 = blk.t0 + a.f.chunk < a.d.length ? blk.t0 + a.f.chunk : a.d.length;
    const int sl = lane / CL, s0 = sl * SPT;
    const int64_t c = blk.c0 + (tid >> 5) * CL + lane % CL;
    const bool live = c < blk.cend;
    const T* dl = row_of<T>(a.d.delta, packed, blk.row) + c;
    const T* z = row_of<T>(a.d.z, packed, blk.row) + c;
    const T* dout = row_of<T>(a.g.dout, packed, blk.row) + c;
    const T* Cp = row_of<T>(a.d.C, packed, blk.row) + blk.g * n;
    const float bias = live && a.d.delta_bias ? a.d.delta_bias[c] : 0.f;
    float2 A2[SPT / 2], m[SPT / 2];
    load_states<SPT>(live ? a.d.A + c * n : nullptr, s0, n, A2);
    load_states<SPT>(nullptr, s0, n, m);
#pragma unroll
    for (int i = 0; i < SPT / 2; ++i) A2[i] = mul2(A2[i], make_float2(kLog2e, kLog2e));
    // the sequence of the token at hand; packed rows walk down through the offsets
    SeqAt sq = seq_at(a.d.offsets, a.d.nseq, a.d.length, blk.row, blk.t1 - 1);
    for (int64_t t = blk.t1 - TK; t > blk.t0 - TK; t -= TK) {  // tile [t, t + TK), from behind
        __syncthreads();
#pragma unroll
        for (int i = 0; i < CN; ++i) {
            const int k = tid + i * kScanThreads;
            const int64_t tt = t + k / NP;
            if (k < TK * NP)
                (&sC[0][0])[k] =
                    tt >= blk.t0 && k % NP < n ? to_f(Cp[tt * a.d.C.tok_stride + k % NP]) : 0.f;
        }
        float od[OWN], oy[OWN];
#pragma unroll
        for (int j = 0; j < OWN; ++j) {
            const int64_t tt = t + sl * OWN + j;
            od[j] = oy[j] = 0.f;
            if (live && tt >= blk.t0) {
                const float e = to_f(dl[tt * a.d.delta.tok_stride]) + bias;
                od[j] = a.d.softplus ? softplus(e) : e;
                oy[j] = to_f(dout[tt * a.g.dout.tok_stride]);
                if (gate) {
                    const float zz = to_f(z[tt * a.d.z.tok_stride]);
                    oy[j] *= zz * sigmoid(zz);
                }
            }
        }
        __syncthreads();
#pragma unroll
        for (int j = TK - 1; j >= 0; --j) {
            if (t + j < blk.t0) break;
            if (packed && t + j < sq.begin) {
                while (sq.q > 0 && t + j < sq.begin) {
                    sq.q -= 1;
                    sq.end = sq.begin;
                    sq.begin = a.d.offsets[sq.q];
                }
            }
            if (t + j + 1 == sq.end)
                load_states<SPT>(live && a.g.dfinal_state
                                     ? a.g.dfinal_state + (sq.q * a.d.channels + c) * n : nullptr,
                                 s0, n, m);
            float d = od[j % OWN], dy = oy[j % OWN];
            if (SL > 1) {
                d = __shfl_sync(0xffffffffu, d, (j / OWN) * CL + lane % CL);
                dy = __shfl_sync(0xffffffffu, dy, (j / OWN) * CL + lane % CL);
            }
            const float2 dd = make_float2(d, d), yy = make_float2(dy, dy);
            const bool start = t + j == sq.begin;
#pragma unroll
            for (int i = 0; i < SPT / 2; ++i) {
                const float2 q = fma2(yy, *reinterpret_cast<const float2*>(&sC[j][s0 + 2 * i]), m[i]);
                m[i] = mul2(decay2(dd, A2[i]), q);
                if (start) m[i] = make_float2(0.f, 0.f);
            }
        }
    }
    if (live)
        store_states<SPT>(a.carry + ((blk.row * a.f.nchunks + blk.chunk) * a.d.channels + c) * NP, s0,
                          NP, m);
}

// From the last chunk to the first: the gradient that enters every chunk from behind.
template <int NP>
__global__ void __launch_bounds__(kCarryThreads) k_scan_back_carry(const ScanBwdArgs a) {
    const int64_t i = (int64_t)blockIdx.x * kCarryThreads + threadIdx.x, per = a.d.channels * NP;
    if (i >= a.f.rows * per) return;
    const int64_t row = i / per, cs = i - row * per, c = cs / NP, nch = a.f.nchunks;
    const int s = (int)(cs - c * NP), n = (int)a.d.states;
    const float A2 = s < n ? a.d.A[c * n + s] * kLog2e : 0.f;
    float* carry = a.carry + row * nch * per + cs;
    const float* dsum = a.f.dsum + row * nch * a.d.channels + c;
    const int* reset = a.f.reset + row * nch;
    float m = 0.f;
    constexpr int U = kCarryAhead;
    for (int64_t k = nch - 1; k >= 0; k -= U) {
        float local[U], sum[U];
        int cut[U];
#pragma unroll
        for (int j = 0; j < U; ++j) {
            const int64_t i = k - j > 0 ? k - j : 0;
            local[j] = carry[i * per];
            sum[j] = dsum[i * a.d.channels];
            // nothing enters the last chunk, and its sum of d is not known
            cut[j] = reset[i] || i == nch - 1;
        }
#pragma unroll
        for (int j = 0; j < U; ++j) sum[j] = ex2(0.5f * A2 * sum[j]);
#pragma unroll
        for (int j = 0; j < U; ++j) {
            if (k - j < 0) break;
            carry[(k - j) * per] = m;
            m = carried(sum[j], m, local[j], cut[j]);
        }
    }
}

template <class T, int SL>
struct BwdShape {
    static constexpr int NW = SL < 4 ? SL : 4, NT = NW * 32, CL = 32 / SL, CW = CL * 4;
    static constexpr int CT = NW * CW, NP = SL * 4;
    static constexpr int TK = kScanTile, TS = 4, PIECES = TK / TS;
    // dB and dC of a token: after one step over channel lanes a lane carries KV of the 8 values
    static constexpr int KV = CL > 1 ? 4 : 8, RS = SL < 32 ? 32 + SL : 32;
    // shared memory, in floats
    static constexpr int kRaw = TK * CT;                         // values of one tensor's tile
    static constexpr int kIn = TK * CT;                          // d, u, dy, and two factors
    static constexpr int kBC = TK * NP * 2;                      // B, C, each value twice
    static constexpr int kStart = (PIECES - 1) * 4 * NT * 4;     // start states of later pieces
    static constexpr int kRed = TS * NW * KV * RS;               // dB, dC of a piece
    static constexpr int kFloats = 5 * kIn + 2 * kBC + kStart + kRed;
    static constexpr int kBytes = kFloats * 4 + 4 * kRaw * (int)sizeof(T) + TK * 8 + 16;
};

// FAST: n == 4 * SL, so that no state beyond n has to be kept at 0 where u is infinite, and rows on
// 16-byte boundaries.
template <class T, int SL, bool FAST>
__global__ void __launch_bounds__(BwdShape<T, SL>::NT) k_scan_bwd(const ScanBwdArgs a) {
    using S = BwdShape<T, SL>;
    constexpr int NT = S::NT, CL = S::CL, CT = S::CT, NP = S::NP, TK = S::TK, TS = S::TS;
    constexpr int KV = S::KV, RS = S::RS;
    constexpr int OWN = SL == 1 ? 4 : (SL == 2 ? 2 : 1);  // channels that a lane owns
    extern __shared__ float4 smem4[];
    float* sd = reinterpret_cast<float*>(smem4);  // d
    float* su = sd + S::kIn;                      // u
    float* sy = su + S::kIn;                      // dy = dout silu(z)
    float* sf = sy + S::kIn;                      // dout silu'(z): dz = sf y
    float* sg = sf + S::kIn;                      // derivative of d by delta
    float* sB = sg + S::kIn;
    float* sC = sB + S::kBC;
    float4* sh = reinterpret_cast<float4*>(sC + S::kBC);  // [piece - 1][channel][thread]
    float* red = reinterpret_cast<float*>(sh) + S::kStart;
    T* raw = reinterpret_cast<T*>(red + S::kRed);  // [tensor][token][channel]
    int64_t* sq_id = reinterpret_cast<int64_t*>(raw + 4 * S::kRaw);  // [TK]
    unsigned* sq_mask = reinterpret_cast<unsigned*>(sq_id + TK);     // tokens that start, that end

    const int n = (int)a.d.states, tid = (int)threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const bool packed = a.d.offsets != nullptr, gate = a.d.z.data != nullptr;
    const int64_t tiles = a.ctiles * a.d.groups, dg = a.d.channels / a.d.groups;
    const int64_t tile = blockIdx.x % tiles, rest = blockIdx.x / tiles;
    const int64_t chunk = rest % a.f.nchunks, row = rest / a.f.nchunks;
    const int64_t g = tile / a.ctiles, ct = tile - g * a.ctiles;
    const int64_t c0 = g * dg + ct * CT, cend = (g + 1) * dg;
    const int width = (int)(cend - c0 < CT ? cend - c0 : CT);
    const int64_t t0 = chunk * a.f.chunk;
    const int64_t t1 = t0 + a.f.chunk < a.d.length ? t0 + a.f.chunk : a.d.length;
    const int sl = lane % SL, cl = lane / SL, s0 = sl * 4;
    const int lc = warp * S::CW + cl * 4;  // the thread's first channel in the block
    // channels that this lane owns after sums over states: lo .. lo + OWN - 1
    const int lo = lc + (SL == 1 ? 0 : (SL == 2 ? sl * 2 : (sl & 3)));
    const bool owner = SL <= 4 || sl < 4;

    const T* src[4] = {row_of<T>(a.d.u, packed, row) + c0, row_of<T>(a.d.delta, packed, row) + c0,
                       row_of<T>(a.g.dout, packed, row) + c0,
                       gate ? row_of<T>(a.d.z, packed, row) + c0 : nullptr};
    const int64_t str[4] = {a.d.u.tok_stride, a.d.delta.tok_stride, a.g.dout.tok_stride,
                            a.d.z.tok_stride};
    const T* Bp = row_of<T>(a.d.B, packed, row) + g * n;
    const T* Cp = row_of<T>(a.d.C, packed, row) + g * n;
    T* du = const_cast<T*>(row_of<T>(a.g.du, packed, row)) + c0 + lo;
    T* ddl = const_cast<T*>(row_of<T>(a.g.ddelta, packed, row)) + c0 + lo;
    T* dz = const_cast<T*>(row_of<T>(a.g.dz, packed, row)) + c0 + lo;

    auto copy = [&](int64_t tl) {  // the tile at tl; zeros outside the chunk
        if (tl < t0) return;
        const int len = t1 - tl < TK ? (int)(t1 - tl) : TK;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (k == 3 && !gate) break;
            copy_tile<T, TK, CT, NT, FAST>(raw + k * S::kRaw, src[k] + tl * str[k], str[k], 0, len, width,
                                     a.f.vec);
        }
        copy_commit();
    };

    // pairs over channels: [state][channel pair]
    float2 A2[4][2], m[4][2], dA[4][2];
    auto load4 = [&](const float* base, int64_t np, float2(&v)[4][2]) {  // [channels][np] rows
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t c = c0 + lc + i;
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const float x = base && c < cend && s0 + s < np ? base[c * np + s0 + s] : 0.f;
                (i & 1 ? v[s][i / 2].y : v[s][i / 2].x) = x;
            }
        }
    };
    auto load_padded = [&](const float* base, float2(&v)[4][2]) {  // rows of NP, 16-byte aligned
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t c = c0 + lc + i;
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            if (c < cend) x = *reinterpret_cast<const float4*>(base + c * NP + s0);
            (i & 1 ? v[0][i / 2].y : v[0][i / 2].x) = x.x;
            (i & 1 ? v[1][i / 2].y : v[1][i / 2].x) = x.y;
            (i & 1 ? v[2][i / 2].y : v[2][i / 2].x) = x.z;
            (i & 1 ? v[3][i / 2].y : v[3][i / 2].x) = x.w;
        }
    };
    auto put = [&](int piece, const float2(&v)[4][2]) {  // a thread's own places
        float4* p = sh + (piece - 1) * 4 * NT + tid;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            p[2 * i * NT] = make_float4(v[0][i].x, v[1][i].x, v[2][i].x, v[3][i].x);
            p[(2 * i + 1) * NT] = make_float4(v[0][i].y, v[1][i].y, v[2][i].y, v[3][i].y);
        }
    };
    auto get = [&](int piece, float2(&v)[4][2]) {
        const float4* p = sh + (piece - 1) * 4 * NT + tid;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float4 x = p[2 * i * NT], y = p[(2 * i + 1) * NT];
            v[0][i] = make_float2(x.x, y.x);
            v[1][i] = make_float2(x.y, y.y);
            v[2][i] = make_float2(x.z, y.z);
            v[3][i] = make_float2(x.w, y.w);
        }
    };
    auto initial = [&](int j, float2(&v)[4][2]) {
        load4(a.d.initial_state ? a.d.initial_state + sq_id[j] * a.d.channels * n : nullptr, n, v);
    };
    const int64_t last_tile = (t1 - 1) / TK * TK, ntiles = (a.d.length + TK - 1) / TK;
    copy(last_tile);
    load4(a.d.A, n, A2);
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            A2[s][p] = mul2(A2[s][p], splat(kLog2e));
            dA[s][p] = m[s][p] = splat(0.f);
        }
    if (a.f.nchunks > 1)
        load_padded(a.carry + (row * a.f.nchunks + chunk) * a.d.channels * NP, m);
    float oD[OWN], aD[OWN] = {}, abias[OWN] = {};
#pragma unroll
    for (int k = 0; k < OWN; ++k) oD[k] = lo + k < width && a.d.D ? a.d.D[c0 + lo + k] : 0.f;
    // the pairs of channels that this thread prepares: one where the block has as many threads
    constexpr int HALF = CT / 2;
    auto bias_of = [&](int pc) {
        float2 v = splat(0.f);
        if (a.d.delta_bias) {
            if (pc < width) v.x = a.d.delta_bias[c0 + pc];
            if (pc + 1 < width) v.y = a.d.delta_bias[c0 + pc + 1];
        }
        return v;
    };
    const float2 own_bias = bias_of(2 * (tid % HALF));
    SeqAt cur = seq_at(a.d.offsets, a.d.nseq, a.d.length, row, t1 - 1);
    auto down_to = [&](int64_t t, SeqAt& s) {  // packed: the sequence that holds an earlier token
        while (s.q > 0 && t < s.begin) {
            s.q -= 1;
            s.end = s.begin;
            s.begin = a.d.offsets[s.q];
        }
    };

    // the sums over tokens go to partial row k and start anew
    auto leave = [&](int64_t k) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                float& v = i & 1 ? dA[s][i / 2].y : dA[s][i / 2].x;
                if (lc + i < width && s0 + s < n)
                    a.pA[(k * a.d.channels + c0 + lc + i) * n + s0 + s] = v;
                v = 0.f;
            }
#pragma unroll
        for (int i = 0; i < OWN; ++i) {
            if (owner && lo + i < width) {
                a.pD[k * a.d.channels + c0 + lo + i] = aD[i];
                a.pbias[k * a.d.channels + c0 + lo + i] = abias[i];
            }
            aD[i] = abias[i] = 0.f;
        }
    };

    for (int64_t tl = last_tile; tl >= t0; tl -= TK) {
        const int len = t1 - tl < TK ? (int)(t1 - tl) : TK;
        copy_wait<0>();
        __syncthreads();  // the tile has landed; the last one's shared memory is free
        if (packed) down_to(tl + len - 1, cur);
        if (warp == 0) {
            SeqAt s = cur;
            bool start = false, end = false;
            if (lane < len) {
                if (packed) down_to(tl + lane, s);
                sq_id[lane] = s.q;
                start = tl + lane == s.begin;
                end = tl + lane + 1 == s.end;
            }
            const unsigned starts = __ballot_sync(0xffffffffu, start);
            const unsigned ends = __ballot_sync(0xffffffffu, end);
            if (lane == 0) {
                sq_mask[0] = starts;
                sq_mask[1] = ends;
            }
        }
#pragma unroll 2
        for (int i = tid; i < TK * HALF; i += NT) {
            const int j = i / HALF, pc = 2 * (i - j * HALF), e = j * CT + pc;
            const float2 bias = NT >= HALF ? own_bias : bias_of(pc);
            const Pack<T, 2> pu = ld_pack<2>(raw + e), pd = ld_pack<2>(raw + S::kRaw + e);
            const Pack<T, 2> po = ld_pack<2>(raw + 2 * S::kRaw + e);
            float2 d = add2(make_float2(to_f(pd.v[0]), to_f(pd.v[1])), bias), slope = splat(1.f);
            if (a.d.softplus) {
                slope = sigmoid2(d);
                d = softplus2(d);
            }
            float2 dy = make_float2(to_f(po.v[0]), to_f(po.v[1])), f = dy;
            if (gate) {
                const Pack<T, 2> pz = ld_pack<2>(raw + 3 * S::kRaw + e);
                const float2 z = make_float2(to_f(pz.v[0]), to_f(pz.v[1])), s = sigmoid2(z);
                f = mul2(dy, mul2(s, fma2(z, fma2(s, splat(-1.f), splat(1.f)), splat(1.f))));
                dy = mul2(dy, mul2(z, s));
            }
            *reinterpret_cast<float2*>(sd + e) = d;
            *reinterpret_cast<float2*>(su + e) = make_float2(to_f(pu.v[0]), to_f(pu.v[1]));
            *reinterpret_cast<float2*>(sy + e) = dy;
            *reinterpret_cast<float2*>(sf + e) = f;
            *reinterpret_cast<float2*>(sg + e) = slope;
        }
        for (int i = tid; i < TK * NP; i += NT) {
            const int j = i / NP, s = i - j * NP;
            const bool in = j < len && s < n;
            const float b = in ? to_f(Bp[(tl + j) * a.d.B.tok_stride + s]) : 0.f;
            const float c = in ? to_f(Cp[(tl + j) * a.d.C.tok_stride + s]) : 0.f;
            *reinterpret_cast<float2*>(sB + 2 * i) = splat(b);
            *reinterpret_cast<float2*>(sC + 2 * i) = splat(c);
        }
        const float* start_states = a.f.tiles + (row * ntiles + tl / TK) * a.d.channels * NP;
        float2 h[4][2];
        load_padded(start_states, h);
        __syncthreads();
        copy(tl - TK);
        const unsigned starts = sq_mask[0], ends = sq_mask[1];
        T* pdu = du + tl * a.g.du.tok_stride;
        T* pdd = ddl + tl * a.g.ddelta.tok_stride;
        T* pdz = dz + tl * a.g.dz.tok_stride;
        const int sdu = (int)a.g.du.tok_stride, sdd = (int)a.g.ddelta.tok_stride;
        const int sdz = (int)a.g.dz.tok_stride;

        auto step = [&](int j) {  // h of token j from h of the token before
            const float4 d4 = *reinterpret_cast<const float4*>(sd + j * CT + lc);
            const float4 u4 = *reinterpret_cast<const float4*>(su + j * CT + lc);
            const float2 dd[2] = {make_float2(d4.x, d4.y), make_float2(d4.z, d4.w)};
            const float2 du2[2] = {mul2(dd[0], make_float2(u4.x, u4.y)),
                                   mul2(dd[1], make_float2(u4.z, u4.w))};
#pragma unroll
            for (int s = 0; s < 4; s += 2) {
                const float4 b4 = *reinterpret_cast<const float4*>(sB + (j * NP + s0 + s) * 2);
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const float2 b = k ? make_float2(b4.z, b4.w) : make_float2(b4.x, b4.y);
#pragma unroll
                    for (int p = 0; p < 2; ++p) {
                        h[s + k][p] = fma2(decay2(dd[p], A2[s + k][p]), h[s + k][p], mul2(du2[p], b));
                        if (!FAST && s0 + s + k >= n) h[s + k][p] = splat(0.f);
                    }
                }
            }
        };
        // a tile inside one sequence, and whole, takes code without questions
        auto walk = [&](auto plain) {
            constexpr bool PLAIN = decltype(plain)::value != 0;
            const int last = PLAIN ? S::PIECES - 1 : (len - 1) / TS;
            for (int piece = 0; piece < last; ++piece) {
#pragma unroll
                for (int j = 0; j < TS; ++j) {
                    if (!PLAIN && starts >> (piece * TS + j) & 1) initial(piece * TS + j, h);
                    step(piece * TS + j);
                }
                put(piece + 1, h);
            }
            for (int piece = last; piece >= 0; --piece) {
                float2 hist[TS + 1][4][2];  // the states before the piece and after its tokens
                if (piece < last) {
                    if (piece > 0)
                        get(piece, h);
                    else
                        load_padded(start_states, h);
                }
#pragma unroll
                for (int j = 0; j <= TS; ++j) {
#pragma unroll
                    for (int s = 0; s < 4; ++s)
#pragma unroll
                        for (int p = 0; p < 2; ++p) hist[j][s][p] = h[s][p];
                    if (j < TS && (PLAIN || piece * TS + j < len)) {
                        if (!PLAIN && starts >> (piece * TS + j) & 1) initial(piece * TS + j, h);
                        step(piece * TS + j);
                    }
                }
#pragma unroll
                for (int jj = TS - 1; jj >= 0; --jj) {
                    const int j = piece * TS + jj;
                    if (!PLAIN && j >= len) continue;
                    if (!PLAIN && ends >> j & 1)
                        load4(a.g.dfinal_state ? a.g.dfinal_state + sq_id[j] * a.d.channels * n : nullptr,
                              n, m);
                    // before a sequence's first token stands its initial state; what stands there is
                    // also the state after the token before, kept in a place that is free by now
                    if (!PLAIN && starts >> j & 1) {
                        put(piece ? piece : 1, hist[jj]);
                        initial(j, hist[jj]);
                    }
                    const float4 d4 = *reinterpret_cast<const float4*>(sd + j * CT + lc);
                    const float4 u4 = *reinterpret_cast<const float4*>(su + j * CT + lc);
                    const float4 y4 = *reinterpret_cast<const float4*>(sy + j * CT + lc);
                    const float2 dd[2] = {make_float2(d4.x, d4.y), make_float2(d4.z, d4.w)};
                    const float2 dy[2] = {make_float2(y4.x, y4.y), make_float2(y4.z, y4.w)};
                    const float2 du2[2] = {mul2(dd[0], make_float2(u4.x, u4.y)),
                                           mul2(dd[1], make_float2(u4.z, u4.w))};
                    float2 yv[2] = {}, qb[2] = {}, qa[2] = {};
                    float bc[8];
#pragma unroll
                    for (int s = 0; s < 4; ++s) {
                        const float2 b = *reinterpret_cast<const float2*>(sB + (j * NP + s0 + s) * 2);
                        const float2 c = *reinterpret_cast<const float2*>(sC + (j * NP + s0 + s) * 2);
                        float2 db, dc;
#pragma unroll
                        for (int p = 0; p < 2; ++p) {
                            const float2 q = fma2(dy[p], c, m[s][p]);
                            const float2 aq = mul2(decay2(dd[p], A2[s][p]), q);
                            const float2 w = mul2(aq, hist[jj][s][p]);
                            yv[p] = fma2(c, hist[jj + 1][s][p], yv[p]);
                            qb[p] = fma2(q, b, qb[p]);
                            qa[p] = fma2(w, A2[s][p], qa[p]);
                            dA[s][p] = fma2(w, dd[p], dA[s][p]);
                            db = p ? fma2(q, du2[p], db) : mul2(q, du2[p]);
                            dc = p ? fma2(dy[p], hist[jj + 1][s][p], dc) : mul2(dy[p], hist[jj + 1][s][p]);
                            m[s][p] = aq;
                        }
                        bc[s] = db.x + db.y;
                        bc[4 + s] = dc.x + dc.y;
                    }
                    if (!PLAIN && starts >> j & 1) {  // the sequence's first token
                        if (a.g.dinitial_state) {
#pragma unroll
                            for (int i = 0; i < 4; ++i)
#pragma unroll
                                for (int s = 0; s < 4; ++s)
                                    if (lc + i < width && s0 + s < n)
                                        a.g.dinitial_state[(sq_id[j] * a.d.channels + c0 + lc + i) * n + s0 + s] =
                                            i & 1 ? m[s][i / 2].y : m[s][i / 2].x;
                        }
#pragma unroll
                        for (int s = 0; s < 4; ++s)
#pragma unroll
                            for (int p = 0; p < 2; ++p) m[s][p] = splat(0.f);
                        get(piece ? piece : 1, hist[jj]);
                    }
                    // sums over states, handed out to the lanes of a channel group
                    float vy[4] = {yv[0].x, yv[0].y, yv[1].x, yv[1].y};
                    float vb[4] = {qb[0].x, qb[0].y, qb[1].x, qb[1].y};
                    float va[4] = {qa[0].x, qa[0].y, qa[1].x, qa[1].y};
                    if constexpr (SL >= 4) {
                        hand_out<4, 2, 1>(vy, sl);
                        hand_out<4, 2, 1>(vb, sl);
                        hand_out<4, 2, 1>(va, sl);
#pragma unroll
                        for (int w = 4; w < SL; w *= 2) {
                            vy[0] += __shfl_xor_sync(0xffffffffu, vy[0], w);
                            vb[0] += __shfl_xor_sync(0xffffffffu, vb[0], w);
                            va[0] += __shfl_xor_sync(0xffffffffu, va[0], w);
                        }
                    } else if constexpr (SL == 2) {
                        hand_out<4, 1, 1>(vy, sl);
                        hand_out<4, 1, 1>(vb, sl);
                        hand_out<4, 1, 1>(va, sl);
                    }
#pragma unroll
                    for (int k = 0; k < OWN; ++k) {
                        const int e = j * CT + lo + k;
                        const float d = sd[e], uu = su[e], dyk = sy[e];
                        const float dv = fmaf(d, vb[k], dyk * oD[k]);
                        const float de = fmaf(uu, vb[k], va[k] * kLn2) * sg[e];  // A = A2 ln 2
                        abias[k] += de;
                        aD[k] = fmaf(dyk, uu, aD[k]);
                        if (owner && lo + k < width) {
                            pdu[(int64_t)j * sdu + k] = from_f<T>(dv);
                            pdd[(int64_t)j * sdd + k] = from_f<T>(de);
                            if (gate) pdz[(int64_t)j * sdz + k] = from_f<T>(sf[e] * fmaf(oD[k], uu, vy[k]));
                        }
                    }
                    // sums over channels: one step between lanes, the rest through shared memory
                    if constexpr (CL > 1) {
                        const bool up = cl & (CL / 2);
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const float send = up ? bc[k] : bc[k + 4], keep = up ? bc[k + 4] : bc[k];
                            bc[k] = keep + __shfl_xor_sync(0xffffffffu, send, CL / 2 * SL);
                        }
                    }
#pragma unroll
                    for (int k = 0; k < KV; ++k) red[((jj * S::NW + warp) * KV + k) * RS + lane] = bc[k];
                }
                __syncthreads();
                // the piece's dB and dC: value v (dB of 4 states, dC of 4 states) of state lane i
                const int plen = PLAIN || len - piece * TS > TS ? TS : len - piece * TS;
                for (int o = tid; o < plen * 8 * SL; o += NT) {
                    const int jj = o / (8 * SL), v = o / SL % 8, i = o % SL, state = i * 4 + (v & 3);
                    constexpr int LANES = CL > 1 ? CL / 2 : 1;
                    const float* p = red + (jj * S::NW * KV + (CL > 1 ? v & 3 : v)) * RS + i +
                                     (CL > 1 ? (v >> 2) * (CL / 2) * SL : 0);
                    float x = 0.f;
#pragma unroll
                    for (int w = 0; w < S::NW; ++w)
#pragma unroll
                        for (int k = 0; k < LANES; ++k) x += p[w * KV * RS + k * SL];
                    if (state < n) {
                        const int64_t t = tl + piece * TS + jj;
                        a.bc[((((ct * a.f.rows + row) * a.d.length + t) * a.d.groups + g) * 2 + (v >> 2)) * n +
                             state] = x;
                    }
                }
                if (piece) __syncthreads();  // the next piece writes the same places
            }
        };
        if (len == TK && !(starts | ends))
            walk(Count<1>{});
        else
            walk(Count<0>{});
        if ((tl - t0) % kScanPart == 0) leave(row * a.parts + chunk * a.cuts + (tl - t0) / kScanPart);
    }
    copy_wait<0>();
}

// dB and dC: the channel tiles' partial sums, added in order.
template <class T>
__global__ void __launch_bounds__(256) k_scan_bc(const ScanBwdArgs a) {
    const int64_t per = a.d.groups * a.d.states, all = a.f.rows * a.d.length * per;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= all) return;
    const int64_t n = a.d.states, tok = i / per, gs = i - tok * per, g = gs / n, s = gs - g * n;
    const float* p = a.bc + (tok * a.d.groups + g) * 2 * n + s;
    float b = 0.f, c = 0.f;
    for (int64_t k = 0; k < a.ctiles; ++k) {
        b += p[k * all * 2];
        c += p[k * all * 2 + n];
    }
    const int64_t row = tok / a.d.length, t = tok - row * a.d.length;
    const bool packed = a.d.offsets != nullptr;
    const_cast<T*>(row_of<T>(a.g.dB, packed, row))[t * a.g.dB.tok_stride + gs] = from_f<T>(b);
    const_cast<T*>(row_of<T>(a.g.dC, packed, row))[t * a.g.dC.tok_stride + gs] = from_f<T>(c);
}

// A sequence without tokens hands the gradient of its final state to its initial one.
template <class T>
__global__ void __launch_bounds__(256) k_scan_back_empty(const ScanBwdArgs a) {
    const int64_t q = blockIdx.x, per = a.d.channels * a.d.states;
    const bool empty = a.d.offsets ? a.d.offsets[q] >= a.d.offsets[q + 1] : a.d.length == 0;
    if (!empty) return;
    for (int64_t i = threadIdx.x; i < per; i += 256)
        a.g.dinitial_state[q * per + i] = a.g.dfinal_state ? a.g.dfinal_state[q * per + i] : 0.f;
}

template <class T, int SL, bool FAST>
cudaError_t scan_bwd_launch(const ScanBwdArgs& a, cudaStream_t s) {
    using S = BwdShape<T, SL>;
    static LaunchCache cache;
    LaunchGeom geo;
    cudaError_t e = cache.get([](int dev, LaunchGeom* g) {
        return setup_persistent(k_scan_bwd<T, SL, FAST>, S::NT, S::kBytes, dev, g);
    }, &geo);
    if (e != cudaSuccess) return e;
    const int64_t blocks = a.f.rows * a.f.nchunks * a.ctiles * a.d.groups;
    if (blocks > INT32_MAX) return cudaErrorInvalidValue;
    k_scan_bwd<T, SL, FAST><<<(unsigned)blocks, S::NT, S::kBytes, s>>>(a);
    return cudaGetLastError();
}
template <class T, int SL>
cudaError_t scan_bwd_main(const ScanBwdArgs& a, cudaStream_t s) {
    return a.d.states == 4 * SL && a.f.vec >= 16 ? scan_bwd_launch<T, SL, true>(a, s)
                                : scan_bwd_launch<T, SL, false>(a, s);
}
template <int NP>
cudaError_t scan_bwd_carry(const ScanBwdArgs& a, cudaStream_t s) {
    k_scan_back_carry<NP>
        <<<(unsigned)((a.f.rows * a.d.channels * NP + kCarryThreads - 1) / kCarryThreads),
           kCarryThreads, 0, s>>>(a);
    return cudaGetLastError();
}
template <class T, int SPT, bool FAST>
cudaError_t scan_bwd_pair_launch(const ScanBwdArgs& a, cudaStream_t s) {
    constexpr int bytes = 3 * 3 * kPairTile * kPairChannels * (int)sizeof(T) + 2 * kPairTile * SPT * 4;
    static LaunchCache cache;
    LaunchGeom geo;
    const cudaError_t e = cache.get([](int dev, LaunchGeom* g) {
        return setup_persistent(k_scan_back_pair<T, SPT, FAST>, kPairThreads, bytes, dev, g);
    }, &geo);
    if (e != cudaSuccess) return e;
    const int64_t blocks = a.f.rows * (a.f.nchunks - 1) * a.f.ctiles * a.d.groups;
    k_scan_back_pair<T, SPT, FAST><<<(unsigned)blocks, kPairThreads, bytes, s>>>(a);
    return scan_bwd_carry<SPT>(a, s);
}
template <class T, int SPT>
cudaError_t scan_bwd_back_pair(const ScanBwdArgs& a, cudaStream_t s) {
    if constexpr (whole_states<T>(SPT)) {
        if (a.d.states == SPT && a.f.vec >= 16 && a.f.wide) return scan_bwd_pair_launch<T, SPT, true>(a, s);
    }
    return scan_bwd_pair_launch<T, SPT, false>(a, s);
}
template <class T, int SPT, int SL>
cudaError_t scan_bwd_back(const ScanBwdArgs& a, cudaStream_t s) {
    k_scan_back<T, SPT, SL><<<(unsigned)(a.f.rows * (a.f.nchunks - 1) * a.back_ctiles * a.d.groups),
                              kScanThreads, 0, s>>>(a);
    return scan_bwd_carry<SPT * SL>(a, s);
}

template <class T>
cudaError_t scan_bwd_run(ScanBwdArgs a, cudaStream_t s) {
    cudaError_t e = cudaSuccess;
    auto rows_on = [&](const fft_seq& q, int64_t bytes) {
        return !q.data || (aligned_to(q.data, bytes) && q.tok_stride * sizeof(T) % bytes == 0 &&
                           (a.d.offsets || q.seq_stride * sizeof(T) % bytes == 0));
    };
    auto all_on = [&](int64_t bytes) {
        return a.d.channels / a.d.groups * sizeof(T) % bytes == 0 && rows_on(a.d.u, bytes) &&
               rows_on(a.d.delta, bytes) && rows_on(a.d.z, bytes) && rows_on(a.g.dout, bytes);
    };
    a.f.vec = all_on(16) ? 16 : (all_on(4) ? 4 : 0);
    a.f.wide = rows_on(a.d.B, 16) && rows_on(a.d.C, 16) && a.d.states * sizeof(T) % 16 == 0;
    const int64_t n = a.d.states, parts = a.f.rows * a.parts;
    if (a.d.length > 0) {
        if (a.f.rows * a.f.nchunks * a.back_ctiles * a.d.groups > INT32_MAX) return cudaErrorInvalidValue;
        e = scan_run<T, SCAN_TILES>(a.f, s);
        if (e == cudaSuccess && a.f.nchunks > 1) {
            switch (scan_np(n)) {
                case 4: e = scan_bwd_back_pair<T, 4>(a, s); break;
                case 8: e = scan_bwd_back_pair<T, 8>(a, s); break;
                case 16: e = scan_bwd_back_pair<T, 16>(a, s); break;
                case 32: e = scan_bwd_back<T, 16, 2>(a, s); break;
                case 64: e = scan_bwd_back<T, 16, 4>(a, s); break;
                default: e = scan_bwd_back<T, 16, 8>(a, s); break;
            }
        }
        if (e != cudaSuccess) return e;
        switch (bwd_sl(n)) {
            case 1: e = scan_bwd_main<T, 1>(a, s); break;
            case 2: e = scan_bwd_main<T, 2>(a, s); break;
            case 4: e = scan_bwd_main<T, 4>(a, s); break;
            case 8: e = scan_bwd_main<T, 8>(a, s); break;
            case 16: e = scan_bwd_main<T, 16>(a, s); break;
            default: e = scan_bwd_main<T, 32>(a, s); break;
        }
        if (e != cudaSuccess) return e;
        const int64_t all = a.f.rows * a.d.length * a.d.groups * n;
        if ((all + 255) / 256 > INT32_MAX) return cudaErrorInvalidValue;
        k_scan_bc<T><<<(unsigned)((all + 255) / 256), 256, 0, s>>>(a);
    }
    if (a.g.dinitial_state && (a.d.offsets || a.d.length == 0))
        k_scan_back_empty<T><<<(unsigned)a.d.nseq, 256, 0, s>>>(a);
    e = cudaGetLastError();
    const int64_t np = a.d.length > 0 ? parts : 0, ch = a.d.channels;
    if (e == cudaSuccess && a.g.dA) e = run_sum_parts(a.pA, np, ch * n, ch * n, a.g.dA, ch * n, 1, s);
    if (e == cudaSuccess && a.g.dD) e = run_sum_parts(a.pD, np, ch, ch, a.g.dD, ch, 1, s);
    if (e == cudaSuccess && a.g.ddelta_bias)
        e = run_sum_parts(a.pbias, np, ch, ch, a.g.ddelta_bias, ch, 1, s);
    return e;
}

}  // namespace gbfft
