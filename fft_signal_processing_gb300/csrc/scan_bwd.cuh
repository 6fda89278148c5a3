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
// time: forward over the tile (start states of its 4-token pieces to shared memory), then
// piece by piece backwards with the piece's states in registers.
//
// Main kernel: a thread holds 4 channels x 4 states, so the sums over states (for du, dd and y)
// and over channels (for dB and dC) are mostly within the thread; what crosses lanes is summed
// with the values handed out to the lanes (each step halves what a lane carries).  Channel tiles
// leave partial dB and dC, and chunks partial dA, dD, ddelta_bias, added up in a fixed order.
#pragma once

#include "scan.cuh"
#include "scan_bwd.h"

namespace gbfft {

// The gradient that a chunk sends back, with nothing entering from behind.
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
                const float2 arg = mul2(dd, A2[i]);
                const float2 q = fma2(yy, *reinterpret_cast<const float2*>(&sC[j][s0 + 2 * i]), m[i]);
                m[i] = mul2(make_float2(ex2(arg.x), ex2(arg.y)), q);
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
        for (int j = 0; j < U; ++j) {
            if (k - j < 0) break;
            carry[(k - j) * per] = m;
            m = cut[j] ? local[j] : fmaf(ex2(A2 * sum[j]), m, local[j]);
        }
    }
}

template <int SL>
struct BwdShape {
    static constexpr int NW = SL < 4 ? SL : 4, NT = NW * 32, CL = 32 / SL, CW = CL * 4;
    static constexpr int CT = NW * CW, NP = SL * 4;
    static constexpr int TK = kScanTile, TS = 4, PIECES = TK / TS;
    // shared memory, in floats
    static constexpr int kIn = TK * CT;               // d, u, dy
    static constexpr int kBC = TK * NP * 2;           // B, C, each value twice
    static constexpr int kStart = PIECES * 4 * NT * 4;  // start states of the pieces
    static constexpr int kRed = NW * TS * 8 * SL;     // dB, dC of the warps, double buffered
    static constexpr int kFloats = 3 * kIn + 2 * kBC + kStart + 2 * kRed;
    static constexpr int kBytes = kFloats * 4 + TK * 16;
};

template <class T, int SL>
__global__ void __launch_bounds__(BwdShape<SL>::NT) k_scan_bwd(const ScanBwdArgs a) {
    using S = BwdShape<SL>;
    constexpr int NT = S::NT, CL = S::CL, CT = S::CT, NP = S::NP, TK = S::TK, TS = S::TS;
    constexpr int OWN = SL == 1 ? 4 : (SL == 2 ? 2 : 1);  // channels that a lane owns
    extern __shared__ float4 smem4[];
    float* sd = reinterpret_cast<float*>(smem4);
    float* su = sd + S::kIn;
    float* sy = su + S::kIn;
    float* sB = sy + S::kIn;
    float* sC = sB + S::kBC;
    float4* sh = reinterpret_cast<float4*>(sC + S::kBC);  // [piece][channel][thread]
    float* sred = reinterpret_cast<float*>(sh) + S::kStart;
    int64_t* sq_id = reinterpret_cast<int64_t*>(sred + 2 * S::kRed);  // [TK]
    int* sq_flag = reinterpret_cast<int*>(sq_id + TK);                // [TK] 1: start, 2: end

    const int n = (int)a.d.states, tid = (int)threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const bool packed = a.d.offsets != nullptr, gate = a.d.z.data != nullptr;
    const int64_t tiles = a.ctiles * a.d.groups, dg = a.d.channels / a.d.groups;
    const int64_t tile = blockIdx.x % tiles, rest = blockIdx.x / tiles;
    const int64_t chunk = rest % a.f.nchunks, row = rest / a.f.nchunks;
    const int64_t g = tile / a.ctiles, ct = tile - g * a.ctiles;
    const int64_t c0 = g * dg + ct * CT, cend = (g + 1) * dg;
    const int64_t t0 = chunk * a.f.chunk;
    const int64_t t1 = t0 + a.f.chunk < a.d.length ? t0 + a.f.chunk : a.d.length;
    const int sl = lane % SL, cl = lane / SL, s0 = sl * 4;
    const int lc = warp * S::CW + cl * 4;  // the thread's first channel in the block
    // channels that this lane owns after sums over states: lo .. lo + OWN - 1
    const int lo = lc + (SL == 1 ? 0 : (SL == 2 ? sl * 2 : (sl & 3)));
    const bool owner = SL <= 4 || sl < 4;

    const T* u = row_of<T>(a.d.u, packed, row);
    const T* dl = row_of<T>(a.d.delta, packed, row);
    const T* z = row_of<T>(a.d.z, packed, row);
    const T* dout = row_of<T>(a.g.dout, packed, row);
    const T* Bp = row_of<T>(a.d.B, packed, row) + g * n;
    const T* Cp = row_of<T>(a.d.C, packed, row) + g * n;
    T* du = const_cast<T*>(row_of<T>(a.g.du, packed, row));
    T* ddl = const_cast<T*>(row_of<T>(a.g.ddelta, packed, row));
    T* dz = const_cast<T*>(row_of<T>(a.g.dz, packed, row));

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
    auto put = [&](int piece, const float2(&v)[4][2]) {
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            sh[(piece * 4 + 2 * p) * NT + tid] = make_float4(v[0][p].x, v[1][p].x, v[2][p].x, v[3][p].x);
            sh[(piece * 4 + 2 * p + 1) * NT + tid] =
                make_float4(v[0][p].y, v[1][p].y, v[2][p].y, v[3][p].y);
        }
    };
    auto get = [&](int piece, float2(&v)[4][2]) {
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            const float4 x = sh[(piece * 4 + 2 * p) * NT + tid], y = sh[(piece * 4 + 2 * p + 1) * NT + tid];
            v[0][p] = make_float2(x.x, y.x);
            v[1][p] = make_float2(x.y, y.y);
            v[2][p] = make_float2(x.z, y.z);
            v[3][p] = make_float2(x.w, y.w);
        }
    };
    auto initial = [&](int j, float2(&v)[4][2]) {
        load4(a.d.initial_state ? a.d.initial_state + sq_id[j] * a.d.channels * n : nullptr, n, v);
    };
    load4(a.d.A, n, A2);
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            A2[s][p] = mul2(A2[s][p], make_float2(kLog2e, kLog2e));
            dA[s][p] = make_float2(0.f, 0.f);
            m[s][p] = make_float2(0.f, 0.f);
        }
    if (a.f.nchunks > 1)
        load_padded(a.carry + (row * a.f.nchunks + chunk) * a.d.channels * NP, m);
    float oD[OWN], obias[OWN], aD[OWN] = {}, abias[OWN] = {};
#pragma unroll
    for (int k = 0; k < OWN; ++k) {
        const int64_t c = c0 + lo + k;
        oD[k] = c < cend && a.d.D ? a.d.D[c] : 0.f;
        obias[k] = c < cend && a.d.delta_bias ? a.d.delta_bias[c] : 0.f;
    }
    const int64_t ntiles = (a.d.length + TK - 1) / TK;
    int rbuf = 0;

    for (int64_t tl = (t1 - 1) / TK * TK; tl >= t0; tl -= TK) {
        const int len = t1 - tl < TK ? (int)(t1 - tl) : TK;
        __syncthreads();  // the last tile's shared memory is free
        if (warp == 0) {
            SeqAt s = seq_at(a.d.offsets, a.d.nseq, a.d.length, row, tl);
            if (lane < len) {
                seq_next(a.d.offsets, a.d.nseq, tl + lane, &s);
                sq_id[lane] = s.q;
                sq_flag[lane] = (tl + lane == s.begin ? 1 : 0) | (tl + lane + 1 == s.end ? 2 : 0);
            }
        }
        for (int i = tid; i < TK * CT; i += NT) {
            const int j = i / CT, k = i - j * CT;
            const int64_t c = c0 + k, t = tl + j;
            float d = 0.f, uu = 0.f, dy = 0.f;
            if (j < len && c < cend) {
                d = to_f(dl[t * a.d.delta.tok_stride + c]);
                if (a.d.delta_bias) d += a.d.delta_bias[c];
                if (a.d.softplus) d = softplus(d);
                uu = to_f(u[t * a.d.u.tok_stride + c]);
                dy = to_f(dout[t * a.g.dout.tok_stride + c]);
                if (gate) {
                    const float zz = to_f(z[t * a.d.z.tok_stride + c]);
                    dy *= zz * sigmoid(zz);
                }
            }
            sd[i] = d;
            su[i] = uu;
            sy[i] = dy;
        }
        for (int i = tid; i < TK * NP; i += NT) {
            const int j = i / NP, s = i - j * NP;
            const bool in = j < len && s < n;
            const float b = in ? to_f(Bp[(tl + j) * a.d.B.tok_stride + s]) : 0.f;
            const float c = in ? to_f(Cp[(tl + j) * a.d.C.tok_stride + s]) : 0.f;
            sB[2 * i] = sB[2 * i + 1] = b;
            sC[2 * i] = sC[2 * i + 1] = c;
        }
        __syncthreads();

        float2 h[4][2];
        auto step = [&](int j) {  // h of token j from h of the token before
            const float4 d4 = *reinterpret_cast<const float4*>(sd + j * CT + lc);
            const float4 u4 = *reinterpret_cast<const float4*>(su + j * CT + lc);
            const float2 dd[2] = {make_float2(d4.x, d4.y), make_float2(d4.z, d4.w)};
            const float2 du2[2] = {mul2(dd[0], make_float2(u4.x, u4.y)),
                                   mul2(dd[1], make_float2(u4.z, u4.w))};
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const float2 b = *reinterpret_cast<const float2*>(sB + (j * NP + s0 + s) * 2);
#pragma unroll
                for (int p = 0; p < 2; ++p) {
                    const float2 e = mul2(dd[p], A2[s][p]);
                    h[s][p] = fma2(make_float2(ex2(e.x), ex2(e.y)), h[s][p], mul2(du2[p], b));
                    if (s0 + s >= n) h[s][p] = make_float2(0.f, 0.f);
                }
            }
        };
        load_padded(a.f.tiles + (row * ntiles + tl / TK) * a.d.channels * NP, h);
        const int last = (len - 1) / TS;
        for (int piece = 0; piece <= last; ++piece) {
            put(piece, h);
            if (piece < last) {
#pragma unroll
                for (int j = 0; j < TS; ++j) {
                    if (sq_flag[piece * TS + j] & 1) initial(piece * TS + j, h);
                    step(piece * TS + j);
                }
            }
        }
        for (int piece = last; piece >= 0; --piece) {
            float2 hist[TS][4][2], hs[4][2];
            get(piece, h);
#pragma unroll
            for (int s = 0; s < 4; ++s)
#pragma unroll
                for (int p = 0; p < 2; ++p) hs[s][p] = h[s][p];
#pragma unroll
            for (int j = 0; j < TS; ++j) {
                if (piece * TS + j < len) {
                    if (sq_flag[piece * TS + j] & 1) initial(piece * TS + j, h);
                    step(piece * TS + j);
                }
#pragma unroll
                for (int s = 0; s < 4; ++s)
#pragma unroll
                    for (int p = 0; p < 2; ++p) hist[j][s][p] = h[s][p];
            }
            float* red = sred + rbuf * S::kRed;
#pragma unroll
            for (int jj = TS - 1; jj >= 0; --jj) {
                const int j = piece * TS + jj;
                if (j >= len) continue;
                const int64_t t = tl + j;
                const int flag = sq_flag[j];
                // what the owner of a channel still needs of its inputs
                float ro[OWN], rz[OWN], re[OWN];
#pragma unroll
                for (int k = 0; k < OWN; ++k) {
                    const int64_t c = c0 + lo + k;
                    const bool in = owner && c < cend;
                    ro[k] = in && gate ? to_f(dout[t * a.g.dout.tok_stride + c]) : 0.f;
                    rz[k] = in && gate ? to_f(z[t * a.d.z.tok_stride + c]) : 0.f;
                    re[k] = in && a.d.softplus ? to_f(dl[t * a.d.delta.tok_stride + c]) + obias[k] : 0.f;
                }
                if (flag & 2)
                    load4(a.g.dfinal_state ? a.g.dfinal_state + sq_id[j] * a.d.channels * n : nullptr,
                          n, m);
                float2 hp[4][2];  // the state before the token
                if (flag & 1) {
                    initial(j, hp);
                } else {
#pragma unroll
                    for (int s = 0; s < 4; ++s)
#pragma unroll
                        for (int p = 0; p < 2; ++p) hp[s][p] = jj > 0 ? hist[jj > 0 ? jj - 1 : 0][s][p] : hs[s][p];
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
                    float2 db = make_float2(0.f, 0.f), dc = make_float2(0.f, 0.f);
#pragma unroll
                    for (int p = 0; p < 2; ++p) {
                        const float2 e = mul2(dd[p], A2[s][p]);
                        const float2 q = fma2(dy[p], c, m[s][p]);
                        const float2 aq = mul2(make_float2(ex2(e.x), ex2(e.y)), q);
                        const float2 w = mul2(aq, hp[s][p]);
                        yv[p] = fma2(c, hist[jj][s][p], yv[p]);
                        qb[p] = fma2(q, b, qb[p]);
                        qa[p] = fma2(w, A2[s][p], qa[p]);
                        dA[s][p] = fma2(w, dd[p], dA[s][p]);
                        db = fma2(q, du2[p], db);
                        dc = fma2(dy[p], hist[jj][s][p], dc);
                        m[s][p] = aq;
                    }
                    bc[s] = db.x + db.y;
                    bc[4 + s] = dc.x + dc.y;
                }
                if (flag & 1) {  // the sequence's first token
                    if (a.g.dinitial_state) {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
#pragma unroll
                            for (int s = 0; s < 4; ++s)
                                if (c0 + lc + i < cend && s0 + s < n)
                                    a.g.dinitial_state[(sq_id[j] * a.d.channels + c0 + lc + i) * n + s0 + s] =
                                        i & 1 ? m[s][i / 2].y : m[s][i / 2].x;
                    }
#pragma unroll
                    for (int s = 0; s < 4; ++s)
#pragma unroll
                        for (int p = 0; p < 2; ++p) m[s][p] = make_float2(0.f, 0.f);
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
                    const int64_t c = c0 + lo + k;
                    if (!owner || c >= cend) continue;
                    const float d = sd[j * CT + lo + k], uu = su[j * CT + lo + k], dyk = sy[j * CT + lo + k];
                    du[t * a.g.du.tok_stride + c] = from_f<T>(fmaf(d, vb[k], dyk * oD[k]));
                    float e = fmaf(uu, vb[k], va[k] * kLn2);  // A = A2 ln 2
                    if (a.d.softplus) e *= sigmoid(re[k]);
                    ddl[t * a.g.ddelta.tok_stride + c] = from_f<T>(e);
                    abias[k] += e;
                    aD[k] = fmaf(dyk, uu, aD[k]);
                    if (gate) {
                        const float y = fmaf(oD[k], uu, vy[k]), sg = sigmoid(rz[k]);
                        dz[t * a.g.dz.tok_stride + c] =
                            from_f<T>(ro[k] * y * (sg * (1.f + rz[k] * (1.f - sg))));
                    }
                }
                // sums over channels, handed out to the channel lanes
                constexpr int LEFT = CL >= 8 ? 1 : 8 / CL;
                hand_out<8, CL / 2, SL>(bc, cl);
                int vi = 0;
                if (CL >= 2) vi += (cl & (CL / 2)) ? 4 : 0;
                if (CL >= 4) vi += (cl & (CL / 4)) ? 2 : 0;
                if (CL >= 8) vi += (cl & (CL / 8)) ? 1 : 0;
                if (CL <= 8 || cl % (CL / 8) == 0) {
#pragma unroll
                    for (int k = 0; k < LEFT; ++k)
                        red[((warp * TS + jj) * 8 + vi + k) * SL + sl] = bc[k];
                }
            }
            __syncthreads();
            // the piece's dB and dC, summed over the warps; the other buffer is filled meanwhile
            const int plen = len - piece * TS < TS ? len - piece * TS : TS;
            for (int i = tid; i < plen * 8 * SL; i += NT) {
                const int jj = i / (8 * SL), v = (i / SL) % 8, state = (i % SL) * 4 + (v & 3);
                float x = 0.f;
#pragma unroll
                for (int w = 0; w < S::NW; ++w) x += red[w * TS * 8 * SL + i];
                if (state < n) {
                    const int64_t t = tl + piece * TS + jj;
                    a.bc[((((ct * a.f.rows + row) * a.d.length + t) * a.d.groups + g) * 2 + (v >> 2)) * n +
                         state] = x;
                }
            }
            rbuf ^= 1;
        }
    }
    const int64_t part = row * a.f.nchunks + chunk;
    if (a.pA) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int s = 0; s < 4; ++s)
                if (c0 + lc + i < cend && s0 + s < n)
                    a.pA[(part * a.d.channels + c0 + lc + i) * n + s0 + s] =
                        i & 1 ? dA[s][i / 2].y : dA[s][i / 2].x;
    }
#pragma unroll
    for (int k = 0; k < OWN; ++k) {
        const int64_t c = c0 + lo + k;
        if (!owner || c >= cend) continue;
        if (a.pD) a.pD[part * a.d.channels + c] = aD[k];
        if (a.pbias) a.pbias[part * a.d.channels + c] = abias[k];
    }
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

template <class T, int SL>
cudaError_t scan_bwd_main(const ScanBwdArgs& a, cudaStream_t s) {
    using S = BwdShape<SL>;
    static LaunchCache cache;
    LaunchGeom geo;
    cudaError_t e = cache.get([](int dev, LaunchGeom* g) {
        return setup_persistent(k_scan_bwd<T, SL>, S::NT, S::kBytes, dev, g);
    }, &geo);
    if (e != cudaSuccess) return e;
    const int64_t blocks = a.f.rows * a.f.nchunks * a.ctiles * a.d.groups;
    if (blocks > INT32_MAX) return cudaErrorInvalidValue;
    k_scan_bwd<T, SL><<<(unsigned)blocks, S::NT, S::kBytes, s>>>(a);
    return cudaGetLastError();
}
template <class T, int SPT, int SL>
cudaError_t scan_bwd_back(const ScanBwdArgs& a, cudaStream_t s) {
    const int64_t tiles = a.back_ctiles * a.d.groups;
    k_scan_back<T, SPT, SL>
        <<<(unsigned)(a.f.rows * (a.f.nchunks - 1) * tiles), kScanThreads, 0, s>>>(a);
    k_scan_back_carry<SPT * SL>
        <<<(unsigned)((a.f.rows * a.d.channels * SPT * SL + kCarryThreads - 1) / kCarryThreads),
           kCarryThreads, 0, s>>>(a);
    return cudaGetLastError();
}

template <class T>
cudaError_t scan_bwd_run(const ScanBwdArgs& a, cudaStream_t s) {
    cudaError_t e = cudaSuccess;
    const int64_t n = a.d.states, parts = a.f.rows * a.f.nchunks;
    if (a.d.length > 0) {
        if (parts * a.back_ctiles * a.d.groups > INT32_MAX) return cudaErrorInvalidValue;
        e = scan_run<T, SCAN_TILES>(a.f, s);
        if (e == cudaSuccess && a.f.nchunks > 1) {
            switch (scan_np(n)) {
                case 4: e = scan_bwd_back<T, 4, 1>(a, s); break;
                case 8: e = scan_bwd_back<T, 8, 1>(a, s); break;
                case 16: e = scan_bwd_back<T, 16, 1>(a, s); break;
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
