// Selective state-space scan, forward (fft_scan_forward).
//
//   h[t] = exp(d[t] A) h[t-1] + d[t] u[t] B[t];  y[t] = sum_s C[t,s] h[t,s] + D u[t]
//
// A thread holds SPT states of one channel in registers and walks the tokens; SL lanes share a
// channel.  Tiles of 8 tokens: B and C (shared by all channels of a group) are staged in shared
// memory as float32, double buffered; u, delta and z are loaded a tile ahead into the registers
// of the lane that owns the token, which also computes d and the gate, so nothing is done twice.
// Per state: one ex2, and a multiply (d A), a multiply (d u B) and two fused multiply-adds, two
// states to an instruction.
//
// With too few channels for the GPU, time is cut into chunks.  A chunk's effect on the state is
// h -> exp(A sum d) h + h_local, so pass 1 computes h_local and sum d of every chunk (from zero),
// pass 2 runs along the chunks, and pass 3 is the full scan of each chunk from its true start.
#pragma once

#include "scan.h"

namespace gbfft {

struct ScanBlock {
    int64_t row, chunk, c0, cend;  // channels [c0, cend) of the block
    int64_t g;
    int64_t t0, t1;
};
__device__ __forceinline__ ScanBlock scan_block(const ScanArgs& a, int64_t id, int64_t nchunks,
                                                int ct) {
    ScanBlock b;
    const int64_t tiles = a.ctiles * a.d.groups, dg = a.d.channels / a.d.groups;
    const int64_t tile = id % tiles, rest = id / tiles;
    b.chunk = rest % nchunks;
    b.row = rest / nchunks;
    b.g = tile / a.ctiles;
    b.c0 = b.g * dg + (tile - b.g * a.ctiles) * ct;
    b.cend = (b.g + 1) * dg;
    b.t0 = b.chunk * a.chunk;
    b.t1 = b.t0 + a.chunk < a.d.length ? b.t0 + a.chunk : a.d.length;
    return b;
}

template <class T>
__device__ __forceinline__ const T* row_of(const fft_seq& s, bool packed, int64_t row) {
    return static_cast<const T*>(s.data) + (packed ? 0 : row * s.seq_stride);
}

// SPT states from a [channels][n] row; the states beyond n are zero.
template <int SPT>
__device__ __forceinline__ void load_states(const float* p, int s0, int n, float2 (&h)[SPT / 2]) {
#pragma unroll
    for (int i = 0; i < SPT / 2; ++i) {
        h[i].x = p && s0 + 2 * i < n ? p[s0 + 2 * i] : 0.f;
        h[i].y = p && s0 + 2 * i + 1 < n ? p[s0 + 2 * i + 1] : 0.f;
    }
}
template <int SPT>
__device__ __forceinline__ void store_states(float* p, int s0, int n, const float2 (&h)[SPT / 2]) {
#pragma unroll
    for (int i = 0; i < SPT / 2; ++i) {
        if (s0 + 2 * i < n) p[s0 + 2 * i] = h[i].x;
        if (s0 + 2 * i + 1 < n) p[s0 + 2 * i + 1] = h[i].y;
    }
}

// A state beyond n has A = B = C = 0; EXACT (n == SPT * SL) drops the selects that keep such
// states at 0 where u is infinite.
template <class T, int SPT, int SL, int PASS, bool EXACT>
__global__ void __launch_bounds__(kScanThreads) k_scan(const ScanArgs a) {
    constexpr int NP = SPT * SL, CT = kScanThreads / SL, TK = kScanTile, OWN = TK / SL;
    constexpr int CL = 32 / SL;  // channels of a warp
    constexpr bool SUMMARY = PASS == SCAN_SUMMARY, OUTPUT = PASS == SCAN_OUTPUT;
    constexpr int BCN = (TK * NP + kScanThreads - 1) / kScanThreads;  // B values per thread, tile
    __shared__ alignas(16) float sB[2][TK][NP];
    __shared__ alignas(16) float sC[2][OUTPUT ? TK : 1][NP];
    const int n = (int)a.d.states, tid = (int)threadIdx.x, lane = tid & 31;
    const bool packed = a.d.offsets != nullptr;
    const int64_t nch = SUMMARY ? a.nchunks - 1 : a.nchunks;
    const int64_t mains = a.rows * nch * a.ctiles * a.d.groups;
    if (OUTPUT && (int64_t)blockIdx.x >= mains) {
        // the blocks behind: a sequence without tokens ends in its initial state
        const int64_t q = blockIdx.x - mains, per = a.d.channels * n;
        const bool empty = packed ? a.d.offsets[q] >= a.d.offsets[q + 1] : a.d.length == 0;
        if (empty)
            for (int64_t i = tid; i < per; i += kScanThreads)
                a.final_state[q * per + i] = a.d.initial_state ? a.d.initial_state[q * per + i] : 0.f;
        return;
    }
    const ScanBlock blk = scan_block(a, blockIdx.x, nch, CT);
    SeqAt sq = seq_at(a.d.offsets, a.d.nseq, a.d.length, blk.row, blk.t0);
    const int sl = lane / CL;
    const int64_t c = blk.c0 + (tid >> 5) * CL + lane % CL;
    const bool live = c < blk.cend;
    const int s0 = sl * SPT;
    const T* u = row_of<T>(a.d.u, packed, blk.row) + c;
    const T* dl = row_of<T>(a.d.delta, packed, blk.row) + c;
    const T* z = row_of<T>(a.d.z, packed, blk.row) + c;
    const T* Bp = row_of<T>(a.d.B, packed, blk.row) + blk.g * n;
    const T* Cp = row_of<T>(a.d.C, packed, blk.row) + blk.g * n;
    T* out = const_cast<T*>(row_of<T>(a.out, packed, blk.row)) + c;
    const bool gate = a.d.z.data != nullptr;

    float2 A2[SPT / 2], h[SPT / 2];
    load_states<SPT>(live ? a.d.A + c * n : nullptr, s0, n, A2);
#pragma unroll
    for (int i = 0; i < SPT / 2; ++i) A2[i] = mul2(A2[i], make_float2(kLog2e, kLog2e));
    const float bias = live && a.d.delta_bias ? a.d.delta_bias[c] : 0.f;
    const float D = live && a.d.D ? a.d.D[c] : 0.f;
    auto initial = [&]() {
        load_states<SPT>(live && a.d.initial_state
                             ? a.d.initial_state + (sq.q * a.d.channels + c) * n : nullptr, s0, n, h);
    };
    const int64_t carry_at = ((blk.row * a.nchunks + blk.chunk) * a.d.channels + c) * NP;
    bool has_reset = sq.begin == blk.t0;
    if (sq.begin == blk.t0)
        initial();
    else if (SUMMARY)
        load_states<SPT>(nullptr, s0, n, h);
    else
        load_states<SPT>(live ? a.carry + carry_at : nullptr, s0, NP, h);
    float dsum = 0.f;

    T pu[OWN], pd[OWN], pz[OWN], pB[BCN], pC[BCN];
    auto fetch = [&](int64_t t) {  // tile at t into registers; zeros outside
#pragma unroll
        for (int j = 0; j < OWN; ++j) {
            const int64_t tt = t + sl * OWN + j;
            const bool in = live && tt < blk.t1;
            pu[j] = in ? u[tt * a.d.u.tok_stride] : from_f<T>(0.f);
            pd[j] = in ? dl[tt * a.d.delta.tok_stride] : from_f<T>(0.f);
            if (OUTPUT) pz[j] = in && gate ? z[tt * a.d.z.tok_stride] : from_f<T>(0.f);
        }
#pragma unroll
        for (int i = 0; i < BCN; ++i) {
            const int k = tid + i * kScanThreads;
            const int64_t tt = t + k / NP;
            const bool in = k < TK * NP && k % NP < n && tt < blk.t1;
            pB[i] = in ? Bp[tt * a.d.B.tok_stride + k % NP] : from_f<T>(0.f);
            if (OUTPUT) pC[i] = in ? Cp[tt * a.d.C.tok_stride + k % NP] : from_f<T>(0.f);
        }
    };
    auto stage = [&](int buf) {
#pragma unroll
        for (int i = 0; i < BCN; ++i) {
            const int k = tid + i * kScanThreads;
            if (k < TK * NP) {
                (&sB[buf][0][0])[k] = to_f(pB[i]);
                if (OUTPUT) (&sC[buf][0][0])[k] = to_f(pC[i]);
            }
        }
    };
    fetch(blk.t0);
    stage(0);
    __syncthreads();
    int buf = 0;
    for (int64_t t = blk.t0; t < blk.t1; t += TK) {
        float od[OWN], ou[OWN], oz[OWN];  // the tokens that this lane owns
#pragma unroll
        for (int j = 0; j < OWN; ++j) {
            const float e = to_f(pd[j]) + bias;
            od[j] = a.d.softplus ? softplus(e) : e;
            ou[j] = to_f(pu[j]);
            if (OUTPUT) oz[j] = to_f(pz[j]);
        }
        if (PASS == SCAN_TILES && t % kScanStateTile == 0 && live) {
            const int64_t tiles = (a.d.length + kScanStateTile - 1) / kScanStateTile;
            store_states<SPT>(a.tiles + ((blk.row * tiles + t / kScanStateTile) * a.d.channels + c) * NP,
                              s0, NP, h);
        }
        if (t + TK < blk.t1) fetch(t + TK);
        float y[TK];
#pragma unroll
        for (int j = 0; j < TK; ++j) {
            if (t + j >= blk.t1) {
                y[j] = 0.f;
                continue;
            }
            if (t + j >= sq.end) {  // packed: the next sequence begins
                seq_next(a.d.offsets, a.d.nseq, t + j, &sq);
                initial();
                has_reset = true;
            }
            float d = od[j % OWN], uu = ou[j % OWN];
            if (SL > 1) {
                d = __shfl_sync(0xffffffffu, d, (j / OWN) * CL + lane % CL);
                uu = __shfl_sync(0xffffffffu, uu, (j / OWN) * CL + lane % CL);
            }
            if (SUMMARY) dsum += d;
            const float2 dd = make_float2(d, d), du = make_float2(d * uu, d * uu);
            float2 acc = make_float2(0.f, 0.f);
#pragma unroll
            for (int i = 0; i < SPT / 2; ++i) {
                const float2 arg = mul2(dd, A2[i]);
                const float2 b = mul2(du, *reinterpret_cast<const float2*>(&sB[buf][j][s0 + 2 * i]));
                h[i] = fma2(make_float2(ex2(arg.x), ex2(arg.y)), h[i], b);
                if (!EXACT) {
                    if (s0 + 2 * i >= n) h[i].x = 0.f;
                    if (s0 + 2 * i + 1 >= n) h[i].y = 0.f;
                }
                if (OUTPUT)
                    acc = fma2(*reinterpret_cast<const float2*>(&sC[buf][j][s0 + 2 * i]), h[i], acc);
            }
            y[j] = acc.x + acc.y;
            if (OUTPUT && a.final_state && t + j + 1 == sq.end && live)
                store_states<SPT>(a.final_state + (sq.q * a.d.channels + c) * n, s0, n, h);
        }
        if (OUTPUT) {
            // sums over the SL lanes: each step halves the tokens that a lane still carries
#pragma unroll
            for (int w = SL / 2, cnt = TK / 2; w; w /= 2, cnt /= 2) {
                const bool up = sl & w;
#pragma unroll
                for (int j = 0; j < cnt; ++j) {
                    const float send = up ? y[j] : y[j + cnt], keep = up ? y[j + cnt] : y[j];
                    y[j] = keep + __shfl_xor_sync(0xffffffffu, send, w * CL);
                }
            }
#pragma unroll
            for (int j = 0; j < OWN; ++j) {
                const int64_t tt = t + sl * OWN + j;
                float v = fmaf(D, ou[j], y[j]);
                if (gate) v *= oz[j] * sigmoid(oz[j]);
                if (live && tt < blk.t1) out[tt * a.out.tok_stride] = from_f<T>(v);
            }
        }
        if (t + TK < blk.t1) {
            buf ^= 1;
            stage(buf);
            __syncthreads();
        }
    }
    if (SUMMARY) {
        if (live) {
            store_states<SPT>(a.carry + carry_at, s0, NP, h);
            if (sl == 0) a.dsum[(blk.row * a.nchunks + blk.chunk) * a.d.channels + c] = dsum;
        }
        if (tid == 0 && blk.c0 == 0) a.reset[blk.row * a.nchunks + blk.chunk] = has_reset;
    }
}

// Pass 2: along the chunks of every (row, channel, state); the state after a chunk that a
// sequence starts in does not depend on what came before.
template <int NP>
__global__ void __launch_bounds__(256) k_scan_carry(const ScanArgs a) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, per = a.d.channels * NP;
    if (i >= a.rows * per) return;
    const int64_t row = i / per, cs = i - row * per, c = cs / NP;
    const int s = (int)(cs - c * NP), n = (int)a.d.states;
    const float A2 = s < n ? a.d.A[c * n + s] * kLog2e : 0.f;
    float* carry = a.carry + row * a.nchunks * per + cs;
    const float* dsum = a.dsum + row * a.nchunks * a.d.channels + c;
    const int* reset = a.reset + row * a.nchunks;
    float h = 0.f;
    constexpr int U = 8;
    for (int64_t k = 0; k < a.nchunks; k += U) {
        float local[U], decay[U];
#pragma unroll
        for (int j = 0; j < U; ++j) {
            if (k + j < a.nchunks - 1) {
                local[j] = carry[(k + j) * per];
                decay[j] = reset[k + j] ? -1.f : ex2(A2 * dsum[(k + j) * a.d.channels]);
            }
        }
#pragma unroll
        for (int j = 0; j < U; ++j) {
            if (k + j >= a.nchunks) break;
            carry[(k + j) * per] = h;
            if (k + j < a.nchunks - 1) h = decay[j] < 0.f ? local[j] : fmaf(decay[j], h, local[j]);
        }
    }
}

// Passes 1 and 2 where time is cut, then the pass that was asked for.
template <class T, int SPT, int SL, int PASS, bool EXACT>
cudaError_t scan_launch(const ScanArgs& a, cudaStream_t s) {
    const int64_t tiles = a.ctiles * a.d.groups;
    const bool empties = PASS == SCAN_OUTPUT && a.final_state && (a.d.offsets || a.d.length == 0);
    const int64_t blocks = a.rows * a.nchunks * tiles + (empties ? a.d.nseq : 0);
    if (blocks < 1) return cudaSuccess;
    if (blocks > INT32_MAX) return cudaErrorInvalidValue;
    if (a.nchunks > 1) {
        k_scan<T, SPT, SL, SCAN_SUMMARY, EXACT>
            <<<(unsigned)(a.rows * (a.nchunks - 1) * tiles), kScanThreads, 0, s>>>(a);
        k_scan_carry<SPT * SL>
            <<<(unsigned)((a.rows * a.d.channels * SPT * SL + 255) / 256), 256, 0, s>>>(a);
    }
    k_scan<T, SPT, SL, PASS, EXACT><<<(unsigned)blocks, kScanThreads, 0, s>>>(a);
    return cudaGetLastError();
}

template <class T, int SPT, int SL, int PASS>
cudaError_t scan_exact(const ScanArgs& a, cudaStream_t s) {
    return a.d.states == SPT * SL ? scan_launch<T, SPT, SL, PASS, true>(a, s)
                                  : scan_launch<T, SPT, SL, PASS, false>(a, s);
}
template <class T, int PASS>
cudaError_t scan_run(const ScanArgs& a, cudaStream_t s) {
    const ScanShape sh = scan_shape(a.d.states);
    if (sh.sl == 1)
        return sh.spt == 4 ? scan_exact<T, 4, 1, PASS>(a, s)
                           : (sh.spt == 8 ? scan_exact<T, 8, 1, PASS>(a, s)
                                          : scan_exact<T, 16, 1, PASS>(a, s));
    return sh.sl == 2 ? scan_exact<T, 16, 2, PASS>(a, s)
                      : (sh.sl == 4 ? scan_exact<T, 16, 4, PASS>(a, s)
                                    : scan_exact<T, 16, 8, PASS>(a, s));
}

}  // namespace gbfft
