// Selective state-space scan, forward (fft_scan_forward).
//
//   h[t] = exp(d[t] A) h[t-1] + d[t] u[t] B[t];  y[t] = sum_s C[t,s] h[t,s] + D u[t]
//
// A thread holds the states of its channels in registers and walks the tokens.  Per state and
// token that costs one ex2, and a multiply (d A), a multiply (d u B) and two fused multiply-adds,
// two states to an instruction; the multiply-add pipe and the exponential unit are about equally
// busy, and both far busier than HBM.  Up to 16 states: k_scan, two channels per thread, so that
// one load of B and C from shared memory serves both (with one channel per thread those loads
// filled the shared-memory pipe).  More states, or more channels: k_scan_lanes, several lanes per
// channel.  Measured, bfloat16, 16 states, gated: one sequence of 16384 x 2048 247 us (the
// exponential unit 50 to 62% and the multiply-add pipe 57% busy at 12 warps of an SM), 8 x 2048 x
// 4096 in one pass 404 us (35% and 45%).  What carried it: softplus and gates of 8 tokens side by
// side (their chains are long: 175 -> 153 us for the last pass of the long sequence), and kernels
// without questions for whole 16-byte rows (153 -> 136 us).
//
// With too few channels for the GPU, time is cut into chunks.  A chunk's effect on the state is
// h -> exp(A sum d) h + h_local, so pass 1 computes h_local and sum d of every chunk (from zero),
// pass 2 runs along the chunks, and pass 3 is the full scan of each chunk from its true start.
#pragma once

#include "launch_cache.cuh"
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

// The same for rows padded to a multiple of four states, 16-byte aligned.
template <int SPT>
__device__ __forceinline__ void load_row(const float* p, float2 (&h)[SPT / 2]) {
#pragma unroll
    for (int i = 0; i < SPT / 4; ++i) {
        const float4 v = *reinterpret_cast<const float4*>(p + 4 * i);
        h[2 * i] = make_float2(v.x, v.y);
        h[2 * i + 1] = make_float2(v.z, v.w);
    }
}
template <int SPT>
__device__ __forceinline__ void store_row(float* p, const float2 (&h)[SPT / 2]) {
#pragma unroll
    for (int i = 0; i < SPT / 4; ++i)
        *reinterpret_cast<float4*>(p + 4 * i) =
            make_float4(h[2 * i].x, h[2 * i].y, h[2 * i + 1].x, h[2 * i + 1].y);
}

// Tokens t .. t + TK - 1 of a tensor (p: token 0, the block's first channel) into dst[token][CT],
// zeros beyond `len` tokens and `width` channels.  align: bytes that every row starts on, 16 (the
// only case of FAST kernels) or 4; smaller: single values, and then not asynchronously.
template <class T, int TK, int CT, int NT, bool FAST>
__device__ __forceinline__ void copy_tile(T* dst, const T* p, int64_t stride, int t, int len,
                                          int width, int align) {
    const int tid = (int)threadIdx.x;
    if (FAST || align >= 16) {
        constexpr int V = 16 / sizeof(T), R = CT / V;  // accesses of a row
        if constexpr (NT % R == 0 && TK % (NT / R) == 0) {
            constexpr int STEP = NT / R;
            static_assert(STEP > 0, "the loop ends");
            const int j0 = tid / R, x = (tid - j0 * R) * V;
            const T* q = p + (t + j0) * stride + x;
#pragma unroll
            for (int j = 0; j < TK; j += STEP, q += STEP * stride) {
                const bool in = t + j0 + j < len && x < width;
                copy16(dst + (j0 + j) * CT + x, in ? q : p, in);
            }
        } else {
#pragma unroll
            for (int e = tid; e < TK * R; e += NT) {
                const int j = e / R, x = (e - j * R) * V;
                const bool in = t + j < len && x < width;
                copy16(dst + j * CT + x, in ? p + (t + j) * stride + x : p, in);
            }
        }
    } else if (align >= 4) {
        constexpr int V = 4 / sizeof(T), R = CT / V;
#pragma unroll 4
        for (int e = tid; e < TK * R; e += NT) {
            const int j = e / R, x = (e - j * R) * V;
            const bool in = t + j < len && x < width;
            copy4(dst + j * CT + x, in ? p + (t + j) * stride + x : p, in);
        }
    } else {
#pragma unroll 8
        for (int e = tid; e < TK * CT; e += NT) {
            const int j = e / CT, x = e - j * CT;
            dst[e] = t + j < len && x < width ? p[(t + j) * stride + x] : from_f<T>(0.f);
        }
    }
}

// B (and C) of a tile, from global memory through registers to float32 [token][NP] in shared
// memory.  FAST: the n == NP values of a token are whole 16-byte accesses.
template <class T, int TK, int NP, int NT, bool BOTH, bool FAST>
struct RowsAhead {
    static constexpr int V = 16 / sizeof(T);
    static_assert(!FAST || NP % V == 0, "a token's states are whole accesses");
    static constexpr int WIDE = FAST ? (TK * NP / V + NT - 1) / NT : 0;  // accesses per thread
    static constexpr int ONE = (TK * NP + NT - 1) / NT;
    uint4 wide[BOTH ? 2 : 1][FAST ? WIDE : 1];
    T one[BOTH ? 2 : 1][FAST ? 1 : ONE];
    __device__ __forceinline__ void fetch(const T* b, int64_t bs, const T* c, int64_t cs, int t,
                                          int len, int n) {
        const int tid = (int)threadIdx.x;
        if constexpr (FAST) {
#pragma unroll
            for (int i = 0; i < WIDE; ++i) {
                const int e = tid + i * NT, j = e / (NP / V), s = (e - j * (NP / V)) * V;
                const bool in = j < TK && t >= 0 && t + j < len;
                wide[0][i] = in ? *reinterpret_cast<const uint4*>(b + (t + j) * bs + s) : uint4{};
                if (BOTH)
                    wide[BOTH][i] = in ? *reinterpret_cast<const uint4*>(c + (t + j) * cs + s) : uint4{};
            }
        } else {
#pragma unroll
            for (int i = 0; i < ONE; ++i) {
                const int e = tid + i * NT, j = e / NP, s = e - j * NP;
                const bool in = j < TK && s < n && t >= 0 && t + j < len;
                one[0][i] = in ? b[(t + j) * bs + s] : from_f<T>(0.f);
                if (BOTH) one[BOTH][i] = in ? c[(t + j) * cs + s] : from_f<T>(0.f);
            }
        }
    }
    __device__ __forceinline__ void stage(float* sb) {
        const int tid = (int)threadIdx.x;
#pragma unroll
        for (int k = 0; k < (BOTH ? 2 : 1); ++k) {
            float* dst = sb + k * TK * NP;
            if constexpr (FAST) {
#pragma unroll
                for (int i = 0; i < WIDE; ++i) {
                    const int e = tid + i * NT;
                    if (e * V < TK * NP) {
                        const Pack<T, V> p = *reinterpret_cast<const Pack<T, V>*>(&wide[k][i]);
#pragma unroll
                        for (int v = 0; v < V; v += 4)
                            *reinterpret_cast<float4*>(dst + e * V + v) = make_float4(
                                to_f(p.v[v]), to_f(p.v[v + 1]), to_f(p.v[v + 2]), to_f(p.v[v + 3]));
                    }
                }
            } else {
#pragma unroll
                for (int i = 0; i < ONE; ++i) {
                    const int e = tid + i * NT;
                    if (TK * NP % NT == 0 || e < TK * NP) dst[e] = to_f(one[k][i]);
                }
            }
        }
    }
};

// The blocks behind the outputs: a sequence without tokens ends in its initial state.
__device__ __forceinline__ void scan_empty(const ScanArgs& a, int64_t q) {
    const int64_t per = a.d.channels * a.d.states;
    if (a.d.offsets ? a.d.offsets[q] < a.d.offsets[q + 1] : a.d.length != 0) return;
    for (int64_t i = threadIdx.x; i < per; i += blockDim.x)
        a.final_state[q * per + i] = a.d.initial_state ? a.d.initial_state[q * per + i] : 0.f;
}

constexpr int kPairThreads = 64, kPairChannels = 2 * kPairThreads, kPairTile = 8;
constexpr int kPairBatch = 8;  // tokens whose softplus and gates run side by side
template <int N>
struct Count {
    static constexpr int value = N;
};

template <class T, int SPT, int PASS>
struct ScanPairSmem {
    static constexpr bool OUTPUT = PASS == SCAN_OUTPUT;
    static constexpr int kStages = 3, kRaw = kPairTile * kPairChannels, kTensors = OUTPUT ? 3 : 2;
    static constexpr int kBC = kPairTile * SPT * (OUTPUT ? 2 : 1);  // floats of a buffer
    static constexpr int kBytesRaw = kStages * kTensors * kRaw * (int)sizeof(T);
    static constexpr int kBytes = kBytesRaw + 2 * kBC * 4;
};

// Up to 16 states: a thread holds all SPT states of two neighbouring channels.  Tiles of 8
// tokens: u, delta and z come by asynchronous copies two tiles ahead, B and C a tile ahead
// through registers, double buffered in shared memory as float32: one barrier per tile.
// SPT is n rounded up to fours; a state beyond n is kept at 0 (its B is 0, but u may be infinite).
// FAST: n == SPT and all rows are whole 16-byte accesses, the usual case,
// whose code is free of these questions.
template <class T, int SPT, int PASS, bool FAST>
__global__ void __launch_bounds__(kPairThreads, 6) k_scan(const ScanArgs a) {
    using M = ScanPairSmem<T, SPT, PASS>;
    constexpr int NT = kPairThreads, CT = kPairChannels, TK = kPairTile, ST = M::kStages;
    constexpr bool SUMMARY = PASS == SCAN_SUMMARY, OUTPUT = PASS == SCAN_OUTPUT;
    // fours below this one lie within n; the backward pass's 16 may stand for as few as nine
    constexpr int WHOLE = SPT == 16 && !OUTPUT ? 2 : SPT / 4 - 1;
    extern __shared__ float4 smem4[];
    T* raw = reinterpret_cast<T*>(smem4);  // [stage][tensor][token][channel]
    float* sbc = reinterpret_cast<float*>(reinterpret_cast<char*>(smem4) + M::kBytesRaw);

    const int n = (int)a.d.states, tid = (int)threadIdx.x;
    const bool packed = a.d.offsets != nullptr, gate = OUTPUT && a.d.z.data != nullptr;
    const int64_t nch = SUMMARY ? a.nchunks - 1 : a.nchunks;
    const int64_t mains = a.rows * nch * a.ctiles * a.d.groups;
    if (OUTPUT && (int64_t)blockIdx.x >= mains) return scan_empty(a, blockIdx.x - mains);
    const ScanBlock blk = scan_block(a, blockIdx.x, nch, CT);
    SeqAt sq = seq_at(a.d.offsets, a.d.nseq, a.d.length, blk.row, blk.t0);
    const int width = (int)(blk.cend - blk.c0 < CT ? blk.cend - blk.c0 : CT);  // channels here
    const int lc = 2 * tid, len = (int)(blk.t1 - blk.t0);
    const int64_t c = blk.c0 + lc;
    const bool live[2] = {lc < width, lc + 1 < width};
    // token t0 of the chunk; from here on tokens count from t0
    const T* src[3] = {row_of<T>(a.d.u, packed, blk.row) + blk.t0 * a.d.u.tok_stride + blk.c0,
                       row_of<T>(a.d.delta, packed, blk.row) + blk.t0 * a.d.delta.tok_stride + blk.c0,
                       gate ? row_of<T>(a.d.z, packed, blk.row) + blk.t0 * a.d.z.tok_stride + blk.c0
                            : nullptr};
    const int64_t str[3] = {a.d.u.tok_stride, a.d.delta.tok_stride, a.d.z.tok_stride};
    const T* Bp = row_of<T>(a.d.B, packed, blk.row) + blk.t0 * a.d.B.tok_stride + blk.g * n;
    const T* Cp = row_of<T>(a.d.C, packed, blk.row) + blk.t0 * a.d.C.tok_stride + blk.g * n;

    auto copy = [&](int t, int stage) {  // the tile at t
#pragma unroll
        for (int k = 0; k < M::kTensors; ++k) {
            if (k == 2 && !gate) break;
            copy_tile<T, TK, CT, NT, FAST>(raw + (stage * M::kTensors + k) * M::kRaw, src[k], str[k], t, len,
                                     width, a.vec);
        }
        copy_commit();
    };
    RowsAhead<T, TK, SPT, NT, OUTPUT, FAST> bc;
    auto fetch = [&](int t) {
        bc.fetch(Bp, a.d.B.tok_stride, Cp, a.d.C.tok_stride, t, len, n);
    };
    auto stage_bc = [&](int buf) { bc.stage(sbc + buf * M::kBC); };
#pragma unroll
    for (int i = 0; i < ST - 1; ++i) copy(i * TK, i);
    fetch(0);

    float2 A2[2][SPT / 2], h[2][SPT / 2];
    float2 bias = splat(0.f), D = splat(0.f), dsum = splat(0.f);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        load_states<SPT>(live[k] ? a.d.A + (c + k) * n : nullptr, 0, n, A2[k]);
#pragma unroll
        for (int i = 0; i < SPT / 2; ++i) A2[k][i] = mul2(A2[k][i], splat(kLog2e));
        if (live[k] && a.d.delta_bias) (k ? bias.y : bias.x) = a.d.delta_bias[c + k];
        if (OUTPUT && live[k] && a.d.D) (k ? D.y : D.x) = a.d.D[c + k];
    }
    auto initial = [&]() {
#pragma unroll
        for (int k = 0; k < 2; ++k)
            load_states<SPT>(live[k] && a.d.initial_state
                                 ? a.d.initial_state + (sq.q * a.d.channels + c + k) * n : nullptr,
                             0, n, h[k]);
    };
    const int64_t carry_at = ((blk.row * a.nchunks + blk.chunk) * a.d.channels + c) * SPT;
    bool has_reset = starts_at(sq, blk.t0);
    if (has_reset) {
        initial();
    } else {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            if (!SUMMARY && live[k])
                load_row<SPT>(a.carry + carry_at + k * SPT, h[k]);
            else
                load_states<SPT>(nullptr, 0, SPT, h[k]);
        }
    }
    stage_bc(0);
    fetch(TK);
    T* out = OUTPUT ? const_cast<T*>(row_of<T>(a.out, packed, blk.row)) + blk.t0 * a.out.tok_stride + c
                    : nullptr;
    const int64_t ostr = a.out.tok_stride;

    int stage = 0, buf = 0, stop = seq_stop(sq, blk.t0, len);
    for (int t = 0; t < len; t += TK) {
        copy_wait<ST - 2>();
        __syncthreads();  // this tile has landed; the last one's buffers are free
        copy(t + (ST - 1) * TK, stage >= 1 ? stage - 1 : ST - 1);
        stage_bc(buf ^ 1);
        fetch(t + 2 * TK);
        if (PASS == SCAN_TILES && t % kScanTile == 0) {
            const int64_t tiles = (a.d.length + kScanTile - 1) / kScanTile;
            float* p = a.tiles + ((blk.row * tiles + (blk.t0 + t) / kScanTile) * a.d.channels + c) * SPT;
#pragma unroll
            for (int k = 0; k < 2; ++k)
                if (live[k]) store_row<SPT>(p + k * SPT, h[k]);
        }
        const T* ru = raw + stage * M::kTensors * M::kRaw + lc;
        const T* rd = ru + M::kRaw;
        const T* rz = rd + M::kRaw;
        const float* sB = sbc + buf * M::kBC;
        const float* sC = sB + TK * SPT;
        // N tokens at j: first d and d u of all, then the recurrence, then the gates, so that the
        // long chains of softplus and the gate run side by side
        auto tokens = [&](auto count, int j0) {
            constexpr int N = decltype(count)::value;
            float2 d[N], du[N], y[N];
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const Pack<T, 2> pd = ld_pack<2>(rd + (j0 + j) * CT), pu = ld_pack<2>(ru + (j0 + j) * CT);
                d[j] = add2(make_float2(to_f(pd.v[0]), to_f(pd.v[1])), bias);
                du[j] = make_float2(to_f(pu.v[0]), to_f(pu.v[1]));
                y[j] = mul2(D, du[j]);
            }
            if (a.d.softplus) {
#pragma unroll
                for (int j = 0; j < N; ++j) d[j] = softplus2(d[j]);
            }
#pragma unroll
            for (int j = 0; j < N; ++j) {
                du[j] = mul2(d[j], du[j]);
                if (SUMMARY) dsum = add2(dsum, d[j]);
            }
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const float2 dd[2] = {splat(d[j].x), splat(d[j].y)};
                const float2 dv[2] = {splat(du[j].x), splat(du[j].y)};
                float2 acc[2][2] = {};
#pragma unroll
                for (int i = 0; i < SPT / 4; ++i) {
                    const float4 b4 = *reinterpret_cast<const float4*>(sB + (j0 + j) * SPT + 4 * i);
                    float4 c4;
                    if (OUTPUT) c4 = *reinterpret_cast<const float4*>(sC + (j0 + j) * SPT + 4 * i);
#pragma unroll
                    for (int p = 0; p < 2; ++p) {
                        const float2 b = p ? make_float2(b4.z, b4.w) : make_float2(b4.x, b4.y);
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            float2& hh = h[k][2 * i + p];
                            hh = fma2(decay2(dd[k], A2[k][2 * i + p]), hh, mul2(dv[k], b));
                            if (!FAST && i >= WHOLE) {
                                if (4 * i + 2 * p >= n) hh.x = 0.f;
                                if (4 * i + 2 * p + 1 >= n) hh.y = 0.f;
                            }
                            if (OUTPUT)
                                acc[k][p] = fma2(p ? make_float2(c4.z, c4.w) : make_float2(c4.x, c4.y),
                                                 hh, acc[k][p]);
                        }
                    }
                }
                if (OUTPUT) {
                    const float2 s0 = add2(acc[0][0], acc[0][1]), s1 = add2(acc[1][0], acc[1][1]);
                    y[j] = add2(y[j], make_float2(s0.x + s0.y, s1.x + s1.y));
                }
            }
            if (OUTPUT) {
                if (gate) {
#pragma unroll
                    for (int j = 0; j < N; ++j) {
                        const Pack<T, 2> pz = ld_pack<2>(rz + (j0 + j) * CT);
                        const float2 z = make_float2(to_f(pz.v[0]), to_f(pz.v[1]));
                        y[j] = mul2(y[j], mul2(z, sigmoid2(z)));
                    }
                }
                T* o = out + (t + j0) * ostr;
#pragma unroll
                for (int j = 0; j < N; ++j, o += ostr) {
                    const Pack<T, 2> po = from_f2<T>(y[j]);
                    if (a.pair) {
                        if (live[0]) st_pack<2>(o, po);
                    } else {
                        if (live[0]) o[0] = po.v[0];
                        if (live[1]) o[1] = po.v[1];
                    }
                }
            }
        };
        const int64_t at = blk.t0 + t;
        if (t + TK < stop) {  // no sequence ends here
#pragma unroll 1
            for (int j = 0; j < TK; j += kPairBatch) tokens(Count<kPairBatch>{}, j);
        } else {
            const int tl = len - t < TK ? len - t : TK;
            int j = 0;
            while (j < tl) {
                if (at + j >= sq.end) {  // packed: the next sequence begins
                    const int64_t q = sq.q;
                    seq_next(a.d.offsets, a.d.nseq, at + j, &sq);
                    stop = seq_stop(sq, blk.t0, len);
                    if (sq.q != q) {
                        initial();
                        has_reset = true;
                    }
                }
                const int je = sq.end > at + j && sq.end < at + tl ? (int)(sq.end - at) : tl;
#pragma unroll 1
                for (; j < je; ++j) tokens(Count<1>{}, j);
                if (OUTPUT && a.final_state && at + j == sq.end) {
#pragma unroll
                    for (int k = 0; k < 2; ++k)
                        if (live[k])
                            store_states<SPT>(a.final_state + (sq.q * a.d.channels + c + k) * n, 0, n,
                                              h[k]);
                }
            }
        }
        stage = stage + 1 < ST ? stage + 1 : 0;
        buf ^= 1;
    }
    copy_wait<0>();
    if (SUMMARY) {
#pragma unroll
        for (int k = 0; k < 2; ++k)
            if (live[k]) {
                store_row<SPT>(a.carry + carry_at + k * SPT, h[k]);
                a.dsum[(blk.row * a.nchunks + blk.chunk) * a.d.channels + c + k] = k ? dsum.y : dsum.x;
            }
        if (tid == 0 && blk.c0 == 0) a.reset[blk.row * a.nchunks + blk.chunk] = has_reset;
    }
}

constexpr int kLanesThreads = 64, kLanesTile = 16, kLanesBatch = 8;

template <class T, int SPT, int SL, int PASS>
struct ScanLanesSmem {
    static constexpr bool OUTPUT = PASS == SCAN_OUTPUT;
    static constexpr int CT = kLanesThreads / SL, NP = SPT * SL;
    static constexpr int kStages = 3, kRaw = kLanesTile * CT, kTensors = OUTPUT ? 3 : 2;
    static constexpr int kBC = kLanesTile * NP * (OUTPUT ? 2 : 1);  // floats of a buffer
    static constexpr int kBytesRaw = kStages * kTensors * kRaw * (int)sizeof(T);
    static constexpr int kBytes = kBytesRaw + 2 * kBC * 4;
};

// SL lanes share a channel, SPT states each: more than 16 states, or enough channels to fill the
// GPU without cutting time when each has more threads.  Tiles of 16 tokens in two batches of 8.
// In a batch each lane prepares and finishes its own 8 / SL tokens (softplus, gate, store); d and
// d u are broadcast from the token's lane, and the partial sums over states handed back to it.
template <class T, int SPT, int SL, int PASS, bool FAST>
__global__ void __launch_bounds__(kLanesThreads) k_scan_lanes(const ScanArgs a) {
    using M = ScanLanesSmem<T, SPT, SL, PASS>;
    constexpr int NT = kLanesThreads, CT = M::CT, CL = 32 / SL, NP = M::NP, TK = kLanesTile;
    constexpr int ST = M::kStages, N = kLanesBatch, OWN = N / SL;
    constexpr bool SUMMARY = PASS == SCAN_SUMMARY, OUTPUT = PASS == SCAN_OUTPUT;
    extern __shared__ float4 smem4[];
    T* raw = reinterpret_cast<T*>(smem4);  // [stage][tensor][token][channel]
    float* sbc = reinterpret_cast<float*>(reinterpret_cast<char*>(smem4) + M::kBytesRaw);

    const int n = (int)a.d.states, tid = (int)threadIdx.x, lane = tid & 31;
    const bool packed = a.d.offsets != nullptr, gate = OUTPUT && a.d.z.data != nullptr;
    const int64_t nch = SUMMARY ? a.nchunks - 1 : a.nchunks;
    const int64_t mains = a.rows * nch * a.ctiles * a.d.groups;
    if (OUTPUT && (int64_t)blockIdx.x >= mains) return scan_empty(a, blockIdx.x - mains);
    const ScanBlock blk = scan_block(a, blockIdx.x, nch, CT);
    SeqAt sq = seq_at(a.d.offsets, a.d.nseq, a.d.length, blk.row, blk.t0);
    const int width = (int)(blk.cend - blk.c0 < CT ? blk.cend - blk.c0 : CT);  // channels here
    const int sl = lane / CL, ch = lane % CL, lc = (tid >> 5) * CL + ch, s0 = sl * SPT;
    const int len = (int)(blk.t1 - blk.t0);
    const int64_t c = blk.c0 + lc;
    const bool live = lc < width;
    // token t0 of the chunk; from here on tokens count from t0
    const T* src[3] = {row_of<T>(a.d.u, packed, blk.row) + blk.t0 * a.d.u.tok_stride + blk.c0,
                       row_of<T>(a.d.delta, packed, blk.row) + blk.t0 * a.d.delta.tok_stride + blk.c0,
                       gate ? row_of<T>(a.d.z, packed, blk.row) + blk.t0 * a.d.z.tok_stride + blk.c0
                            : nullptr};
    const int64_t str[3] = {a.d.u.tok_stride, a.d.delta.tok_stride, a.d.z.tok_stride};
    const T* Bp = row_of<T>(a.d.B, packed, blk.row) + blk.t0 * a.d.B.tok_stride + blk.g * n;
    const T* Cp = row_of<T>(a.d.C, packed, blk.row) + blk.t0 * a.d.C.tok_stride + blk.g * n;

    auto copy = [&](int t, int stage) {  // the tile at t
#pragma unroll
        for (int k = 0; k < M::kTensors; ++k) {
            if (k == 2 && !gate) break;
            copy_tile<T, TK, CT, NT, FAST>(raw + (stage * M::kTensors + k) * M::kRaw, src[k], str[k], t, len,
                                     width, a.vec);
        }
        copy_commit();
    };
    RowsAhead<T, TK, NP, NT, OUTPUT, FAST> bc;
    auto fetch = [&](int t) {
        bc.fetch(Bp, a.d.B.tok_stride, Cp, a.d.C.tok_stride, t, len, n);
    };
    auto stage_bc = [&](int buf) { bc.stage(sbc + buf * M::kBC); };
#pragma unroll
    for (int i = 0; i < ST - 1; ++i) copy(i * TK, i);
    fetch(0);

    float2 A2[SPT / 2], h[SPT / 2];
    load_states<SPT>(live ? a.d.A + c * n : nullptr, s0, n, A2);
#pragma unroll
    for (int i = 0; i < SPT / 2; ++i) A2[i] = mul2(A2[i], splat(kLog2e));
    const float bias = live && a.d.delta_bias ? a.d.delta_bias[c] : 0.f;
    const float D = OUTPUT && live && a.d.D ? a.d.D[c] : 0.f;
    auto initial = [&]() {
        load_states<SPT>(live && a.d.initial_state
                             ? a.d.initial_state + (sq.q * a.d.channels + c) * n : nullptr, s0, n, h);
    };
    const int64_t carry_at = ((blk.row * a.nchunks + blk.chunk) * a.d.channels + c) * NP;
    bool has_reset = starts_at(sq, blk.t0);
    if (has_reset)
        initial();
    else if (!SUMMARY && live)
        load_row<SPT>(a.carry + carry_at + s0, h);
    else
        load_states<SPT>(nullptr, 0, SPT, h);
    float dsum = 0.f;
    stage_bc(0);
    fetch(TK);
    T* out = OUTPUT ? const_cast<T*>(row_of<T>(a.out, packed, blk.row)) + blk.t0 * a.out.tok_stride + c
                    : nullptr;
    const int64_t ostr = a.out.tok_stride;

    int stage = 0, buf = 0, stop = seq_stop(sq, blk.t0, len);
    for (int t = 0; t < len; t += TK) {
        copy_wait<ST - 2>();
        __syncthreads();  // this tile has landed; the last one's buffers are free
        copy(t + (ST - 1) * TK, stage >= 1 ? stage - 1 : ST - 1);
        stage_bc(buf ^ 1);
        fetch(t + 2 * TK);
        static_assert(kLanesTile == kScanTile, "states are written once a tile");
        if (PASS == SCAN_TILES && live) {
            const int64_t tiles = (a.d.length + kScanTile - 1) / kScanTile;
            store_row<SPT>(
                a.tiles + ((blk.row * tiles + (blk.t0 + t) / kScanTile) * a.d.channels + c) * NP + s0, h);
        }
        const T* ru = raw + stage * M::kTensors * M::kRaw + lc;
        const T* rd = ru + M::kRaw;
        const T* rz = rd + M::kRaw;
        const float* sB = sbc + buf * M::kBC + s0;
        const float* sC = sB + TK * NP;
        // the recurrence over one token; the sum over this lane's states
        auto step = [&](int j, float d, float du) {
            const float2 dd = splat(d), dv = splat(du);
            float2 acc[2] = {};
#pragma unroll
            for (int i = 0; i < SPT / 4; ++i) {
                const float4 b4 = *reinterpret_cast<const float4*>(sB + j * NP + 4 * i);
                float4 c4;
                if (OUTPUT) c4 = *reinterpret_cast<const float4*>(sC + j * NP + 4 * i);
#pragma unroll
                for (int p = 0; p < 2; ++p) {
                    float2& hh = h[2 * i + p];
                    hh = fma2(decay2(dd, A2[2 * i + p]), hh,
                              mul2(dv, p ? make_float2(b4.z, b4.w) : make_float2(b4.x, b4.y)));
                    if (!FAST) {
                        if (s0 + 4 * i + 2 * p >= n) hh.x = 0.f;
                        if (s0 + 4 * i + 2 * p + 1 >= n) hh.y = 0.f;
                    }
                    if (OUTPUT)
                        acc[p] = fma2(p ? make_float2(c4.z, c4.w) : make_float2(c4.x, c4.y), hh, acc[p]);
                }
            }
            const float2 y = add2(acc[0], acc[1]);
            return y.x + y.y;
        };
        const int64_t at = blk.t0 + t;
        if (t + TK < stop) {  // no sequence ends here
#pragma unroll 1
            for (int j0 = 0; j0 < TK; j0 += N) {
                float2 d[(OWN + 1) / 2], du[(OWN + 1) / 2], uu[(OWN + 1) / 2];  // pairs of own tokens
                const int own = j0 + sl;  // tokens own, own + SL, ...: apart in shared memory's banks
#pragma unroll
                for (int j = 0; j < OWN; ++j) {
                    (j & 1 ? d[j / 2].y : d[j / 2].x) = to_f(rd[(own + j * SL) * CT]) + bias;
                    (j & 1 ? uu[j / 2].y : uu[j / 2].x) = to_f(ru[(own + j * SL) * CT]);
                }
                if (OWN == 1) d[0].y = uu[0].y = 0.f;
#pragma unroll
                for (int j = 0; j < (OWN + 1) / 2; ++j) {
                    if (a.d.softplus) d[j] = softplus2(d[j]);
                    du[j] = mul2(d[j], uu[j]);
                }
                float y[N];
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    const int k = j / SL, from = j % SL * CL + ch;
                    const float dj = __shfl_sync(0xffffffffu, k & 1 ? d[k / 2].y : d[k / 2].x, from);
                    const float duj = __shfl_sync(0xffffffffu, k & 1 ? du[k / 2].y : du[k / 2].x, from);
                    if (SUMMARY) dsum += dj;
                    y[j] = step(j0 + j, dj, duj);
                }
                if (OUTPUT) {
#pragma unroll
                    for (int w = 1, cnt = N / 2; w < SL; w *= 2, cnt /= 2) {
                        const bool up = sl & w;
#pragma unroll
                        for (int j = 0; j < N / 2; ++j) {
                            if (j < cnt) {
                                const float send = up ? y[2 * j] : y[2 * j + 1];
                                const float keep = up ? y[2 * j + 1] : y[2 * j];
                                y[j] = keep + __shfl_xor_sync(0xffffffffu, send, w * CL);
                            }
                        }
                    }
                    T* o = out + (t + own) * ostr;
#pragma unroll
                    for (int j = 0; j < OWN; ++j, o += SL * ostr) {
                        float v = fmaf(D, j & 1 ? uu[j / 2].y : uu[j / 2].x, y[j]);
                        if (gate) {
                            const float z = to_f(rz[(own + j * SL) * CT]);
                            v *= z * sigmoid(z);
                        }
                        if (live) *o = from_f<T>(v);
                    }
                }
            }
        } else {  // token by token, every lane preparing it
            const int tl = len - t < TK ? len - t : TK;
            int j = 0;
            while (j < tl) {
                if (at + j >= sq.end) {  // packed: the next sequence begins
                    const int64_t q = sq.q;
                    seq_next(a.d.offsets, a.d.nseq, at + j, &sq);
                    stop = seq_stop(sq, blk.t0, len);
                    if (sq.q != q) {
                        initial();
                        has_reset = true;
                    }
                }
                const int je = sq.end > at + j && sq.end < at + tl ? (int)(sq.end - at) : tl;
#pragma unroll 1
                for (; j < je; ++j) {
                    float d = to_f(rd[j * CT]) + bias;
                    const float uj = to_f(ru[j * CT]);
                    if (a.d.softplus) d = softplus(d);
                    if (SUMMARY) dsum += d;
                    float y = step(j, d, d * uj);
                    if (OUTPUT) {
#pragma unroll
                        for (int w = 1; w < SL; w *= 2) y += __shfl_xor_sync(0xffffffffu, y, w * CL);
                        y = fmaf(D, uj, y);
                        if (gate) {
                            const float z = to_f(rz[j * CT]);
                            y *= z * sigmoid(z);
                        }
                        if (live && sl == 0) out[(t + j) * ostr] = from_f<T>(y);
                    }
                }
                if (OUTPUT && a.final_state && at + j == sq.end && live)
                    store_states<SPT>(a.final_state + (sq.q * a.d.channels + c) * n, s0, n, h);
            }
        }
        stage = stage + 1 < ST ? stage + 1 : 0;
        buf ^= 1;
    }
    copy_wait<0>();
    if (SUMMARY) {
        if (live) {
            store_row<SPT>(a.carry + carry_at + s0, h);
            if (sl == 0) a.dsum[(blk.row * a.nchunks + blk.chunk) * a.d.channels + c] = dsum;
        }
        if (tid == 0 && blk.c0 == 0) a.reset[blk.row * a.nchunks + blk.chunk] = has_reset;
    }
}

// A state h carried over a chunk that takes it to e^2 h + local.  Steps below zero make states grow,
// and e^2 may then be infinite where the product is not: it is multiplied in two halves, and a state
// of 0 has not grown.  cut: the chunk does not go on from h.
__device__ __forceinline__ float carried(float e, float h, float local, bool cut) {
    const float grown = fmaf(e, e * h, local);
    return cut | (h == 0.f) ? local : grown;
}

// Few threads and a chain of chunks: small blocks on many SMs, and many chunks loaded at once.
constexpr int kCarryThreads = 64, kCarryAhead = 16;

// Pass 2: along the chunks of every (row, channel, state); the state after a chunk that a
// sequence starts in does not depend on what came before.
template <int NP>
__global__ void __launch_bounds__(kCarryThreads) k_scan_carry(const ScanArgs a) {
    const int64_t i = (int64_t)blockIdx.x * kCarryThreads + threadIdx.x, per = a.d.channels * NP;
    if (i >= a.rows * per) return;
    const int64_t row = i / per, cs = i - row * per, c = cs / NP;
    const int s = (int)(cs - c * NP), n = (int)a.d.states;
    const float A2 = s < n ? a.d.A[c * n + s] * kLog2e : 0.f;
    float* carry = a.carry + row * a.nchunks * per + cs;
    const float* dsum = a.dsum + row * a.nchunks * a.d.channels + c;
    const int* reset = a.reset + row * a.nchunks;
    float h = 0.f;
    constexpr int U = kCarryAhead;
    for (int64_t k = 0; k < a.nchunks; k += U) {
        float local[U], sum[U];
        int cut[U];
#pragma unroll
        for (int j = 0; j < U; ++j) {  // no branches: the loads have to be in flight together
            const int64_t i = k + j < a.nchunks ? k + j : a.nchunks - 1;
            local[j] = carry[i * per];
            sum[j] = dsum[i * a.d.channels];
            cut[j] = reset[i];
        }
#pragma unroll
        for (int j = 0; j < U; ++j) sum[j] = ex2(0.5f * A2 * sum[j]);
#pragma unroll
        for (int j = 0; j < U; ++j) {
            if (k + j >= a.nchunks) break;
            carry[(k + j) * per] = h;
            h = carried(sum[j], h, local[j], cut[j]);
        }
    }
}

// SL 0: k_scan, otherwise k_scan_lanes.
template <class T, int SPT, int SL, int PASS, bool FAST>
cudaError_t scan_kernel(const ScanArgs& a, int64_t blocks, cudaStream_t s) {
    static LaunchCache cache;
    LaunchGeom geo;
    if constexpr (SL == 0) {
        constexpr int bytes = ScanPairSmem<T, SPT, PASS>::kBytes;
        const cudaError_t e = cache.get([](int dev, LaunchGeom* g) {
            return setup_persistent(k_scan<T, SPT, PASS, FAST>, kPairThreads, bytes, dev, g);
        }, &geo);
        if (e != cudaSuccess) return e;
        k_scan<T, SPT, PASS, FAST><<<(unsigned)blocks, kPairThreads, bytes, s>>>(a);
    } else {
        constexpr int bytes = ScanLanesSmem<T, SPT, SL, PASS>::kBytes;
        const cudaError_t e = cache.get([](int dev, LaunchGeom* g) {
            return setup_persistent(k_scan_lanes<T, SPT, SL, PASS, FAST>, kLanesThreads, bytes, dev, g);
        }, &geo);
        if (e != cudaSuccess) return e;
        k_scan_lanes<T, SPT, SL, PASS, FAST><<<(unsigned)blocks, kLanesThreads, bytes, s>>>(a);
    }
    return cudaGetLastError();
}

// Passes 1 and 2 where time is cut, then the pass that was asked for.
template <class T, int SPT, int SL, int PASS, bool FAST>
cudaError_t scan_launch(const ScanArgs& a, cudaStream_t s) {
    const int64_t tiles = a.ctiles * a.d.groups;
    const bool empties = PASS == SCAN_OUTPUT && a.final_state && (a.d.offsets || a.d.length == 0);
    const int64_t blocks = a.rows * a.nchunks * tiles + (empties ? a.d.nseq : 0);
    if (blocks < 1) return cudaSuccess;
    if (blocks > INT32_MAX) return cudaErrorInvalidValue;
    if (a.nchunks > 1) {
        const cudaError_t e = scan_kernel<T, SPT, SL, SCAN_SUMMARY, FAST>(
            a, a.rows * (a.nchunks - 1) * tiles, s);
        if (e != cudaSuccess) return e;
        constexpr int NP = SPT * (SL ? SL : 1);
        k_scan_carry<NP><<<(unsigned)((a.rows * a.d.channels * NP + kCarryThreads - 1) / kCarryThreads),
                           kCarryThreads, 0, s>>>(a);
    }
    return scan_kernel<T, SPT, SL, PASS, FAST>(a, blocks, s);
}

// Whether NP states of type T can be whole 16-byte accesses.
template <class T>
constexpr bool whole_states(int np) {
    return np * sizeof(T) % 16 == 0;
}
template <class T, int SPT, int SL, int PASS>
cudaError_t scan_fast(const ScanArgs& a, cudaStream_t s) {
    constexpr int NP = SPT * (SL ? SL : 1);
    if constexpr (whole_states<T>(NP)) {
        if (a.d.states == NP && a.vec >= 16 && a.wide) return scan_launch<T, SPT, SL, PASS, true>(a, s);
    }
    return scan_launch<T, SPT, SL, PASS, false>(a, s);
}
template <class T, int PASS>
cudaError_t scan_run(ScanArgs a, cudaStream_t s) {
    const bool packed = a.d.offsets != nullptr;
    const int64_t dg = a.d.channels / a.d.groups;
    auto rows_on = [&](const fft_seq& q, int64_t bytes) {
        return !q.data || (aligned_to(q.data, bytes) && q.tok_stride * sizeof(T) % bytes == 0 &&
                           (packed || q.seq_stride * sizeof(T) % bytes == 0));
    };
    auto all_on = [&](int64_t bytes) {
        return dg * sizeof(T) % bytes == 0 && rows_on(a.d.u, bytes) && rows_on(a.d.delta, bytes) &&
               rows_on(a.d.z, bytes);
    };
    a.vec = all_on(16) ? 16 : (all_on(4) ? 4 : 0);
    a.wide = rows_on(a.d.B, 16) && rows_on(a.d.C, 16) && a.d.states * sizeof(T) % 16 == 0;
    a.pair = dg % 2 == 0 && rows_on(a.out, 2 * sizeof(T));
    // nine to twelve states: the backward pass keeps rows of 16
    if (PASS == SCAN_OUTPUT && a.sl == 0 && scan_out_np(a.d.states) == 12)
        return scan_fast<T, 12, 0, SCAN_OUTPUT>(a, s);
    switch (scan_np(a.d.states) * 100 + a.sl) {
        case 400: return scan_fast<T, 4, 0, PASS>(a, s);
        case 800: return scan_fast<T, 8, 0, PASS>(a, s);
        case 802: return scan_fast<T, 4, 2, PASS>(a, s);
        case 1600: return scan_fast<T, 16, 0, PASS>(a, s);
        case 1602: return scan_fast<T, 8, 2, PASS>(a, s);
        case 3202: return scan_fast<T, 16, 2, PASS>(a, s);
        case 6404: return scan_fast<T, 16, 4, PASS>(a, s);
        case 12808: return scan_fast<T, 16, 8, PASS>(a, s);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace gbfft
