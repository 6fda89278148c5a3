// Linear attention with a decay for each head and token, in chunks of 64 tokens.
//
// With G[r] the sum of the log decays from the chunk's first token to r and S the state before the
// chunk, the recurrence S[t] = exp(g[t]) S[t-1] + y[t] z[t]^T is, over a chunk,
//   out = (P o (x y^T)) z + exp(G) x S,   P[r][c] = exp(G[r] - G[c]) for c <= r
//   S'  = exp(G[last]) S + sum_c exp(G[last] - G[c]) y[c] z[c]^T
// and with time reversed (P for c >= r, exp(G[last] - G) and exp(G) change places) the same form
// gives the gradients: dq = (dout, v, k), dv = reversed (k, q, dout), dk = reversed (v, dout, q).
// All factors are at most 1 since a decay is at most 0, so nothing overflows on the way.
//
// Matrix units multiply bfloat16 with float32 sums, so values of more bits go in pieces of 8 bits,
// x = x0 + x1 + x2 with |x1| <= 2^-9 |x|, and products of pieces i and j are left out where i + j is
// beyond the order that the result needs: float32 has three pieces (order 2: errors of 2^-24),
// float16 two, bfloat16 one.  The state is float32 and stays float32: what is added to it goes in
// three pieces for every type.  Weighted scores and the state that x is multiplied with are rounded
// to one piece for bfloat16 outputs (each such rounding is 2^-9 of one term, as that of the output
// itself), to two in the gradients, whose products with q and k are summed along the sequence for
// the decay's gradient, and for float16, to three for float32.
//
// A block keeps 16 columns of S^T per warp in registers (S^T, since the accumulators of one product
// are then the operand of the next) and walks along a segment of time; rows of x, y and z wait in
// shared memory, the next chunk's under way where two fit.
//
// This kernel takes what the tcgen05 one does not: float32, float16, rows off 16-byte boundaries, dk
// above 128.  Measured: packed 10007 tokens of 6 heads of 40 x 72 float32 191 to 203 us; gradients of packed 4001
// tokens of 8 heads of 64 x 96 float16 403 to 420 us (250 and 480 with columns and warps beyond the sizes at work); 1 x 16384 tokens of 16 heads of 128 x 128 bfloat16 364 us,
// where the tensor pipe was busy 15% at 1.3 instructions a cycle: bound by latency at 8 warps of 255
// registers to an SM.
#pragma once

#include <type_traits>

#include "launch_cache.cuh"
#include "linattn.h"

namespace gbfft {
namespace {

using bf16 = __nv_bfloat16;

// ---- pieces ---------------------------------------------------------------------------------

// Two neighbouring values (along the summed index) as they lie in memory.
template <class T> struct PairOf { using type = uint32_t; };
template <> struct PairOf<float> { using type = float2; };
template <class T> using Pair = typename PairOf<T>::type;

__device__ __forceinline__ float2 values(float2 p, float) { return p; }
__device__ __forceinline__ float2 values(uint32_t p, bf16) {
    return make_float2(__uint_as_float(p << 16), __uint_as_float(p & 0xffff0000u));
}
__device__ __forceinline__ float2 values(uint32_t p, __half) {
    return __half22float2(*reinterpret_cast<const __half2*>(&p));
}
__device__ __forceinline__ uint32_t bf16x2(float2 v) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(v.y), "f"(v.x));
    return r;
}
// What a piece leaves over; nothing where the piece is not finite.
__device__ __forceinline__ float rest(float v, float piece) {
    return fabsf(piece) < INFINITY ? v - piece : 0.f;
}
template <int N>
__device__ __forceinline__ void split(float2 v, uint32_t (&p)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
        p[i] = bf16x2(v);
        if (i + 1 < N) {
            const float2 h = values(p[i], bf16());
            v = make_float2(rest(v.x, h.x), rest(v.y, h.y));
        }
    }
}

template <class T> constexpr int kPieces = std::is_same<T, bf16>::value ? 1 : (std::is_same<T, __half>::value ? 2 : 3);
template <class T>
__device__ __forceinline__ void pieces(Pair<T> v, uint32_t (&p)[kPieces<T>]) {
    if constexpr (std::is_same<T, bf16>::value) {
        p[0] = v;
    } else {
        split<kPieces<T>>(values(v, T()), p);
    }
}
// Four pairs of a 16 x 16 block.
template <class T>
__device__ __forceinline__ void block_pieces(const Pair<T> (&v)[4], uint32_t (&p)[kPieces<T>][4]) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        uint32_t q[kPieces<T>];
        pieces<T>(v[k], q);
#pragma unroll
        for (int i = 0; i < kPieces<T>; ++i) p[i][k] = q[i];
    }
}

// ---- blocks of 16 x 16 values in shared memory ----------------------------------------------
//
// Thread l holds of a block B (rows: outputs of the product, columns: the summed index) the pairs
// f[0] = B[l/4][2(l%4)], f[1] = B[l/4 + 8][..], f[2], f[3]: the same at columns + 8.  That is the
// first operand of an m16n8k16 product, and {f[t], f[t + 2]} its second operand for the rows 8t.

__device__ __forceinline__ uint32_t smem_of(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

template <class T, bool TRANS>
__device__ __forceinline__ void ldmatrix(const T* p, uint32_t (&f)[4]) {
    if constexpr (TRANS)
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                     : "=r"(f[0]), "=r"(f[1]), "=r"(f[2]), "=r"(f[3]) : "r"(smem_of(p)) : "memory");
    else
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                     : "=r"(f[0]), "=r"(f[1]), "=r"(f[2]), "=r"(f[3]) : "r"(smem_of(p)) : "memory");
}
// Rows of the block are rows of the tile, from (r, c).
template <class T>
__device__ __forceinline__ void load_rows(const T* s, int stride, int r, int c, Pair<T> (&f)[4]) {
    const int l = (int)threadIdx.x & 31;
    if constexpr (sizeof(T) == 2) {
        ldmatrix<T, false>(s + (r + (l & 15)) * stride + c + (l >> 4) * 8, f);
    } else {
        const T* p = s + (r + l / 4) * stride + c + 2 * (l & 3);
        f[0] = *reinterpret_cast<const float2*>(p);
        f[1] = *reinterpret_cast<const float2*>(p + 8 * stride);
        f[2] = *reinterpret_cast<const float2*>(p + 8);
        f[3] = *reinterpret_cast<const float2*>(p + 8 * stride + 8);
    }
}
// Rows of the block are columns of the tile: the summed index is the tile's row, from (r, c).
template <class T>
__device__ __forceinline__ void load_cols(const T* s, int stride, int r, int c, Pair<T> (&f)[4]) {
    const int l = (int)threadIdx.x & 31;
    if constexpr (sizeof(T) == 2) {
        ldmatrix<T, true>(s + (r + (l & 7) + (l >> 4) * 8) * stride + c + ((l >> 3) & 1) * 8, f);
    } else {
        const T* p = s + (r + 2 * (l & 3)) * stride + c + l / 4;
        f[0] = make_float2(p[0], p[stride]);
        f[1] = make_float2(p[8], p[stride + 8]);
        f[2] = make_float2(p[8 * stride], p[9 * stride]);
        f[3] = make_float2(p[8 * stride + 8], p[9 * stride + 8]);
    }
}
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// d += a b with a in NA pieces and b in NB, products of pieces i and j up to i + j = ORDER, the small
// ones first.  Where all 24 bits are wanted the products are summed by themselves and then added: the
// units cut their sums off where float32 additions round, and a chain of a hundred would lose 4 bits.
template <int NA, int NB, int ORDER>
__device__ __forceinline__ void mma_pieces(float (&d)[4], const uint32_t (&a)[NA][4], const uint32_t (&b)[NB][4], int h) {
    float t[4] = {};
    float(&sum)[4] = NB == 3 ? t : d;
#pragma unroll
    for (int u = NA - 1; u >= 0; --u)
#pragma unroll
        for (int v = NB - 1; v >= 0; --v)
            if (u + v <= ORDER) mma(sum, a[u], b[v][h], b[v][h + 2]);
    if (NB == 3) {
#pragma unroll
        for (int k = 0; k < 4; ++k) d[k] += t[k];
    }
}

// ---- sizes ----------------------------------------------------------------------------------

template <class T, int DX, int WARPS, bool BWD>
struct AttnShape {
    static constexpr int kThreads = WARPS * 32, kZ = WARPS * 16, kC = kAttnChunk;
    static constexpr int kNP = kPieces<T>;
    // pieces of weighted scores and of the state as an operand, less one
    static constexpr int kOrder = kNP == 1 ? (BWD ? 1 : 0) : kNP - 1;
    static constexpr int kXS = DX + 8, kZS = kZ + (sizeof(T) == 4 ? 4 : 8), kPS = kC + 8;
    static constexpr int kTile = kC * (2 * kXS + (BWD ? 2 : 1) * kZS);  // values of a stage
    static constexpr size_t kFixed = (size_t)(kOrder + 1) * kC * kPS * 2 + (BWD ? 2 * WARPS * kC * 4 : 0);
    static constexpr size_t kSmall = 2 * (4 * kC + 4) * 4 + 512;  // static: decays, sums over warps
    static constexpr int kStages = kFixed + 2 * kTile * sizeof(T) + kSmall <= 227 * 1024 ? 2 : 1;
    static constexpr size_t kBytes = kFixed + (size_t)kStages * kTile * sizeof(T);
    static constexpr int kBlocks = kBytes + kSmall + 1024 <= 114 * 1024 && DX <= 128 ? 2 : 1;
};

// The decays of a chunk: G in two floats (its log2, 48 bits, as differences of large sums are
// wanted), the factors of the state in the outputs and of a token in the state.
struct Decays {
    float hi[kAttnChunk], lo[kAttnChunk], inter[kAttnChunk], update[kAttnChunk];
    float total, total_log2;
};

// Copies `count` rows of `dim` values into rows of D, zeros behind them.
template <class T, int D, int THREADS>
__device__ __forceinline__ void load_tile(T* s, int stride, const T* g, int64_t tok, int count,
                                          int dim, int vec) {
    if (vec == 16) {
        constexpr int V = 16 / sizeof(T), N = D / V;
        for (int i = (int)threadIdx.x; i < kAttnChunk * N; i += THREADS) {
            const int r = i / N, c = (i % N) * V;
            const bool in = r < count && c < dim;
            copy16(s + r * stride + c, in ? g + r * tok + c : g, in);
        }
    } else if (vec == 4) {
        constexpr int V = 4 / sizeof(T), N = D / V;
        for (int i = (int)threadIdx.x; i < kAttnChunk * N; i += THREADS) {
            const int r = i / N, c = (i % N) * V;
            const bool in = r < count && c < dim;
            copy4(s + r * stride + c, in ? g + r * tok + c : g, in);
        }
    } else {
        for (int i = (int)threadIdx.x; i < kAttnChunk * D; i += THREADS) {
            const int r = i / D, c = i % D;
            s[r * stride + c] = r < count && c < dim ? g[r * tok + c] : from_f<T>(0.f);
        }
    }
}

template <class T>
__device__ __forceinline__ const T* rows_at(const AttnRows& r, int64_t row, int64_t head) {
    return static_cast<const T*>(r.data) + row * r.seq + (head / r.share) * r.head;
}

// The chunk's sums and factors from the log decays of tokens 2 lane and 2 lane + 1: one warp.
__device__ __forceinline__ void make_decays(Decays& dc, float g0, float g1, bool reverse, float inter, float update) {
    const int lane = (int)threadIdx.x & 31;
    const Two d0 = log2_decay(g0), own = add(d0, log2_decay(g1));
    Two sum = own;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const Two v = {__shfl_up_sync(0xffffffffu, sum.hi, o), __shfl_up_sync(0xffffffffu, sum.lo, o)};
        if (lane >= o) sum = add(v, sum);
    }
    const Two all = {__shfl_sync(0xffffffffu, sum.hi, 31), __shfl_sync(0xffffffffu, sum.lo, 31)};
    Two before = {__shfl_up_sync(0xffffffffu, sum.hi, 1), __shfl_up_sync(0xffffffffu, sum.lo, 1)};
    if (lane == 0) before = {0.f, 0.f};
    const Two G[2] = {add(before, d0), sum};
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const float gone = ex2(G[k].hi), left = ex2((all.hi - G[k].hi) + (all.lo - G[k].lo));
        dc.hi[2 * lane + k] = G[k].hi;
        dc.lo[2 * lane + k] = G[k].lo;
        dc.inter[2 * lane + k] = (reverse ? left : gone) * inter;
        dc.update[2 * lane + k] = (reverse ? gone : left) * update;
    }
    if (lane == 0) dc.total = ex2(all.hi), dc.total_log2 = all.hi;
}

// The part of a segment that belongs to one sequence.
struct Part {
    int64_t begin, end, seq;
    bool first, last;  // begins with the sequence's first token, ends with its last
};
__device__ __forceinline__ Part part_of(const AttnArgs& a, int64_t row, int64_t t0, int64_t t1,
                                        int64_t at) {
    const SeqAt s = seq_at(a.offsets, a.nseq, a.length, row, at);
    Part p;
    p.seq = s.q;
    // offsets of any kind: the part holds token `at` and stays in the segment
    p.begin = s.begin > at ? at : (s.begin < t0 ? t0 : s.begin);
    p.end = s.end <= at ? at + 1 : (s.end > t1 ? t1 : s.end);
    p.first = p.begin == 0 || (s.begin >= t0 && s.begin <= at);
    p.last = p.end == a.length || (s.end <= t1 && s.end > at);
    return p;
}

template <class T, int DX, int WARPS, bool BWD>
__global__ void __launch_bounds__(WARPS * 32, AttnShape<T, DX, WARPS, BWD>::kBlocks)
    k_linattn(const AttnArgs a) {
    using Shape = AttnShape<T, DX, WARPS, BWD>;
    constexpr int C = kAttnChunk, THREADS = Shape::kThreads, Z = Shape::kZ, NP = Shape::kNP;
    constexpr int ORDER = Shape::kOrder, PO = ORDER + 1, XS = Shape::kXS, ZS = Shape::kZS, PS = Shape::kPS;
    constexpr int NX = DX / 8;
    extern __shared__ uint4 dynamic[];
    bf16* weighted = reinterpret_cast<bf16*>(dynamic);  // [piece][row][column]
    float* sums = reinterpret_cast<float*>(weighted + PO * C * PS);  // BWD: [2][warp][row]
    T* tiles = reinterpret_cast<T*>(sums + (BWD ? 2 * WARPS * C : 0));
    __shared__ Decays decays[2];
    __shared__ float warp_sums[WARPS], diagonal[BWD ? C : 1];

    const int tid = (int)threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int lr = lane >> 2, lc = 2 * (lane & 3);
    int64_t b = blockIdx.x;
    const int64_t zt = b % a.ztiles;
    b /= a.ztiles;
    const int64_t head = b % a.heads;
    b /= a.heads;
    const int64_t seg = b % a.nsegments, row = b / a.nsegments;
    const int64_t t0 = seg * a.segment, t1 = t0 + a.segment < a.length ? t0 + a.segment : a.length;
    const int z0 = (int)zt * Z, dz = (int)a.dz - z0 < Z ? (int)a.dz - z0 : Z, dx = (int)a.dx;
    const bool reverse = a.reverse, summary = a.summary;
    const bool busy = warp * 16 < dz;  // this warp has columns

    const T* px = summary ? nullptr : rows_at<T>(a.x, row, head);
    const T* py = rows_at<T>(a.y, row, head);
    const T* pz = rows_at<T>(a.z, row, head) + z0;
    const T* pp = BWD && a.partner.data ? rows_at<T>(a.partner, row, head) + z0 : nullptr;
    const T* pg = static_cast<const T*>(a.decay.data) + row * a.decay.seq_stride + head;

    auto stage = [&](int k) { return tiles + (Shape::kStages == 2 ? k * Shape::kTile : 0); };
    auto fetch = [&](int k, int64_t t, int count) {
        T* s = stage(k);
        if (!summary) load_tile<T, DX, THREADS>(s, XS, px + t * a.x.tok, a.x.tok, count, dx, a.x.vec);
        load_tile<T, DX, THREADS>(s + C * XS, XS, py + t * a.y.tok, a.y.tok, count, dx, a.y.vec);
        load_tile<T, Z, THREADS>(s + 2 * C * XS, ZS, pz + t * a.z.tok, a.z.tok, count, dz, a.z.vec);
        if (BWD && pp && !summary)
            load_tile<T, Z, THREADS>(s + 2 * C * XS + C * ZS, ZS, pp + t * a.partner.tok, a.partner.tok,
                                     count, dz, a.partner.vec);
        copy_commit();
    };

    float S[NX][4];  // S^T: columns warp * 16 + lr (and + 8) of the tile, rows 8 j + lc and + 1
    auto clear = [&] {
#pragma unroll
        for (int j = 0; j < NX; ++j)
#pragma unroll
            for (int k = 0; k < 4; ++k) S[j][k] = 0.f;
    };
    // f(register, x, z) of every value of the state that this thread holds
    auto each_state = [&](auto f) {
#pragma unroll
        for (int j = 0; j < NX; ++j)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int x = 8 * j + lc + (k & 1), z = warp * 16 + lr + (k & 2) * 4;
                if (x < dx && z < dz) f(S[j][k], x * a.state_x + (z0 + z) * a.state_z);
            }
    };
    const int64_t carry_at =
        (((row * a.nsegments + seg) * a.heads + head) * a.ztiles + zt) * (DX * Z) + tid * 4;

    // The parts of the segment, in the direction of the pass; a summary takes the one that
    // reaches the next segment.
    int64_t at = summary == reverse ? t0 : t1 - 1;
    if (!summary) at = reverse ? t1 - 1 : t0;
    double gone = 0.0;  // log2 of a summary's decay
    bool from_start = false;
    while (true) {
        const Part part = part_of(a, row, t0, t1, at);
        const bool begins = reverse ? part.last : part.first, ends = reverse ? part.first : part.last;
        const int64_t state_at = (part.seq * a.heads + head) * a.dx * a.dz;
        bool some = false;  // S is not all zeros
        clear();
        if (begins) {
            if (a.initial) {
                const float* p = a.initial + state_at;
                each_state([&](float& v, int64_t i) { v = p[i]; });
                some = true;
            }
        } else if (!summary && a.nsegments > 1) {
            const float4* p = reinterpret_cast<const float4*>(a.carry + carry_at);
#pragma unroll
            for (int j = 0; j < NX; ++j) {
                const float4 v = p[j * THREADS];
                S[j][0] = v.x, S[j][1] = v.y, S[j][2] = v.z, S[j][3] = v.w;
            }
            some = true;
        }
        from_start = begins;

        const int chunks = (int)((part.end - part.begin + C - 1) / C);
        auto chunk_at = [&](int i) { return part.begin + (int64_t)(reverse ? chunks - 1 - i : i) * C; };
        auto count_at = [&](int64_t t) { return (int)(part.end - t < C ? part.end - t : C); };
        float g0 = 0.f, g1 = 0.f;  // one warp: the log decays of tokens 2 lane and 2 lane + 1
        auto fetch_decays = [&](int64_t t, int count) {
            const T* p = pg + t * a.decay.tok_stride;
            g0 = 2 * lane < count ? to_f(p[2 * lane * a.decay.tok_stride]) : 0.f;
            g1 = 2 * lane + 1 < count ? to_f(p[(2 * lane + 1) * a.decay.tok_stride]) : 0.f;
        };
        fetch(0, chunk_at(0), count_at(chunk_at(0)));
        if (warp == 0) {
            fetch_decays(chunk_at(0), count_at(chunk_at(0)));
            make_decays(decays[0], g0, g1, reverse, a.scale_inter, a.scale_update);
        }

        for (int i = 0; i < chunks; ++i) {
            const int64_t t = chunk_at(i);
            const int count = count_at(t);
            const Decays& dc = decays[i & 1];
            copy_wait<0>();
            __syncthreads();
            // the next chunk's decays are one warp's, another one's each time
            const bool ahead = i + 1 < chunks && warp == (i + 1) % WARPS;
            if (i + 1 < chunks) {
                const int64_t tn = chunk_at(i + 1);
                if (Shape::kStages == 2) fetch((i + 1) & 1, tn, count_at(tn));
                if (ahead) fetch_decays(tn, count_at(tn));
            }
            if (summary) gone += dc.total_log2;
            const T* sx = stage(i & 1);
            const T* sy = sx + C * XS;
            const T* sz = sy + C * XS;
            const T* sp = sz + C * ZS;

            if (!summary) {
                // scores of 16 rows and 32 or 64 columns per warp, weighted
                constexpr int COLS = WARPS == 8 ? 32 : 64;
                const int m = warp & 3, c0 = WARPS == 8 ? (warp >> 2) * 32 : 0;
                float acc[COLS / 8][4] = {};
#pragma unroll 2
                for (int k = 0; k < DX / 16; ++k) {
                    if (k * 16 >= dx) break;
                    Pair<T> fa[4];
                    uint32_t pa[NP][4];
                    load_rows<T>(sx, XS, m * 16, k * 16, fa);
                    block_pieces<T>(fa, pa);
#pragma unroll
                    for (int n = 0; n < COLS / 16; ++n) {
                        const int cb = c0 / 16 + n;
                        if (reverse ? cb < m : cb > m) continue;
                        Pair<T> fb[4];
                        uint32_t pb[NP][4];
                        load_rows<T>(sy, XS, cb * 16, k * 16, fb);
                        block_pieces<T>(fb, pb);
#pragma unroll
                        for (int h = 0; h < 2; ++h) mma_pieces<NP, NP, NP - 1>(acc[2 * n + h], pa, pb, h);
                    }
                }
#pragma unroll
                for (int n = 0; n < COLS / 8; ++n) {
                    const int cb = c0 / 16 + n / 2;
                    if (reverse ? cb < m : cb > m) continue;
                    const int c = c0 + n * 8 + lc;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int r = m * 16 + lr + 8 * h;
                        float2 w;
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const float d = (dc.hi[r] - dc.hi[c + e]) + (dc.lo[r] - dc.lo[c + e]);
                            const bool in = reverse ? c + e >= r : c + e <= r;
                            float v = in ? acc[n][2 * h + e] * (ex2(reverse ? -d : d) * a.scale_pair) : 0.f;
                            if (BWD && c + e == r) diagonal[r] = v, v = 0.f;
                            (e ? w.y : w.x) = v;
                        }
                        uint32_t p[PO];
                        split<PO>(w, p);
#pragma unroll
                        for (int u = 0; u < PO; ++u)
                            *reinterpret_cast<uint32_t*>(weighted + (u * C + r) * PS + c) = p[u];
                    }
                }
            }

            float o[4][2][4];  // rows 16 m + lr (+ 8), columns warp * 16 + 8 n + lc (+ 1)
            float dot[4][2];
            if (!summary) {
#pragma unroll
                for (int m = 0; m < 4; ++m)
#pragma unroll
                    for (int n = 0; n < 2; ++n)
#pragma unroll
                        for (int k = 0; k < 4; ++k) o[m][n][k] = 0.f;
                if (some && busy) {
#pragma unroll
                    for (int k = 0; k < DX / 16; ++k) {
                        if (k * 16 >= dx) break;
                        uint32_t ps[PO][4];
#pragma unroll
                        for (int h = 0; h < 4; ++h) {
                            uint32_t q[PO];
                            split<PO>(make_float2(S[2 * k + (h >> 1)][2 * (h & 1)],
                                                  S[2 * k + (h >> 1)][2 * (h & 1) + 1]), q);
#pragma unroll
                            for (int u = 0; u < PO; ++u) ps[u][h] = q[u];
                        }
#pragma unroll
                        for (int m = 0; m < 4; ++m) {
                            Pair<T> fa[4];
                            uint32_t pa[NP][4];
                            load_rows<T>(sx, XS, m * 16, k * 16, fa);
                            block_pieces<T>(fa, pa);
#pragma unroll
                            for (int h = 0; h < 2; ++h) mma_pieces<NP, PO, ORDER>(o[m][h], pa, ps, h);
                        }
                    }
#pragma unroll
                    for (int m = 0; m < 4; ++m)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const float e = dc.inter[m * 16 + lr + 8 * h];
#pragma unroll
                            for (int n = 0; n < 2; ++n) o[m][n][2 * h] *= e, o[m][n][2 * h + 1] *= e;
                        }
                }
                __syncthreads();  // the weighted scores are there
            }
            // Products of the outputs with their partner rows, summed over this warp's columns.
            auto dots = [&](int which) {
                if constexpr (BWD) {
#pragma unroll
                    for (int m = 0; m < 4; ++m)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const int r = m * 16 + lr + 8 * h;
                            float v = 0.f;
#pragma unroll
                            for (int n = 0; n < 2; ++n) {
                                const T* p = sp + r * ZS + warp * 16 + 8 * n + lc;
                                v += o[m][n][2 * h] * to_f(p[0]) + o[m][n][2 * h + 1] * to_f(p[1]);
                            }
                            dot[m][h] = v;
                        }
#pragma unroll
                    for (int m = 0; m < 4; ++m)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            float v = dot[m][h];
                            v += __shfl_xor_sync(0xffffffffu, v, 1);
                            v += __shfl_xor_sync(0xffffffffu, v, 2);
                            if ((lane & 3) == 0) sums[(which * WARPS + warp) * C + m * 16 + lr + 8 * h] = v;
                        }
                }
            };
            if (BWD && pp && !summary) dots(0);

            // this warp's columns of z, all tokens: second operand of the outputs, first of the state
            Pair<T> fz[4][4];
            float odd = 0.f;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                load_cols<T>(sz, ZS, k * 16, warp * 16, fz[k]);
                if (!summary) {
#pragma unroll
                    for (int h = 0; h < 4; ++h) {
                        const float2 v = values(fz[k][h], T());
                        odd = fmaf(v.x, 0.f, fmaf(v.y, 0.f, odd));
                    }
                }
            }
            if (!summary) {
                if (!busy) {
                } else if (!__any_sync(0xffffffffu, !(odd == 0.f))) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        uint32_t pv[NP][4];
                        block_pieces<T>(fz[k], pv);
#pragma unroll
                        for (int m = 0; m < 4; ++m) {
                            if (reverse ? k < m : k > m) continue;
                            uint32_t pw[PO][4];
#pragma unroll
                            for (int u = 0; u < PO; ++u)
                                ldmatrix<bf16, false>(weighted + (u * C + m * 16 + (lane & 15)) * PS + k * 16 + (lane >> 4) * 8,
                                                      pw[u]);
#pragma unroll
                            for (int h = 0; h < 2; ++h) mma_pieces<PO, NP, ORDER>(o[m][h], pw, pv, h);
                        }
                    }
                } else {
                    // A value that is not finite: 0 times it is not 0, and the rows before it do
                    // not take part in it.
#pragma unroll
                    for (int m = 0; m < 4; ++m)
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const int r = m * 16 + lr + (e & 2) * 4, n = e >> 2, z = warp * 16 + 8 * n + lc + (e & 1);
                            float v = o[m][n][e & 3];
                            for (int c = reverse ? r : 0; c < (reverse ? count : r + 1); ++c) {
                                float w = 0.f;
                                for (int u = 0; u < PO; ++u) w += to_f(weighted[(u * C + r) * PS + c]);
                                v += w * to_f(sz[c * ZS + z]);
                            }
                            o[m][n][e & 3] = v;
                        }
                }
                if (BWD && pp) dots(1);
                if constexpr (BWD) {
                    // A token's pair with itself, in float32: it has no part in the decay's gradient,
                    // where it would leave what two roundings of it differ by.
#pragma unroll
                    for (int m = 0; m < 4; ++m)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const int r = m * 16 + lr + 8 * h;
                            const float w = diagonal[r];
#pragma unroll
                            for (int n = 0; n < 2; ++n) {
                                const T* p = sz + r * ZS + warp * 16 + 8 * n + lc;
                                o[m][n][2 * h] = fmaf(w, to_f(p[0]), o[m][n][2 * h]);
                                o[m][n][2 * h + 1] = fmaf(w, to_f(p[1]), o[m][n][2 * h + 1]);
                            }
                        }
                }
#pragma unroll
                for (int m = 0; m < 4; ++m)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int r = m * 16 + lr + 8 * h;
                        if (r >= count) continue;
                        const int64_t base = row * a.out_seq + (t + r) * a.out_tok + head * a.out_head + z0;
#pragma unroll
                        for (int n = 0; n < 2; ++n) {
                            const int z = warp * 16 + 8 * n + lc;
                            const float2 v = make_float2(o[m][n][2 * h], o[m][n][2 * h + 1]);
                            if (a.out_f32) {
                                float* p = static_cast<float*>(a.out) + base + z;
                                if (z < dz) p[0] = v.x;
                                if (z + 1 < dz) p[1] = v.y;
                            } else {
                                T* p = static_cast<T*>(a.out) + base + z;
                                if (a.out_pair) {
                                    if (z < dz) st_pack<2>(p, from_f2<T>(v));
                                } else {
                                    if (z < dz) p[0] = from_f<T>(v.x);
                                    if (z + 1 < dz) p[1] = from_f<T>(v.y);
                                }
                            }
                        }
                    }
            }

            // the state behind the chunk
            // What the chunk adds is summed by itself and then added: the units cut their sums off where
            // float32 additions round, and a state that is kept for long would drift.
            const float total = dc.total;
            uint32_t pz[4][3][4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    const float2 w = *reinterpret_cast<const float2*>(&dc.update[k * 16 + lc + 8 * (h >> 1)]);
                    const float2 v = values(fz[k][h], T());
                    uint32_t q[3];
                    split<3>(make_float2(v.x * w.x, v.y * w.y), q);
#pragma unroll
                    for (int u = 0; u < 3; ++u) pz[k][u][h] = q[u];
                }
            // two blocks of 16 rows at once where there are no more pieces than one: four chains
            constexpr int WIDE = NP == 1 ? 2 : 1;
#pragma unroll
            for (int j = 0; j < NX / 2; j += WIDE) {
                if (!busy || j * 16 >= dx) break;
                float add[WIDE][2][4] = {};
#pragma unroll
                for (int k = 0; k < 4; ++k)
#pragma unroll
                    for (int w = 0; w < WIDE; ++w) {
                        Pair<T> fy[4];
                        uint32_t py2[NP][4];
                        load_cols<T>(sy, XS, k * 16, (j + w) * 16, fy);
                        block_pieces<T>(fy, py2);
#pragma unroll
                        for (int h = 0; h < 2; ++h) mma_pieces<3, NP, 2>(add[w][h], pz[k], py2, h);
                    }
#pragma unroll
                for (int w = 0; w < WIDE; ++w)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            S[2 * (j + w) + h][k] = fmaf(total, S[2 * (j + w) + h][k], add[w][h][k]);
            }
            some = true;
            if (ahead) make_decays(decays[(i + 1) & 1], g0, g1, reverse, a.scale_inter, a.scale_update);

            if (BWD && pp && !summary) {
                __syncthreads();
                if (tid < count) {
                    float v[2] = {0.f, 0.f};
#pragma unroll
                    for (int k = 0; k < 2; ++k)
#pragma unroll
                        for (int w = 0; w < WARPS; ++w) v[k] += sums[(k * WARPS + w) * C + tid];
                    const int64_t i2 = (zt * a.heads + head) * (a.rows * a.length) + row * a.length + t + tid;
                    a.dots_inter[i2] = v[0];
                    a.dots_all[i2] = v[1];
                }
            }
            if (Shape::kStages == 1 && i + 1 < chunks) {
                __syncthreads();
                fetch(0, chunk_at(i + 1), count_at(chunk_at(i + 1)));
            }
        }
        __syncthreads();  // the last chunk's tiles are free

        if (summary) break;
        if (ends) {
            if (a.final_state) {
                float* p = a.final_state + state_at;
                each_state([&](float& v, int64_t i) { p[i] = v; });
            }
            if (BWD && a.final_dot) {
                const float* p = a.final_dot + state_at;
                float sum = 0.f;
                each_state([&](float& v, int64_t i) { sum = fmaf(v, p[i], sum); });
#pragma unroll
                for (int o2 = 16; o2; o2 >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o2);
                if (lane == 0) warp_sums[warp] = sum;
                __syncthreads();
                if (tid == 0) {
                    float v = 0.f;
                    for (int w = 0; w < WARPS; ++w) v += warp_sums[w];
                    a.final_dots[(zt * a.nseq + part.seq) * a.heads + head] = v;
                }
                __syncthreads();
            }
        }
        at = reverse ? part.begin - 1 : part.end;
        if (reverse ? at < t0 : at >= t1) break;
    }
    if (summary) {
        float4* p = reinterpret_cast<float4*>(a.carry + carry_at);
#pragma unroll
        for (int j = 0; j < NX; ++j) p[j * THREADS] = make_float4(S[j][0], S[j][1], S[j][2], S[j][3]);
        if (zt == 0 && tid == 0) {
            const int64_t i = (row * a.nsegments + seg) * a.heads + head;
            a.carry_decay[i] = (float)gone;
            a.carry_reset[i] = from_start;
        }
    }
}

template <class T, int DX, int WARPS, bool BWD>
cudaError_t launch_attn(const AttnArgs& args, cudaStream_t s) {
    using Shape = AttnShape<T, DX, WARPS, BWD>;
    static LaunchCache cache;
    LaunchGeom g;
    cudaError_t e = cache.get(
        [](int dev, LaunchGeom* out) {
            return setup_persistent(k_linattn<T, DX, WARPS, BWD>, Shape::kThreads, Shape::kBytes, dev, out);
        },
        &g);
    if (e != cudaSuccess) return e;
    AttnArgs a = args;
    const int64_t blocks = a.rows * a.nsegments * a.heads * a.ztiles;
    if (blocks > INT32_MAX) return cudaErrorInvalidValue;
    if (a.nsegments > 1) {
        a.summary = 1;
        k_linattn<T, DX, WARPS, BWD><<<(unsigned)blocks, Shape::kThreads, Shape::kBytes, s>>>(a);
        e = cudaGetLastError();
        if (e != cudaSuccess) return e;
        e = attn_carry_pass(a, a.ztiles * (DX * Shape::kZ / 4), s);
        if (e != cudaSuccess) return e;
        a.summary = 0;
    }
    k_linattn<T, DX, WARPS, BWD><<<(unsigned)blocks, Shape::kThreads, Shape::kBytes, s>>>(a);
    return cudaGetLastError();
}

template <class T, bool BWD>
cudaError_t attn_any(const AttnArgs& a, int dtype, cudaStream_t s) {
    const int dx = attn_pad(a.dx), warps = attn_warps(dtype, a.dx, a.dz);
    if (warps == 4)
        return dx == 64 ? launch_attn<T, 64, 4, BWD>(a, s)
                        : (dx == 128 ? launch_attn<T, 128, 4, BWD>(a, s) : launch_attn<T, 256, 4, BWD>(a, s));
    if (dx == 64) return launch_attn<T, 64, 8, BWD>(a, s);
    if constexpr (!std::is_same<T, float>::value)
        if (dx == 256) return launch_attn<T, 256, 8, BWD>(a, s);
    return launch_attn<T, 128, 8, BWD>(a, s);
}

}  // namespace
}  // namespace gbfft
