// Linear attention in bfloat16 on the fifth-generation tensor cores (tcgen05): chunks of 128 tokens,
// the same products as linattn.cuh, for heads of up to 128 values whose rows lie on 16-byte
// boundaries.
//
// Operands lie in shared memory in the 128-byte swizzle, panels of 64 columns, rows of tokens; the
// same tile is an operand summed over its columns (scores) and one summed over its rows (outputs,
// state).  Accumulators lie in tensor memory:
//   columns   0..127  scores, then the weighted ones as an operand (in place, one or two pieces)
//           128..255  outputs
//           256..383  what the chunk adds to S^T: row = column of z, column = column of x
//           384..511  the first two pieces of the weighted z^T, an operand; the third is in shared
//                     memory
// The state itself is float32 in the registers of the warps that own the rows of S^T: what a chunk
// adds is summed by itself and then added, since the units cut their sums off where float32
// additions round.  One block per SM (what is spilled has no room in its level-1 cache
// beside the tiles, so warps are counted by their registers):
//   A (four warps, a token each thread; eight in the gradients, half its columns): weights of the
//   scores, outputs
//   B (eight warps, half a row of S^T each thread): weighted z^T, the state
//   one warp each issues the products, sums the decays, copies rows of y and z, copies rows of x:
//   a fence before the units read shared memory waits for the thread's copies under way, so those
//   that copy do nothing else.
// A weight exp(G[r] - G[c]) of another block of 32 columns than the row's own is a product of one
// factor for each row and one for each column, both from the end of the columns' block (at most 1).
// They meet at mbarriers only, each of which completes once per chunk (twice-buffered ones every other
// chunk).  Every wait is bounded in time, and a warp's lanes give up together, so that none of them goes
// on into an instruction of the whole warp alone.  A warp that gives up goes to the block's end; those that
// wait for it give up in turn, the warp that issues products waits for them there, and so no product
// outlives its block.
//
// Measured: one sequence of 16384 tokens, 16 heads of 128 x 128, time cut in 9: 158 us, 1.7 TB/s of q, k,
// v and outputs; 8 x 2048 tokens of 32 heads of 128 x 64 175 us; gradients of 4 x 2048 tokens of 16 heads
// 459 us.  A chunk took about 9300 cycles at 148 us, the units' products about 4500 of them (scores 1000, with
// the state 1000, outputs 600, state 1800): bound by the chain from weighted z over the state's product to
// the next chunk's, and within it by the latency of the weighting at three warps a scheduler.
#pragma once

#include "linattn.h"
#include "tma.cuh"

namespace gbfft {
namespace {

using bf16 = __nv_bfloat16;
constexpr int kTcB = 256;  // threads of B

// ---- tcgen05 --------------------------------------------------------------------------------

// Shared-memory operand in the 128-byte swizzle: 8 rows of 128 bytes are 1024 bytes (the stride
// offset); `lead` bytes from a panel of 64 columns to the next (for operands summed over rows).
__device__ __forceinline__ uint64_t tc_desc(uint32_t addr, uint32_t lead) {
    return (uint64_t)((addr & 0x3ffffu) >> 4) | (uint64_t)((lead & 0x3ffffu) >> 4) << 16 | (uint64_t)(1024 >> 4) << 32 |
           (uint64_t)1 << 46 | (uint64_t)2 << 61;
}
// float32 sums of bfloat16 products, 128 rows by n columns; b_rows: the second operand is summed over its rows.
constexpr uint32_t tc_idesc(int n, bool b_rows) {
    return 1u << 4 | 1u << 7 | 1u << 10 | (b_rows ? 1u << 16 : 0u) | (uint32_t)(n >> 3) << 17 | (128u >> 4) << 24;
}
__device__ __forceinline__ void tc_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc),
        "r"((uint32_t)add)
        : "memory");
}
__device__ __forceinline__ void tc_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(a), "l"(b), "r"(idesc),
        "r"((uint32_t)add)
        : "memory");
}
// Sixteen summed values a step: operands summed over their columns go 32 bytes on within a panel of
// 64 columns, operands summed over their rows 16 rows.  Loops that stay loops: descriptors that are
// kept for a whole part would need more registers than there are.
__device__ __forceinline__ uint64_t tc_columns(uint32_t tile, int panel, int k) {
    return tc_desc(tile + (k >> 2) * panel + (k & 3) * 32, 16);
}
__device__ __forceinline__ void tc_commit(uint64_t* bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar))
                 : "memory");
}
__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
// Loads have landed; `r` is among what they have written (so that no use of it moves ahead).
__device__ __forceinline__ void tc_wait_ld(uint32_t (&r)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                   "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                   "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31]));
}
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Accesses to tensor memory and matrix loads keep their order (volatile) but do not hold up others:
// barriers and fences do. 32 columns of this warp's 32 rows, one row per thread.
__device__ __forceinline__ void tc_ld32(uint32_t addr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr));
}
__device__ __forceinline__ void tc_st32(uint32_t addr, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(addr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
        "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
        "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31]));
}
__device__ __forceinline__ void tc_st16(uint32_t addr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16};" ::"r"(addr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]));
}
__device__ __forceinline__ void tc_st8(uint32_t addr, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(addr), "r"(r[0]),
                 "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]));
}
__device__ __forceinline__ void tc_ld16(uint32_t addr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(addr));
}
__device__ __forceinline__ void tc_wait_ld16(uint32_t (&r)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]));
}
// 16 rows by 8 columns in the layout of a matrix load: thread l has rows l / 4 (r[0], r[2]) and
// l / 4 + 8, columns l % 4 (r[0], r[1]) and l % 4 + 4.
__device__ __forceinline__ void tc_st_block(uint32_t addr, const uint32_t (&r)[4]) {
    asm volatile("tcgen05.st.sync.aligned.16x128b.x2.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(r[0]), "r"(r[1]),
                 "r"(r[2]), "r"(r[3]));
}
// Four 8 x 8 blocks of shared memory, row addresses from lanes 0..7, 8..15, ...; transposed.
__device__ __forceinline__ void tc_ldmatrix_t(uint32_t addr, uint32_t (&f)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(f[0]), "=r"(f[1]), "=r"(f[2]), "=r"(f[3])
                 : "r"(addr));
}
__device__ __forceinline__ void tc_stmatrix(uint32_t addr, const uint32_t (&f)[4]) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(f[0]), "r"(f[1]),
                 "r"(f[2]), "r"(f[3]));
}
__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}
// Sixteen bytes at byte `at` of a swizzled tile: chunk c of row r of a panel.
__device__ __forceinline__ int tc_chunk(int r, int c) { return r * 128 + ((c ^ (r & 7)) << 4); }

__device__ __forceinline__ uint32_t tc_pack(float x, float y) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(y), "f"(x));
    return r;
}
__device__ __forceinline__ float2 tc_values(uint32_t p) {
    return make_float2(__uint_as_float(p << 16), __uint_as_float(p & 0xffff0000u));
}
// Pieces of 8 bits (of an infinity: itself and no numbers).
template <int N>
__device__ __forceinline__ void tc_split(float2 v, uint32_t (&p)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
        p[i] = tc_pack(v.x, v.y);
        if (i + 1 < N) v = fma2(tc_values(p[i]), splat(-1.f), v);
    }
}

// ---- sizes ----------------------------------------------------------------------------------

template <int DX, int DZ, bool BWD>
struct TcShape {
    static constexpr int kSides = BWD ? 2 : 1, kA = 128 * kSides;  // threads of A
    static constexpr int kThreads = kA + kTcB + 128;
    static constexpr int kPO = BWD ? 2 : 1;  // pieces of weighted scores and of the state as an operand
    static constexpr int kTileX = kTcChunk * DX * 2, kTileZ = kTcChunk * DZ * 2, kTileS = kPO * DZ * DX * 2,
                         kTileW = kTcChunk * kTcChunk * 2;
    static constexpr int kOne = 2 * kTileX + kTileZ + kTileS + kTileW;  // every tile once
    // y and z twice where that fits, y alone else
    static constexpr int kStageZ = kOne + kTileX + kTileZ <= 224 * 1024 ? 2 : 1;
    static constexpr int kStageY = 2;
    static constexpr int kTiles = kTileX + kStageY * kTileX + kStageZ * kTileZ + kTileS + kTileW;
};

enum { TC_X, TC_Y0, TC_Y1, TC_Z0, TC_Z1, TC_SCORES, TC_INTER, TC_OUT, TC_UPDATE0, TC_UPDATE1, TC_WEIGHTED, TC_STATE, TC_WZ, TC_TAKEN0, TC_TAKEN1, TC_DECAYS,
       TC_FREE, TC_PAIR0, TC_PAIR1, TC_PAIR2, TC_PAIR3, TC_MEET, TC_DRAIN, TC_BARS };

// Behind the tiles.  BUFFERS: stages of z.
template <bool BWD, int BUFFERS>
struct TcSmall {
    float2 G[kTcChunk];  // the sums of the decays (log2) in two floats
    float update[kTcChunk];
    float column[kTcChunk];  // factors of the columns of scores, from the end of their block of 32
    float total, all_hi, all_lo;
    uint64_t bars[TC_BARS];
    // of every column of z, by halves of the tokens, the place of a value that is not finite, plus 1:
    // the first one, 255 for none; reversed the last one, 0 for none.  Set where bad_any is.
    alignas(8) unsigned char bad_at[BUFFERS][2][kTcChunk];
    unsigned char bad_any[BUFFERS][8];  // by warps
    float diagonal[BWD ? kTcChunk : 1];  // weighted scores of tokens with themselves
    float warp_sums[8];
    uint32_t tmem;
};
template <int DX, int DZ, bool BWD> constexpr int tc_bytes() {
    using Shape = TcShape<DX, DZ, BWD>;
    constexpr int bytes = Shape::kTiles + (int)sizeof(TcSmall<BWD, Shape::kStageZ>);
    static_assert(bytes <= 227 * 1024, "shared memory");
    return bytes;
}

// The part of a segment that belongs to one sequence (offsets of any kind: it holds token `at` and
// stays in the segment).
struct TcPart {
    int begin, end, seq;
    bool first, last;
};
__device__ __forceinline__ TcPart tc_part(const AttnArgs& a, int row, int t0, int t1, int at) {
    const SeqAt s = seq_at(a.offsets, a.nseq, a.length, row, at);
    TcPart p;
    p.seq = (int)s.q;
    p.begin = s.begin > at ? at : (s.begin < t0 ? t0 : (int)s.begin);
    p.end = s.end <= at ? at + 1 : (s.end > t1 ? t1 : (int)s.end);
    p.first = p.begin == 0 || (s.begin >= t0 && s.begin <= at);
    p.last = p.end == a.length || (s.end <= t1 && s.end > at);
    return p;
}

// Copies rows of up to D values into a swizzled tile, zeros beyond count and dim: one warp.
template <int D>
__device__ __forceinline__ void tc_load(char* tile, const bf16* g, int64_t tok, int count, int dim, int lane) {
    constexpr int N = D / 8, STEP = 32 / N;  // 16-byte pieces of a row; rows that the warp takes at once
    static_assert(8 % STEP == 0, "rows of a lane");
    const int c = lane % N, r = lane / N;
    const bf16* src = g + r * tok + c * 8;
    char* dst = tile + (c >> 3) * (kTcChunk * 128) + r * 128;
    const int live = c * 8 < dim ? count : 0, swizzled = (c & 7) ^ r;
#pragma unroll 4
    for (int k = 0; k < kTcChunk; k += STEP) {
        const bool in = r + k < live;
        copy16(dst + k * 128 + ((swizzled ^ (k & 7)) << 4), in ? src : g, in);
        src += STEP * tok;
    }
}
// Pieces of 16 bytes change places within four lanes: piece j of lane i becomes piece i of lane j.
__device__ __forceinline__ void tc_transpose(uint4 (&p)[4], int lane) {
    auto swap = [&](uint4& lo, uint4& hi, int bit) {
        const bool up = lane & bit;
        uint4 v = up ? lo : hi;
        v.x = __shfl_xor_sync(0xffffffffu, v.x, bit);
        v.y = __shfl_xor_sync(0xffffffffu, v.y, bit);
        v.z = __shfl_xor_sync(0xffffffffu, v.z, bit);
        v.w = __shfl_xor_sync(0xffffffffu, v.w, bit);
        if (up) lo = v;
        else hi = v;
    };
    swap(p[0], p[2], 2);
    swap(p[1], p[3], 2);
    swap(p[0], p[1], 1);
    swap(p[2], p[3], 1);
}

// Waits for at most `limit` nanoseconds, by the low half of the timer, which passes 0 every 4.3 s.
__device__ __forceinline__ uint32_t tc_ns() {
    uint32_t t;
    asm volatile("mov.u32 %0, %%globaltimer_lo;" : "=r"(t));
    return t;
}
__device__ __forceinline__ bool tc_lane_wait(uint64_t* bar, uint32_t parity, uint32_t limit) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint32_t begun = tc_ns();
    while (!mbar_try_wait(bar, parity))
        if (tc_ns() - begun > limit) return false;
    return true;
}

template <int DX, int DZ, bool BWD>
__global__ void __launch_bounds__(TcShape<DX, DZ, BWD>::kThreads, 1) k_linattn_tc(const AttnArgs a, int* err) {
    using Shape = TcShape<DX, DZ, BWD>;
    constexpr int C = kTcChunk, PO = Shape::kPO, PANEL = C * 128, SIDES = Shape::kSides;
    constexpr int B0 = Shape::kA / 32, M0 = B0 + kTcB / 32;  // first warps of B and of the others
    extern __shared__ __align__(1024) char base[];
    char* tile_x = base;
    char* tile_y = tile_x + Shape::kTileX;
    char* tile_z = tile_y + Shape::kStageY * Shape::kTileX;
    char* tile_s = tile_z + Shape::kStageZ * Shape::kTileZ;
    char* tile_w = tile_s + Shape::kTileS;
    using Small = TcSmall<BWD, Shape::kStageZ>;
    Small& sm = *reinterpret_cast<Small*>(base + Shape::kTiles);
    uint64_t* bars = sm.bars;
    if (!tma_stage_aligned(base, err) || (smem_addr(base) & 1023)) return;  // every thread alike
    if (a.wait_ns == 0) {  // a limit of 0: no wait is begun
        if (threadIdx.x == 0) atomicCAS(err, 0, KERR_WAIT_TIMEOUT);
        return;
    }

    const int tid = (int)threadIdx.x, warp = tid >> 5, lane = tid & 31;
    // lengths and counts of blocks are below 2^31
    unsigned b = blockIdx.x;
    const int zt = (int)(b % (unsigned)a.ztiles);
    b /= (unsigned)a.ztiles;
    const int head = (int)(b % (unsigned)a.heads);
    b /= (unsigned)a.heads;
    const int seg = (int)(b % (unsigned)a.nsegments), row = (int)(b / (unsigned)a.nsegments);
    const int t0 = (int)(seg * a.segment), t1 = (int)(t0 + a.segment < a.length ? t0 + a.segment : a.length);
    const int z0 = zt * DZ, dz = (int)a.dz - z0 < DZ ? (int)a.dz - z0 : DZ, dx = (int)a.dx;
    const bool reverse = a.reverse, summary = a.summary;

    if (warp == M0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(&sm.tmem))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    if (tid == 0) {
        for (int i = 0; i < TC_BARS; ++i) {
            const bool commit = i == TC_SCORES || i == TC_INTER || i == TC_OUT || i == TC_UPDATE0 || i == TC_UPDATE1 || i == TC_DRAIN;
            const bool warps = i == TC_DECAYS || (i >= TC_X && i <= TC_Z1);
            const bool all_b = i == TC_STATE || i == TC_WZ || i == TC_MEET, pair = i >= TC_PAIR0 && i <= TC_PAIR3;
            mbar_init(&bars[i], commit ? 1 : (warps ? 32 : (pair ? 64 : (i == TC_FREE ? Shape::kA + kTcB : (all_b ? kTcB : Shape::kA)))));
        }
        fence_mbar_init();
    }
    tc_before();
    __syncthreads();
    tc_after();
    const uint32_t tmem = sm.tmem;
    const uint32_t kOut = tmem + 128, kAdd = tmem + 256, kWz = tmem + 384;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // this warp's rows: 32 (warp mod 4) in bits 16 up

    // The votes and a limit that is an argument cost 1 to 6% (148, 169 and 455 us without them): a lane that went
    // on alone, or a warp that waited for one that has left, would not end.
    auto lane_wait = [&](int bar, uint32_t phase) { return tc_lane_wait(&bars[bar], phase & 1, a.wait_ns); };
    auto wait = [&](int bar, uint32_t phase) { return __all_sync(0xffffffffu, lane_wait(bar, phase)) != 0; };
    // Calls f(part, n) for every part of the segment in the direction of the pass, n its first
    // chunk's number; a summary takes the part that reaches the next segment.
    auto each_part = [&](auto f) {
        int at = summary == reverse ? t0 : t1 - 1;
        if (!summary) at = reverse ? t1 - 1 : t0;
        uint32_t n = 0;
        while (true) {
            const TcPart p = tc_part(a, row, t0, t1, at);
            const int chunks = (p.end - p.begin + C - 1) / C;
            if (!f(p, chunks, n)) return false;
            n += chunks;
            at = reverse ? p.begin - 1 : p.end;
            if (summary || (reverse ? at < t0 : at >= t1)) return true;
        }
    };
    auto chunk_at = [&](const TcPart& p, int chunks, int i) {
        return p.begin + (reverse ? chunks - 1 - i : i) * C;
    };
    auto count_at = [&](const TcPart& p, int t) { return p.end - t < C ? p.end - t : C; };
    auto begins_at = [&](const TcPart& p) { return reverse ? p.last : p.first; };
    // whether the part's first chunk meets a state that is not zero
    auto starts_with_state = [&](const TcPart& p) { return begins_at(p) ? a.initial != nullptr : !summary && a.nsegments > 1; };

    bool fine = true;
    const int quad = warp & 3;  // rows 32 quad .. of tensor memory
    if (warp < B0) {
        // ---- A: a token, or half of one's columns, each thread ----
        const bf16* pp = BWD && a.partner.data
                             ? static_cast<const bf16*>(a.partner.data) + row * a.partner.seq +
                                   (head / a.partner.share) * a.partner.head + z0
                             : nullptr;
        const int r = tid & 127, side = warp >> 2;
        constexpr int COLUMNS = DZ / SIDES;
        fine = each_part([&](const TcPart& p, int chunks, uint32_t n0) {
            for (int i = 0; i < chunks; ++i) {
                const uint32_t n = n0 + i, half = n & 1;
                const int t = chunk_at(p, chunks, i);
                const int count = count_at(p, t);
                const bool some = i > 0 || starts_with_state(p);
                if (summary) {
                    if (!wait(TC_DECAYS, n)) return false;
                    mbar_arrive(&bars[TC_FREE]);
                    continue;
                }
                if (!wait(TC_DECAYS, n) || !wait(TC_SCORES, n)) return false;
                tc_after();
                const float2 G = sm.G[r];
                const float inter = ex2(reverse ? (sm.all_hi - G.x) + (sm.all_lo - G.y) : G.x) * a.scale_inter;
                auto weigh = [&](int cb, const uint32_t (&s)[32]) {
#pragma unroll
                for (int k = 0; k < 2; ++k) {  // 16 columns at a time
                    const int c0 = cb * 32 + k * 16;
                    const uint32_t* sk = s + k * 16;
                    uint32_t out[PO][8];
                    if (cb == quad) {  // the rows' own block
                        const float sign = reverse ? -1.f : 1.f;
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const float4 g = *reinterpret_cast<const float4*>(&sm.G[c0 + 2 * j]);
                            const float d[2] = {(G.x - g.x) + (G.y - g.y), (G.x - g.z) + (G.y - g.w)};
                            float v[2];
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const int c = k * 16 + 2 * j + e;
                                const float w = __uint_as_float(sk[2 * j + e]) * (ex2(sign * d[e]) * a.scale_pair);
                                v[e] = (reverse ? c >= lane : c <= lane) ? w : 0.f;
                                if (BWD && c == lane) sm.diagonal[r] = v[e], v[e] = 0.f;
                            }
                            uint32_t q[PO];
                            tc_split<PO>(make_float2(v[0], v[1]), q);
#pragma unroll
                            for (int u = 0; u < PO; ++u) out[u][j] = q[u];
                        }
                    } else if (reverse ? cb > quad : cb < quad) {
                        const float2 e = sm.G[reverse ? cb * 32 - 1 : cb * 32 + 31];
                        const float d = (G.x - e.x) + (G.y - e.y);
                        const float2 w = splat(ex2(reverse ? -d : d) * a.scale_pair);
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float4 f = *reinterpret_cast<const float4*>(&sm.column[c0 + 4 * j]);
#pragma unroll
                            for (int e2 = 0; e2 < 2; ++e2) {
                                const float2 v = make_float2(__uint_as_float(sk[4 * j + 2 * e2]),
                                                             __uint_as_float(sk[4 * j + 2 * e2 + 1]));
                                uint32_t q[PO];
                                tc_split<PO>(mul2(mul2(v, e2 ? make_float2(f.z, f.w) : make_float2(f.x, f.y)), w), q);
#pragma unroll
                                for (int u = 0; u < PO; ++u) out[u][2 * j + e2] = q[u];
                            }
                        }
                    } else {
#pragma unroll
                        for (int u = 0; u < PO; ++u)
#pragma unroll
                            for (int j = 0; j < 8; ++j) out[u][j] = 0;
                    }
#pragma unroll
                    for (int u = 0; u < PO; ++u) tc_st8(tmem + lanes + u * 64 + c0 / 2, out[u]);
                }
                };
                // The weighted scores go where scores are that have been read (by the other half's
                // threads too): the first piece in columns 0 to 63, the second in the others.
#pragma unroll 1
                for (int cb = side * 2; cb < side * 2 + 4 / SIDES; cb += 2) {
                    uint32_t s[2][32];
                    tc_ld32(tmem + lanes + cb * 32, s[0]);
                    tc_ld32(tmem + lanes + cb * 32 + 32, s[1]);
                    tc_wait_ld(s[0]);
                    tc_wait_ld(s[1]);
                    if (SIDES == 2) {  // once per chunk, as this loop runs once
                        mbar_arrive(&bars[TC_PAIR0 + quad]);
                        if (!wait(TC_PAIR0 + quad, n)) return false;
                    }
                    weigh(cb, s[0]);
                    weigh(cb + 1, s[1]);
                }
                mbar_arrive(&bars[TC_FREE]);
                // Rows go to and from memory in 64 bytes by four lanes; a lane's own row is among theirs.
                const int r4 = r & ~3;
                // products with the partner's values of 32 columns, zeros beyond dz
                auto dot = [&](int c0, const uint32_t (&v)[32], float sum) {
                    if (!pp) return sum;
                    uint4 q[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int c = c0 + 8 * (lane & 3);
                        q[k] = make_uint4(0, 0, 0, 0);
                        if (r4 + k < count && c < dz)
                            q[k] = *reinterpret_cast<const uint4*>(pp + (int64_t)(t + r4 + k) * a.partner.tok + c);
                    }
                    tc_transpose(q, lane);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint32_t w[4] = {q[k].x, q[k].y, q[k].z, q[k].w};
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float2 f = tc_values(w[e]);
                            sum = fmaf(f.x, __uint_as_float(v[8 * k + 2 * e]), sum);
                            sum = fmaf(f.y, __uint_as_float(v[8 * k + 2 * e + 1]), sum);
                        }
                    }
                    return sum;
                };
                float between = 0.f;
                if (some) {
                    if (!wait(TC_INTER, n)) return false;
                    tc_after();
#pragma unroll 1
                    for (int c0 = side * COLUMNS; c0 < side * COLUMNS + COLUMNS; c0 += 32) {
                        uint32_t v[32];
                        tc_ld32(kOut + lanes + c0, v);
                        tc_wait_ld(v);
#pragma unroll
                        for (int j = 0; j < 32; ++j) v[j] = __float_as_uint(__uint_as_float(v[j]) * inter);
                        tc_st32(kOut + lanes + c0, v);
                        if (BWD) between = dot(c0, v, between);
                    }
                }
                tc_wait_st();
                tc_before();
                mbar_arrive(&bars[TC_WEIGHTED]);
                // B has looked at z by the time that the outputs are there
                if (!wait(TC_OUT, n)) return false;
                tc_after();
                const char* sz = tile_z + (Shape::kStageZ == 2 ? half * Shape::kTileZ : 0);
                const int bz = Shape::kStageZ == 2 ? half : 0;
                const bool bad = *reinterpret_cast<const uint64_t*>(sm.bad_any[bz]) != 0;
                const float diagonal = BWD ? sm.diagonal[r] : 0.f;
                float all = 0.f;
#pragma unroll 1
                for (int c0 = side * COLUMNS; c0 < side * COLUMNS + COLUMNS; c0 += 32) {
                    uint32_t v[32];
                    tc_ld32(kOut + lanes + c0, v);
                    tc_wait_ld(v);
                    if (BWD) {
                        all = dot(c0, v, all);
                        // a token's pair with itself, in float32: it has no part in the decay's gradient
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const int c = c0 / 8 + j;
                            const uint4 q = *reinterpret_cast<const uint4*>(sz + (c >> 3) * PANEL + tc_chunk(r, c & 7));
                            const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const float2 f = tc_values(w[e]);
                                uint32_t &lo = v[8 * j + 2 * e], &hi = v[8 * j + 2 * e + 1];
                                lo = __float_as_uint(fmaf(diagonal, f.x, __uint_as_float(lo)));
                                hi = __float_as_uint(fmaf(diagonal, f.y, __uint_as_float(hi)));
                            }
                        }
                    }
                    if (bad) {  // a value of z that is no number or infinite, by this token
#pragma unroll
                        for (int j = 0; j < 32; ++j) {
                            const int k0 = sm.bad_at[bz][0][c0 + j], k1 = sm.bad_at[bz][1][c0 + j];
                            if (reverse ? r < k0 || r < k1 : r + 1 >= k0 || r + 1 >= k1) v[j] = 0x7fffffffu;
                        }
                    }
                    const int64_t at = row * a.out_seq + (t + r4) * a.out_tok + head * a.out_head + z0;
                    if (a.out_f32) {
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            uint4 q[4];
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                q[k] = make_uint4(v[16 * h + 4 * k], v[16 * h + 4 * k + 1], v[16 * h + 4 * k + 2], v[16 * h + 4 * k + 3]);
                            tc_transpose(q, lane);
                            const int c = c0 + 16 * h + 4 * (lane & 3);
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                if (r4 + k < count && c < dz)
                                    *reinterpret_cast<uint4*>(static_cast<float*>(a.out) + at + k * a.out_tok + c) = q[k];
                        }
                    } else {
                        uint4 q[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            uint32_t w[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                w[e] = tc_pack(__uint_as_float(v[8 * k + 2 * e]), __uint_as_float(v[8 * k + 2 * e + 1]));
                            q[k] = make_uint4(w[0], w[1], w[2], w[3]);
                        }
                        tc_transpose(q, lane);
                        const int c = c0 + 8 * (lane & 3);
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            if (r4 + k < count && c < dz)
                                *reinterpret_cast<uint4*>(static_cast<bf16*>(a.out) + at + k * a.out_tok + c) = q[k];
                    }
                }
                if (pp && r < count) {
                    const int64_t k = ((zt * SIDES + side) * a.heads + head) * (a.rows * a.length) + row * a.length + t + r;
                    a.dots_inter[k] = between;
                    a.dots_all[k] = all;
                }
                tc_before();
                mbar_arrive(&bars[TC_TAKEN0 + half]);
            }
            return true;
        });
    } else if (warp < M0) {
        // ---- B: half a row of S^T each thread; half the tokens of z^T ----
        const int id = tid - Shape::kA, m = id & 127, side = id >> 7;
        constexpr int HALF = DX / 2;
        const int x0 = side * HALF;
        float2 S[HALF / 2];  // row m of S^T, columns x0 ..
        uint32_t met = 0;    // times that all of B has met
        const int64_t carry_at = ((((int64_t)row * a.nsegments + seg) * a.heads + head) * a.ztiles + zt) * (DX * 128) +
                                 (side * (HALF / 4) * 128 + m) * 4;
        // S as an operand: row m, columns in panels of 64
        char* state_row = tile_s + (x0 >> 6) * (DZ * 128) + m * 128;
        const int swizzle = ((m & 7) ^ (x0 / 8 & 7)) << 4;
        auto put_state = [&] {
            if (m < DZ && !summary) {
#pragma unroll
                for (int k = 0; k < HALF / 8; ++k) {
                    uint32_t q[4][PO];
#pragma unroll
                    for (int e = 0; e < 4; ++e) tc_split<PO>(S[4 * k + e], q[e]);
#pragma unroll
                    for (int u = 0; u < PO; ++u)
                        *reinterpret_cast<uint4*>(state_row + u * (DZ * DX * 2) + (swizzle ^ (k << 4))) =
                            make_uint4(q[0][u], q[1][u], q[2][u], q[3][u]);
                }
            }
            fence_proxy_async_smem();
            tc_before();
            mbar_arrive(&bars[TC_STATE]);
        };
        // f(value, address) of the values that this thread holds, in states at p (the next address from
        // the last one: all of them at once would be kept in registers)
        auto each_state = [&](auto* p, auto f) {
            if (m >= dz) return;
            p += x0 * a.state_x;
#pragma unroll
            for (int j = 0; j < HALF; ++j) {
                if (x0 + j < dx) f(j & 1 ? S[j / 2].y : S[j / 2].x, p);
                p += a.state_x;
                asm volatile("" : "+l"(p));
            }
        };
        fine = each_part([&](const TcPart& p, int chunks, uint32_t n0) {
            const int64_t mine = (p.seq * a.heads + head) * a.dx * a.dz + (z0 + m) * a.state_z;
            const bool from_start = begins_at(p);
            // the last chunk's products are over, those with the state among them
#pragma unroll
            for (int j = 0; j < HALF / 2; ++j) S[j] = splat(0.f);
            if (from_start) {
                if (a.initial) each_state(a.initial + mine, [](float& v, const float* q) { v = *q; });
            } else if (!summary && a.nsegments > 1) {
                const float4* q = reinterpret_cast<const float4*>(a.carry + carry_at);
#pragma unroll
                for (int j = 0; j < HALF / 4; ++j) {
                    const float4 v = q[j * 128];
                    S[2 * j] = make_float2(v.x, v.y), S[2 * j + 1] = make_float2(v.z, v.w);
                }
            }
            put_state();
            for (int i = 0; i < chunks; ++i) {
                const uint32_t n = n0 + i, half = n & 1;
                const bool next = i + 1 < chunks;
                if (!wait(TC_Z0 + half, n >> 1) || !wait(TC_DECAYS, n)) return false;
                const float total = sm.total;
                // this warp's 32 columns of z and half of the tokens, weighted, in three pieces
                char* sz = tile_z + (Shape::kStageZ == 2 ? half * Shape::kTileZ : 0);
                const uint32_t z_at = smem_addr(sz), w_at = smem_addr(tile_w);
                float2 odd = splat(0.f);
                // two blocks of 16 columns by four of 16 tokens; a loop, since addresses of all eight would be
                // kept for the whole part
#pragma unroll 1
                for (int it = 0; it < 8; ++it) {
                    const int m0 = quad * 32 + (it & 1) * 16, tk = side * 64 + (it >> 1) * 16;
                    const float2 w0 = *reinterpret_cast<const float2*>(&sm.update[tk + 2 * (lane & 3)]);
                    const float2 w1 = *reinterpret_cast<const float2*>(&sm.update[tk + 8 + 2 * (lane & 3)]);
                    uint32_t f[4] = {}, q[3][4];
                    if (m0 < DZ) {
                        const int at = tk + (lane & 7) + (lane >> 4) * 8, c = m0 / 8 + ((lane >> 3) & 1);
                        tc_ldmatrix_t(z_at + (c >> 3) * PANEL + tc_chunk(at, c & 7), f);
                    }
#pragma unroll
                    for (int h = 0; h < 4; ++h) {
                        const float2 v = tc_values(f[h]);
                        odd = fma2(v, splat(0.f), odd);
                        uint32_t g[3];
                        tc_split<3>(mul2(v, h < 2 ? w0 : w1), g);
#pragma unroll
                        for (int u = 0; u < 3; ++u) q[u][h] = g[u];
                    }
                    const uint32_t to = kWz + lanes + ((uint32_t)(it & 1) << 20) + tk / 2;
                    tc_st_block(to, q[0]);
                    tc_st_block(to + 64, q[1]);
                    // rows m0 .. m0 + 15 of the third piece's tile, 16 tokens
                    const int rw = m0 + (lane & 7) + ((lane >> 3) & 1) * 8, c = (tk & 63) / 8 + (lane >> 4);
                    tc_stmatrix(w_at + side * PANEL + tc_chunk(rw, c), q[2]);
                }
                mbar_arrive(&bars[TC_FREE]);
                if (!summary) {
                    // 0 times what is not finite is not 0: such values leave the tile, and the outputs
                    // that they are in are set by hand
                    const bool any = __any_sync(0xffffffffu, !(odd.x == 0.f && odd.y == 0.f));
                    int k = reverse ? 0 : 255;
                    if (any && m < DZ) {
                        for (int tk = side * 64; tk < side * 64 + 64; ++tk) {
                            unsigned short* u = reinterpret_cast<unsigned short*>(sz + (m >> 6) * PANEL +
                                                                                 tc_chunk(tk, (m >> 3) & 7) + (m & 7) * 2);
                            if ((*u & 0x7f80) == 0x7f80) {
                                *u = 0;
                                if (reverse || k == 255) k = tk + 1;
                            }
                        }
                    }
                    const int bz = Shape::kStageZ == 2 ? half : 0;
                    sm.bad_at[bz][side][m] = (unsigned char)k;
                    if (lane == 0) sm.bad_any[bz][warp - B0] = any;
                }
                tc_wait_st();
                fence_proxy_async_smem();
                tc_before();
                mbar_arrive(&bars[TC_WZ]);

                if (!wait(TC_UPDATE0 + half, n >> 1)) return false;
                tc_after();
#pragma unroll
                for (int c0 = 0; c0 < HALF; c0 += 16) {
                    uint32_t v[16];
                    tc_ld16(kAdd + lanes + x0 + c0, v);
                    tc_wait_ld16(v);
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        S[c0 / 2 + j] = fma2(splat(total), S[c0 / 2 + j],
                                             make_float2(__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1])));
                }
                if (next) put_state();
            }
            if (!summary && (reverse ? p.first : p.last)) {
                if (a.final_state) each_state(a.final_state + mine, [](float& v, float* q) { *q = v; });
                if (BWD && a.final_dot) {
                    float sum = 0.f;
                    each_state(a.final_dot + mine, [&](float& v, const float* q) { sum = fmaf(v, *q, sum); });
#pragma unroll
                    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
                    if (lane == 0) sm.warp_sums[warp - B0] = sum;
                    mbar_arrive(&bars[TC_MEET]);
                    if (!wait(TC_MEET, met++)) return false;
                    if (id == 0) {
                        sum = 0.f;
                        for (int w = 0; w < 8; ++w) sum += sm.warp_sums[w];
                        a.final_dots[(zt * a.nseq + p.seq) * a.heads + head] = sum;
                    }
                    mbar_arrive(&bars[TC_MEET]);
                    if (!wait(TC_MEET, met++)) return false;
                }
            }
            return true;
        });
        if (summary && fine) {
            float4* q = reinterpret_cast<float4*>(a.carry + carry_at);
#pragma unroll
            for (int j = 0; j < HALF / 4; ++j) q[j * 128] = make_float4(S[2 * j].x, S[2 * j].y, S[2 * j + 1].x, S[2 * j + 1].y);
        }
    } else if (warp == M0) {
        // ---- the products, issued by one thread ----
        const uint32_t x = smem_addr(tile_x), y = smem_addr(tile_y), z = smem_addr(tile_z), s = smem_addr(tile_s),
                       w = smem_addr(tile_w);
        bool issued = false;
        fine = each_part([&](const TcPart& p, int chunks, uint32_t n0) {
            bool good = true;
            const bool start = starts_with_state(p);
            auto scores = [&](uint32_t n) {
                const uint32_t yn = y + (n & 1) * Shape::kTileX;
                issued = true;
#pragma unroll
                for (int k = 0; k < DX / 16; ++k)
                    tc_mma(tmem, tc_columns(x, PANEL, k), tc_columns(yn, PANEL, k), tc_idesc(C, false), k > 0);
                tc_commit(&bars[TC_SCORES]);
            };
            if (lane == 0) {
                for (int i = 0; i < chunks && good; ++i) {
                    const uint32_t n = n0 + i, half = n & 1;
                    const uint32_t yn = y + half * Shape::kTileX, zn = z + (Shape::kStageZ == 2 ? half * Shape::kTileZ : 0);
                    const bool some = i > 0 || start;
                    if (i == 0 || summary) {
                        good = lane_wait(TC_Y0 + half, n >> 1) &&
                               (summary || (lane_wait(TC_X, n) && (n == 0 || lane_wait(TC_OUT, n - 1))));
                        if (!good) break;
                        tc_after();
                        if (!summary) scores(n);
                    }
                    good = lane_wait(TC_STATE, n) && (summary || n == 0 || lane_wait(TC_TAKEN0 + (half ^ 1), (n - 1) >> 1));
                    if (!good) break;
                    tc_after();
                    if (!summary) {
                        if (some) {
#pragma unroll
                            for (int u = PO - 1; u >= 0; --u)
#pragma unroll
                                for (int k = 0; k < DX / 16; ++k)
                                    tc_mma(kOut, tc_columns(x, PANEL, k), tc_columns(s + u * (DZ * DX * 2), DZ * 128, k),
                                           tc_idesc(DZ, false), u < PO - 1 || k > 0);
                        }
                        tc_commit(&bars[TC_INTER]);  // once per chunk, whether there was a state or not
                    }
                    // outputs before the state: A works on them meanwhile
                    good = lane_wait(TC_WZ, n) && (summary || lane_wait(TC_WEIGHTED, n));
                    if (!good) break;
                    tc_after();
                    if (!summary) {
#pragma unroll
                        for (int u = PO - 1; u >= 0; --u)
#pragma unroll
                            for (int k = 0; k < C / 16; ++k)
                                tc_mma_ts(kOut, tmem + u * 64 + k * 8, tc_desc(zn + k * 2048, PANEL), tc_idesc(DZ, true),
                                          some || u < PO - 1 || k > 0);
                        tc_commit(&bars[TC_OUT]);
                    }
                    issued = true;
#pragma unroll
                    for (int k = 0; k < C / 16; ++k)
                        tc_mma(kAdd, tc_columns(w, PANEL, k), tc_desc(yn + k * 2048, PANEL), tc_idesc(DX, true), k > 0);
                    // The next chunk's scores between the pieces of the state, so that A has them in time;
                    // they go over this one's weighted scores, whose product is over by then.
                    if (i + 1 < chunks && !summary) {
                        good = lane_wait(TC_Y0 + (half ^ 1), (n + 1) >> 1) && lane_wait(TC_X, n + 1) && lane_wait(TC_OUT, n);
                        if (!good) break;
                        tc_after();
                        scores(n + 1);
                    }
#pragma unroll
                    for (int u = 1; u >= 0; --u)
#pragma unroll
                        for (int k = 0; k < C / 16; ++k)
                            tc_mma_ts(kAdd, kWz + u * 64 + k * 8, tc_desc(yn + k * 2048, PANEL), tc_idesc(DX, true), true);
                    tc_commit(&bars[TC_UPDATE0 + half]);
                }
            }
            return __all_sync(0xffffffffu, good) != 0;
        });
        // no product outlives the block, whoever has given up
        bool over = true;
        if (issued) {  // (by lane 0)
            tc_commit(&bars[TC_DRAIN]);
            over = mbar_wait_bounded(&bars[TC_DRAIN], 0, kDrainLimitNs);
        }
        fine = __all_sync(0xffffffffu, over) && fine;
    } else if (warp == M0 + 1) {
        // ---- decays: four tokens per lane ----
        const bf16* pg = static_cast<const bf16*>(a.decay.data) + row * a.decay.seq_stride + head;
        Two gone = {0.f, 0.f};
        fine = each_part([&](const TcPart& p, int chunks, uint32_t n0) {
            float g[4];
            auto fetch = [&](int i) {
                const int t = chunk_at(p, chunks, i);
                const int count = count_at(p, t);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    g[k] = 4 * lane + k < count ? to_f(pg[(t + 4 * lane + k) * a.decay.tok_stride]) : 0.f;
            };
            fetch(0);
            for (int i = 0; i < chunks; ++i) {
                const uint32_t n = n0 + i;
                Two d[4], sum;
                d[0] = log2_decay(g[0]);
#pragma unroll
                for (int k = 1; k < 4; ++k) d[k] = add(d[k - 1], log2_decay(g[k]));
                sum = d[3];
                if (i + 1 < chunks) fetch(i + 1);
#pragma unroll
                for (int o = 1; o < 32; o *= 2) {
                    const Two v = {__shfl_up_sync(0xffffffffu, sum.hi, o), __shfl_up_sync(0xffffffffu, sum.lo, o)};
                    if (lane >= o) sum = add(v, sum);
                }
                // factors of columns: to the end of their block of 32 tokens, or (reversed) from its start
                const int edge = reverse ? (lane & ~7) - 1 : lane | 7;
                const Two end = {__shfl_sync(0xffffffffu, sum.hi, edge & 31), __shfl_sync(0xffffffffu, sum.lo, edge & 31)};
                const Two all = {__shfl_sync(0xffffffffu, sum.hi, 31), __shfl_sync(0xffffffffu, sum.lo, 31)};
                Two before = {__shfl_up_sync(0xffffffffu, sum.hi, 1), __shfl_up_sync(0xffffffffu, sum.lo, 1)};
                if (lane == 0) before = {0.f, 0.f};
                if (n > 0 && !wait(TC_FREE, n - 1)) return false;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const Two G = add(before, d[k]);
                    sm.G[4 * lane + k] = make_float2(G.hi, G.lo);
                    const float to_end = (end.hi - G.hi) + (end.lo - G.lo);
                    sm.column[4 * lane + k] = edge < 0 ? 0.f : ex2(reverse ? -to_end : to_end);
                    sm.update[4 * lane + k] = ex2(reverse ? G.hi : (all.hi - G.hi) + (all.lo - G.lo)) * a.scale_update;
                }
                if (lane == 0) sm.total = ex2(all.hi), sm.all_hi = all.hi, sm.all_lo = all.lo;
                gone = add(gone, all);
                mbar_arrive(&bars[TC_DECAYS]);
            }
            if (summary && zt == 0 && lane == 0) {
                const int64_t at = ((int64_t)row * a.nsegments + seg) * a.heads + head;
                a.carry_decay[at] = gone.hi;
                a.carry_reset[at] = begins_at(p);
            }
            return true;
        });
    }
    else if (warp == M0 + 2) {
        // ---- rows of y and z ----
        const bf16* py = static_cast<const bf16*>(a.y.data) + row * a.y.seq + (head / a.y.share) * a.y.head;
        const bf16* pz = static_cast<const bf16*>(a.z.data) + row * a.z.seq + (head / a.z.share) * a.z.head + z0;
        fine = each_part([&](const TcPart& p, int chunks, uint32_t n0) {
            for (int i = 0; i < chunks; ++i) {
                const uint32_t n = n0 + i, half = n & 1;
                const int t = chunk_at(p, chunks, i);
                const int count = count_at(p, t);
                // A stage is free when the products of the chunk that was there are over and, in the
                // gradients, A has read its rows of z for the outputs.  (None of these barriers can be a
                // phase ahead of its wait: the next one needs the rows that are copied here.)
                if (n > 1 && !wait(TC_UPDATE0 + half, (n - 2) >> 1)) return false;
                tc_load<DX>(tile_y + half * Shape::kTileX, py + t * a.y.tok, a.y.tok, count, dx, lane);
                copy_commit();
                if (Shape::kStageZ == 1) {
                    copy_wait<0>();
                    fence_proxy_async_smem();
                    mbar_arrive(&bars[TC_Y0 + half]);
                    const int last = summary ? TC_UPDATE0 : TC_TAKEN0;
                    if (n > 0 && !wait(last + (half ^ 1), (n - 1) >> 1)) return false;
                } else if (BWD) {
                    if (n > 1 && !summary && !wait(TC_TAKEN0 + half, (n - 2) >> 1)) return false;
                }
                tc_load<DZ>(tile_z + (Shape::kStageZ == 2 ? half * Shape::kTileZ : 0), pz + t * a.z.tok, a.z.tok, count, dz,
                            lane);
                copy_commit();
                copy_wait<0>();
                fence_proxy_async_smem();
                if (Shape::kStageZ == 2) mbar_arrive(&bars[TC_Y0 + half]);
                mbar_arrive(&bars[TC_Z0 + half]);
            }
            return true;
        });
    } else {
        // ---- rows of x ----
        const bf16* px = static_cast<const bf16*>(a.x.data) + row * a.x.seq + (head / a.x.share) * a.x.head;
        if (!summary)
            fine = each_part([&](const TcPart& p, int chunks, uint32_t n0) {
                for (int i = 0; i < chunks; ++i) {
                    const uint32_t n = n0 + i;
                    const int t = chunk_at(p, chunks, i);
                    if (n > 0 && !wait(TC_INTER, n - 1)) return false;  // scores and those with the state
                    tc_load<DX>(tile_x, px + t * a.x.tok, a.x.tok, count_at(p, t), dx, lane);
                    copy_commit();
                    copy_wait<0>();
                    fence_proxy_async_smem();
                    mbar_arrive(&bars[TC_X]);
                }
                return true;
            });
    }
    copy_wait<0>();
    if (!fine && lane == 0) atomicCAS(err, 0, KERR_WAIT_TIMEOUT);  // `fine` is the whole warp's
    __syncwarp();
    tc_wait_st();
    tc_before();
    __syncthreads();
    if (warp == M0) {
        tc_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
    }
}

}  // namespace

template <int DX, int DZ, bool BWD>
cudaError_t launch_attn_tc(const AttnArgs& args, int* err, cudaStream_t s) {
    using Shape = TcShape<DX, DZ, BWD>;
    static LaunchCache cache;
    LaunchGeom g;
    cudaError_t e = cache.get(
        [](int dev, LaunchGeom* out) {
            return setup_persistent(k_linattn_tc<DX, DZ, BWD>, Shape::kThreads, tc_bytes<DX, DZ, BWD>(), dev, out);
        },
        &g);
    if (e != cudaSuccess) return e;
    AttnArgs a = args;
    const int64_t blocks = a.rows * a.nsegments * a.heads * a.ztiles;
    if (blocks > INT32_MAX) return cudaErrorInvalidValue;
    if (a.nsegments > 1) {
        a.summary = 1;
        k_linattn_tc<DX, DZ, BWD><<<(unsigned)blocks, Shape::kThreads, tc_bytes<DX, DZ, BWD>(), s>>>(a, err);
        e = cudaGetLastError();
        if (e == cudaSuccess) e = attn_carry_pass(a, a.ztiles * (DX * 128 / 4), s);
        if (e != cudaSuccess) return e;
        a.summary = 0;
    }
    k_linattn_tc<DX, DZ, BWD><<<(unsigned)blocks, Shape::kThreads, tc_bytes<DX, DZ, BWD>(), s>>>(a, err);
    return cudaGetLastError();
}

}  // namespace gbfft
