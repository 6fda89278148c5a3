// Group norm, channels last, with SiLU and a gate (fft_gnorm_forward, fft_gnorm_backward):
//   n = (x - mean) rstd over a sequence's tokens and a group's channels, y = n weight + bias,
//   p = y or y sigmoid(y),  out = p or p z sigmoid(z)
// and its gradients, with dy what reaches y and w = weight dy:
//   dx = rstd (w - mean(w) - n mean(w n)),  dweight = sum dy n,  dbias = sum dy.
// A few operations per element: bound by HBM where rows are whole 16-byte pieces.  Measured with inputs
// that change from call to call: 16384 rows of 2048 bfloat16 channels in 16 groups, gated, 43 us, 4.7 TB/s
// (69% of the copy rate; 81 with rows ahead in registers and one value to an instruction); its gradients
// for 8192 rows 60 us; 8 x 4096 tokens of 1024 channels, SiLU, 76 us (first pass 30, joining 13, second 30),
// x read twice; gradients of packed 20011 tokens of 330 float32 channels in groups of 55, value by value, 86 us.
// Sigmoids are approximate exponentials and reciprocals (2^-22): float32 gradients are 2.1e-7 from 64 bits
// where exact ones in float32 are 0.9e-7.
//
// Sequences of one token (what follows the heads of an attention) are read once: the lanes that
// share a group hold its values in registers, keep their channels' weights there too and take rows
// at a stride.  Longer sequences are read twice, by blocks of a tile of tokens and whole groups: the
// first pass leaves mean and sum of squares of every tile, joined by counts (Chan, Golub and
// LeVeque's update), the second one runs through the tiles from the last one on, which the first
// has left in L2.  Sums are taken about the mean of the few values that a thread holds at once and
// runs of them are joined about their means, so that neither a level that all values share nor one
// value far from the rest costs the others their digits.
#include "launch_cache.cuh"
#include "seq_common.cuh"
#include "seq_overlap.h"

namespace gbfft {
namespace {

constexpr int kThreads = 256;
constexpr int kTokenValues = 16;  // of a group per lane: more leave no registers in the gradients

struct GnArgs {
    fft_gnorm_desc d;
    fft_seq out;           // or dx
    fft_seq dout, dz;
    float* mean;           // [sequence][group]
    float* rstd;
    float* records;        // tiles' origin, sum and squares about it, or sums of w and w n: [record][group][3]
    float* sums;           // [sequence][group][2]: mean(w) and mean(w n)
    float* parts;          // [part][2][channels]: dweight, dbias
    int64_t rows, tile, tiles;
    int64_t walks;         // that all rows' tiles are dealt to for the sums of the gradients
    int cg, each, sets;    // channels of a group; groups of a block, blocks for all groups
};

// VEC values as pairs, two float32 operations to an instruction (of one value: the first of a pair
// whose second is 0 throughout).
template <int VEC>
struct Values {
    static constexpr int N = (VEC + 1) / 2;
    float2 v[N];
};
template <class T, int VEC>
__device__ __forceinline__ Values<VEC> unpack(const Pack<T, VEC>& p) {
    Values<VEC> x;
#pragma unroll
    for (int k = 0; k < VEC; k += 2) x.v[k / 2] = make_float2(to_f(p.v[k]), VEC > 1 ? to_f(p.v[k + (VEC > 1)]) : 0.f);
    return x;
}
template <class T, int VEC>
__device__ __forceinline__ Pack<T, VEC> rounded(const Values<VEC>& x) {
    Pack<T, VEC> o;
    if constexpr (VEC == 1) {
        o.v[0] = from_f<T>(x.v[0].x);
    } else {
#pragma unroll
        for (int k = 0; k < VEC; k += 2) {
            const Pack<T, 2> p = from_f2<T>(x.v[k / 2]);
            o.v[k] = p.v[0];
            o.v[k + 1] = p.v[1];
        }
    }
    return o;
}

// A thread's channels: weight and bias in registers.
template <class T, int VEC>
struct Channel {
    Values<VEC> w, b;
    __device__ __forceinline__ void load(const fft_gnorm_desc& d, int64_t c, bool in) {
        const int f32 = d.param_dtype == FFT_F32;
#pragma unroll
        for (int k = 0; k < Values<VEC>::N; ++k) w.v[k] = b.v[k] = splat(0.f);
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
            (k & 1 ? w.v[k / 2].y : w.v[k / 2].x) = in ? (d.weight ? ld_param<T>(d.weight, c + k, f32) : 1.f) : 0.f;
            (k & 1 ? b.v[k / 2].y : b.v[k / 2].x) = in && d.bias ? ld_param<T>(d.bias, c + k, f32) : 0.f;
        }
    }
};
template <class T, int VEC>
__device__ __forceinline__ Pack<T, VEC> load(const T* p, bool in) {
    Pack<T, VEC> v = {};
    if (in) v = ld_pack<VEC>(p);
    return v;
}

// Sigmoids of a pair; of a single value only the first.
template <int VEC>
__device__ __forceinline__ float2 sigmoids(float2 v) {
    if constexpr (VEC == 1) return make_float2(sigmoid(v.x), 0.f);
    return sigmoid2(v);
}
// What an output is of y and the gate, and (gradients) what of g reaches y and the gate: a pack's values,
// asked once what there is.
template <int VEC>
__device__ __forceinline__ void outcome(const fft_gnorm_desc& d, Values<VEC>& y, const Values<VEC>& z) {
    if (d.silu) {
#pragma unroll
        for (int k = 0; k < y.N; ++k) y.v[k] = mul2(y.v[k], sigmoids<VEC>(y.v[k]));
    }
    if (d.z.data) {
#pragma unroll
        for (int k = 0; k < y.N; ++k) y.v[k] = mul2(y.v[k], mul2(z.v[k], sigmoids<VEC>(z.v[k])));
    }
}
// The slope of SiLU at y, s being its sigmoid.
__device__ __forceinline__ float2 slope(float2 y, float2 s) {
    return mul2(s, fma2(y, fma2(s, splat(-1.f), splat(1.f)), splat(1.f)));
}
// y becomes what reaches it; g is used up.
template <int VEC>
__device__ __forceinline__ void reaches(const fft_gnorm_desc& d, Values<VEC>& y, const Values<VEC>& z, Values<VEC>& g,
                                        Values<VEC>& dz) {
    if (d.z.data) {
#pragma unroll
        for (int k = 0; k < y.N; ++k) {
            const float2 s = sigmoids<VEC>(z.v[k]);
            dz.v[k] = mul2(g.v[k], slope(z.v[k], s));
            g.v[k] = mul2(g.v[k], mul2(z.v[k], s));
        }
    } else {
#pragma unroll
        for (int k = 0; k < y.N; ++k) dz.v[k] = splat(0.f);
    }
    if (d.silu) {
#pragma unroll
        for (int k = 0; k < y.N; ++k) {
            const float2 s = sigmoids<VEC>(y.v[k]);
            dz.v[k] = mul2(dz.v[k], mul2(y.v[k], s));
            y.v[k] = mul2(g.v[k], slope(y.v[k], s));
        }
    } else {
#pragma unroll
        for (int k = 0; k < y.N; ++k) {
            dz.v[k] = mul2(dz.v[k], y.v[k]);
            y.v[k] = g.v[k];
        }
    }
}
__device__ __forceinline__ float2 minus(float v) { return splat(-v); }

// ---- sequences of one token -----------------------------------------------------------------

__device__ __forceinline__ float lanes_sum(float v, int lanes, unsigned mask) {
    for (int o = lanes / 2; o; o >>= 1) v += __shfl_xor_sync(mask, v, o);
    return v;
}

// `lanes` threads hold a group: NV packs of VEC values each.  They take the rows row0, row0 + step,
// ... ; of 16-byte packs the rows ahead wait in shared memory, where a thread reads only what it has
// copied itself, so that the ring needs neither a barrier nor registers (of single values the next
// row's are loaded ahead).  Blocks of an SM by the registers of so many values.
template <int VEC, int NV, bool BWD> constexpr int kGnBlocks = NV * VEC <= 8 && VEC > 1 ? (BWD ? 2 : 4) : (VEC > 1 && !BWD ? 2 : 1);
constexpr int kGnAhead = 4;  // rows of the ring
template <class T, int VEC, int NV, bool BWD>
__global__ void __launch_bounds__(kThreads, kGnBlocks<VEC, NV, BWD>) k_gn_token(const GnArgs a, int lanes, int64_t step) {
    constexpr int P = Values<VEC>::N;
    const fft_gnorm_desc& d = a.d;
    const int tid = (int)threadIdx.x, lane = tid & (lanes - 1);
    const unsigned mask = lanes == 32 ? 0xffffffffu : ((1u << lanes) - 1u) << ((tid & 31) & ~(lanes - 1));
    const int64_t sub = ((int64_t)blockIdx.x * kThreads + tid) / lanes;
    const int64_t group = sub % d.groups, row0 = sub / d.groups;
    if (row0 >= step) return;
    Channel<T, VEC> ch[NV];
    const int64_t c0 = group * a.cg + lane * VEC;
    const int hop = lanes * VEC;  // from one pack of the thread to the next
    bool in[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        in[j] = lane * VEC + j * hop < a.cg;
        ch[j].load(d, c0 + j * hop, in[j]);
    }
    Values<VEC> dw[BWD ? NV : 1], db[BWD ? NV : 1];
    if (BWD) {
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int k = 0; k < P; ++k) dw[j].v[k] = db[j].v[k] = splat(0.f);
    }
    const bool gate = d.z.data;
    const T* x = static_cast<const T*>(d.x.data) + row0 * d.x.seq_stride + c0;
    const T* z = static_cast<const T*>(d.z.data) + row0 * d.z.seq_stride + c0;
    const T* g = static_cast<const T*>(a.dout.data) + row0 * a.dout.seq_stride + c0;
    T* out = static_cast<T*>(a.out.data) + row0 * a.out.seq_stride + c0;
    T* oz = static_cast<T*>(a.dz.data) + row0 * a.dz.seq_stride + c0;
    float* mp = a.mean + row0 * d.groups + group;
    float* rp = a.rstd + row0 * d.groups + group;
    const int64_t hx = step * d.x.seq_stride, hz = step * d.z.seq_stride, hg = step * a.dout.seq_stride,
                  ho = step * a.out.seq_stride, hd = step * a.dz.seq_stride, hm = step * d.groups;
    constexpr bool RING = VEC > 1;
    constexpr int PIECES = NV * (BWD ? 3 : 2);
    extern __shared__ uint4 ring[];
    Pack<T, VEC> now[RING ? 1 : 3][RING ? 1 : NV];
    auto piece = [&](int stage, int k) { return ring + (stage * PIECES + k) * kThreads + tid; };
    // the next row of those that come, whether there is one or not
    auto fetch = [&](int stage, bool live) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const bool there = live && in[j];
            if constexpr (RING) {
                copy16(piece(stage, j), there ? x + j * hop : static_cast<const T*>(d.x.data), there);
                if (gate) copy16(piece(stage, NV + j), there ? z + j * hop : static_cast<const T*>(d.z.data), there);
                if (BWD) copy16(piece(stage, 2 * NV + j), there ? g + j * hop : static_cast<const T*>(a.dout.data), there);
            } else {
                now[0][j] = load<T, VEC>(x + j * hop, there);
                if (gate) now[1][j] = load<T, VEC>(z + j * hop, there);
                if (BWD) now[2][j] = load<T, VEC>(g + j * hop, there);
            }
        }
        if (RING) copy_commit();
        x += hx;
        if (gate) z += hz;
        if (BWD) g += hg;
    };
    if constexpr (RING) {
        for (int k = 0; k < kGnAhead - 1; ++k) fetch(k, row0 + k * step < a.rows);
    } else {
        fetch(0, true);
    }
    float nmean = 0.f, nrstd = 0.f;
    if (BWD) nmean = *mp, nrstd = *rp;
    const float inv = 1.f / (float)a.cg;
    int stage = 0;
    for (int64_t row = row0; row < a.rows; row += step) {
        Values<VEC> v[NV], zv[NV], gv[BWD ? NV : 1];
        if constexpr (RING) {
            fetch((stage + kGnAhead - 1) % kGnAhead, row + (kGnAhead - 1) * step < a.rows);
            copy_wait<kGnAhead - 1>();
        }
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            auto take = [&](int k) {
                if constexpr (RING) return *reinterpret_cast<const Pack<T, VEC>*>(piece(stage, k * NV + j));
                else return now[k][j];
            };
            v[j] = unpack<T, VEC>(take(0));
            zv[j] = unpack<T, VEC>(gate ? take(1) : Pack<T, VEC>{});
            if (BWD) gv[j] = unpack<T, VEC>(take(2));
        }
        stage = (stage + 1) % kGnAhead;
        float mean = nmean, rstd = nrstd;
        if (!RING) fetch(0, row + step < a.rows);
        if (BWD && row + step < a.rows) mp += hm, rp += hm, nmean = *mp, nrstd = *rp;
        if constexpr (!BWD) {
            // 2^-9 of the values (a group here has at most 2^9), so that sums of a type's lowest values stay finite
            constexpr float DOWN = 1.f / 512.f;
            static_assert(32 * kTokenValues * DOWN <= 1.f, "sums");
            float2 sum = splat(0.f), sq = splat(0.f);
#pragma unroll
            for (int j = 0; j < NV; ++j)
#pragma unroll
                for (int k = 0; k < P; ++k) sum = fma2(v[j].v[k], splat(DOWN), sum);
            mean = lanes_sum(sum.x + sum.y, lanes, mask) * (inv * (1.f / DOWN));
#pragma unroll
            for (int j = 0; j < NV; ++j)
#pragma unroll
                for (int k = 0; k < P; ++k) {
                    v[j].v[k] = in[j] ? add2(v[j].v[k], minus(mean)) : splat(0.f);
                    if (VEC == 1) v[j].v[k].y = 0.f;
                    sq = fma2(v[j].v[k], v[j].v[k], sq);
                }
            rstd = rsqrtf(fmaf(lanes_sum(sq.x + sq.y, lanes, mask), inv, d.eps));
            if (lane == 0) *mp = mean, *rp = rstd;
#pragma unroll
            for (int j = 0; j < NV; ++j) {
#pragma unroll
                for (int k = 0; k < P; ++k) v[j].v[k] = fma2(mul2(v[j].v[k], splat(rstd)), ch[j].w.v[k], ch[j].b.v[k]);
                outcome<VEC>(d, v[j], zv[j]);
                if (in[j]) st_pack<VEC>(out + j * hop, rounded<T, VEC>(v[j]));
            }
            mp += hm, rp += hm;
        } else {
            float2 s1 = splat(0.f), s2 = splat(0.f);
            Values<VEC> w[NV];
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                Values<VEC> dz;
#pragma unroll
                for (int k = 0; k < P; ++k) {
                    v[j].v[k] = mul2(add2(v[j].v[k], minus(mean)), splat(rstd));
                    if (VEC == 1) v[j].v[k].y = 0.f;
                    w[j].v[k] = fma2(v[j].v[k], ch[j].w.v[k], ch[j].b.v[k]);
                }
                reaches<VEC>(d, w[j], zv[j], gv[j], dz);
                if (in[j] && gate) st_pack<VEC>(oz + j * hop, rounded<T, VEC>(dz));
#pragma unroll
                for (int k = 0; k < P; ++k) {
                    dw[j].v[k] = fma2(w[j].v[k], v[j].v[k], dw[j].v[k]);
                    db[j].v[k] = add2(w[j].v[k], db[j].v[k]);
                    w[j].v[k] = in[j] ? mul2(w[j].v[k], ch[j].w.v[k]) : splat(0.f);
                    s1 = add2(s1, w[j].v[k]);
                    s2 = fma2(w[j].v[k], v[j].v[k], s2);
                }
            }
            const float m1 = lanes_sum(s1.x + s1.y, lanes, mask) * inv, m2 = lanes_sum(s2.x + s2.y, lanes, mask) * inv;
#pragma unroll
            for (int j = 0; j < NV; ++j) {
#pragma unroll
                for (int k = 0; k < P; ++k)
                    w[j].v[k] = mul2(add2(w[j].v[k], fma2(v[j].v[k], minus(m2), minus(m1))), splat(rstd));
                if (in[j]) st_pack<VEC>(out + j * hop, rounded<T, VEC>(w[j]));
            }
            if (gate) oz += hd;
        }
        out += ho;
    }
    copy_wait<0>();  // no copy under way at the end
    if constexpr (BWD) {
        if (!a.parts) return;
        float* p = a.parts + row0 * 2 * d.channels + c0;
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int k = 0; k < VEC; ++k)
                if (in[j]) {
                    p[j * hop + k] = k & 1 ? dw[j].v[k / 2].y : dw[j].v[k / 2].x;
                    p[d.channels + j * hop + k] = k & 1 ? db[j].v[k / 2].y : db[j].v[k / 2].x;
                }
    }
}

// ---- longer sequences -----------------------------------------------------------------------

// The block's part of the grid: a tile of tokens, a set of whole groups.  Thread (tx, ty) takes the
// packs tx, tx + blockDim.x, ... of the set's channels and every blockDim.y-th token.
struct TileAt {
    int64_t row, tile, t0, t1;
    int group0, groups;
};
__device__ __forceinline__ TileAt tile_of_set(const GnArgs& a, int set, int64_t n) {
    TileAt t;
    t.group0 = set * a.each;
    t.tile = n % a.tiles;
    t.row = n / a.tiles;
    t.t0 = t.tile * a.tile;
    t.t1 = t.t0 + a.tile < a.d.length ? t.t0 + a.tile : a.d.length;
    t.groups = (int)a.d.groups - t.group0 < a.each ? (int)a.d.groups - t.group0 : a.each;
    return t;
}
__device__ __forceinline__ TileAt tile_at(const GnArgs& a, bool last_first) {
    const int64_t b = last_first ? (int64_t)gridDim.x - 1 - blockIdx.x : blockIdx.x;
    return tile_of_set(a, (int)(b % a.sets), b / a.sets);
}
// Tokens of one sequence in a tile, from token `at` on; offsets of any kind stay in the tile.
__device__ __forceinline__ SeqAt part_at(const GnArgs& a, int64_t row, int64_t at, int64_t t1) {
    SeqAt s = seq_at(a.d.offsets, a.d.nseq, a.d.length, row, at);
    s.begin = at;
    s.end = s.end <= at ? at + 1 : (s.end > t1 ? t1 : s.end);
    return s;
}
// Where a tile's record of a sequence stands: with packed rows both grow along the row.
__device__ __forceinline__ int64_t record_of(const GnArgs& a, int64_t row, int64_t tile, int64_t q) {
    return a.d.offsets ? tile + q : row * a.tiles + tile;
}

// done(group, lane, first tx, count) for every group of the set: a warp takes one, whose values the
// threads first .. first + count - 1 of every ty have left.
template <class Join>
__device__ __forceinline__ void by_group(int groups, int packs, int single, Join done) {
    const int tid = (int)(threadIdx.y * blockDim.x + threadIdx.x), lane = tid & 31, warps = (int)(blockDim.x * blockDim.y) / 32;
    for (int g = tid / 32; g < groups; g += warps) {
        // the threads tx of group g: all of them where a set is one group
        const int first = single ? 0 : g * packs, count = single ? (int)blockDim.x : packs;
        done(g, lane, first, count);
    }
}

// What a run of values leaves: how many (exact: a tile has fewer than 2^24), their mean in two floats, the
// sum of squares about it.
struct Moments {
    float n, hi, lo, m2;
};
__device__ __forceinline__ Moments join(const Moments& a, const Moments& b) {
    if (b.n == 0.f) return a;
    if (a.n == 0.f) return b;
    const float n = a.n + b.n, part = b.n * rcp(n), delta = (b.hi - a.hi) + (b.lo - a.lo), move = delta * part;
    const float hi = a.hi + move, t = hi - a.hi;
    const float lost = (a.hi - (hi - t)) + (move - t);  // by the rounding of hi
    return {n, hi, a.lo + lost, a.m2 + b.m2 + delta * (a.n * part) * delta};
}

template <class T, int VEC>
__global__ void __launch_bounds__(kThreads) k_gn_moments(const GnArgs a) {
    __shared__ Moments red[kThreads];
    const fft_gnorm_desc& d = a.d;
    const TileAt t = tile_at(a, false);
    const int tx = (int)threadIdx.x, ty = (int)threadIdx.y, bx = (int)blockDim.x, by = (int)blockDim.y;
    const int packs = a.cg / VEC, all = packs * t.groups;
    const T* base = static_cast<const T*>(d.x.data) + t.row * d.x.seq_stride + (int64_t)t.group0 * a.cg;
    constexpr int DEEP = VEC > 1 ? 8 : 16;  // tokens of a run
    for (int64_t at = t.t0; at < t.t1;) {
        const SeqAt s = part_at(a, t.row, at, t.t1);
        const int64_t first = s.begin + ty, hop = by * d.x.tok_stride;
        const int count = s.end > first ? (int)((s.end - first + by - 1) / by) : 0;
        Moments all_of = {};
        for (int p = tx; p < all; p += bx) {
            const T* x = base + p * VEC + first * d.x.tok_stride;
            for (int i0 = 0; i0 < count; i0 += DEEP) {
                Pack<T, VEC> px[DEEP];
#pragma unroll
                for (int u = 0; u < DEEP; ++u) px[u] = load<T, VEC>(x, i0 + u < count), x += hop;
                const int live = count - i0 < DEEP ? count - i0 : DEEP;
                const float n = (float)(live * VEC), inv = rcp(n);
                // near the mean, and the value itself where all are alike
                const float one = to_f(px[0].v[0]);
                float2 v = splat(0.f);
#pragma unroll
                for (int u = 0; u < DEEP; ++u) {
                    if (u >= live) break;
                    const Values<VEC> e = unpack<T, VEC>(px[u]);
#pragma unroll
                    for (int k = 0; k < e.N; ++k) {
                        float2 w = add2(e.v[k], minus(one));
                        if (VEC == 1) w.y = 0.f;
                        v = fma2(w, splat(inv), v);
                    }
                }
                const float mid = one + (v.x + v.y);
                float2 v1 = splat(0.f), v2 = splat(0.f);
#pragma unroll
                for (int u = 0; u < DEEP; ++u) {
                    if (u >= live) break;
                    const Values<VEC> e = unpack<T, VEC>(px[u]);
#pragma unroll
                    for (int k = 0; k < e.N; ++k) {
                        float2 w = add2(e.v[k], minus(mid));
                        if (VEC == 1) w.y = 0.f;
                        v1 = add2(v1, w);
                        v2 = fma2(w, w, v2);
                    }
                }
                const float rest = (v1.x + v1.y) * inv, squares = v2.x + v2.y;
                // (squares beyond float32 stay infinite)
                all_of = join(all_of, {n, mid, rest, squares < INFINITY ? fmaf(-rest * n, rest, squares) : squares});
            }
        }
        red[ty * bx + tx] = all_of;
        __syncthreads();
        by_group(t.groups, packs, a.each == 1, [&](int g, int lane, int first_tx, int threads) {
            Moments m = {};
            for (int i = lane; i < threads * by; i += 32) m = join(m, red[i / threads * bx + first_tx + i % threads]);
#pragma unroll
            for (int o = 16; o; o >>= 1)
                m = join(m, {__shfl_xor_sync(0xffffffffu, m.n, o), __shfl_xor_sync(0xffffffffu, m.hi, o),
                             __shfl_xor_sync(0xffffffffu, m.lo, o), __shfl_xor_sync(0xffffffffu, m.m2, o)});
            if (lane == 0) {
                float* r = a.records + (record_of(a, t.row, t.tile, s.q) * d.groups + t.group0 + g) * 3;
                r[0] = m.hi;  // what the sums are counted from
                r[1] = m.n * m.lo;
                r[2] = fmaf(m.n * m.lo, m.lo, m.m2);
            }
        });
        __syncthreads();
        at = s.end;
    }
}

// Joins the records of a sequence: a warp for each of its groups.
template <bool BWD>
__global__ void __launch_bounds__(kThreads) k_gn_join(const GnArgs a) {
    const fft_gnorm_desc& d = a.d;
    const int64_t i = ((int64_t)blockIdx.x * kThreads + threadIdx.x) / 32;
    const int lane = (int)threadIdx.x & 31;
    if (i >= d.nseq * d.groups) return;
    const int64_t q = i / d.groups, g = i % d.groups;
    int64_t begin = 0, end = d.length;
    if (d.offsets) {  // offsets of any kind: records that there are
        begin = d.offsets[q], end = d.offsets[q + 1];
        begin = begin < 0 ? 0 : (begin > d.length ? d.length : begin);
        end = end > d.length ? d.length : end;
    }
    // sums about the origin of the sequence's first tile: few operations, since those in 64 bits are slow
    double t1 = 0.0, t2 = 0.0;
    float origin = 0.f;
    if (end > begin) {
        const int64_t first = begin / a.tile, last = (end - 1) / a.tile;
        if (!BWD) origin = a.records[(record_of(a, q, first, q) * d.groups + g) * 3];
        for (int64_t k = first + lane; k <= last; k += 32) {
            const float* r = a.records + (record_of(a, q, k, q) * d.groups + g) * 3;
            if constexpr (BWD) {
                t1 += r[0];
                t2 += r[1];
            } else {
                const int64_t lo = k * a.tile > begin ? k * a.tile : begin,
                              hi = (k + 1) * a.tile < end ? (k + 1) * a.tile : end;
                const double c = (double)((int)(hi - lo) * (int64_t)a.cg), o = (double)r[0] - (double)origin;
                t1 += fma(c, o, (double)r[1]);
                t2 += fma(fma(c, o, 2.0 * (double)r[1]), o, (double)r[2]);
            }
        }
    }
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        t1 += __shfl_xor_sync(0xffffffffu, t1, o);
        t2 += __shfl_xor_sync(0xffffffffu, t2, o);
    }
    if (lane) return;
    const double count = end > begin ? (double)(end - begin) * a.cg : 1.0;
    if constexpr (BWD) {
        a.sums[i * 2] = (float)(t1 / count);
        a.sums[i * 2 + 1] = (float)(t2 / count);
    } else {
        const double mean = t1 / count, var = t2 / count - mean * mean;
        a.mean[i] = (float)((double)origin + mean);
        a.rstd[i] = (float)(1.0 / sqrt((var < 0.0 ? 0.0 : var) + (double)d.eps));
    }
}

// Rows ahead of a thread of the second pass, in pieces of 16 bytes.  (Single values
// are loaded four tokens at a time instead, by as many blocks as 64 registers leave room for.)
template <class T, int VEC, bool BWD>
struct GnRing {
    static constexpr int kAhead = 6, kPieces = BWD ? 3 : 2;
    static constexpr size_t kBytes = VEC > 1 ? (size_t)kAhead * kPieces * 16 * kThreads : 0;
};

// Second pass: outputs, or (backward) gradients of x and z.
template <class T, int VEC, bool BWD>
__global__ void __launch_bounds__(kThreads, VEC > 1 ? 2 : 4) k_gn_apply(const GnArgs a) {
    const fft_gnorm_desc& d = a.d;
    const TileAt t = tile_at(a, true);
    const int tx = (int)threadIdx.x, ty = (int)threadIdx.y, bx = (int)blockDim.x, by = (int)blockDim.y;
    const int packs = a.cg / VEC, all = packs * t.groups;
    using Ring = GnRing<T, VEC, BWD>;
    constexpr bool RING = Ring::kBytes > 0;
    constexpr int AHEAD = Ring::kAhead;
    extern __shared__ uint4 ring[];
    auto piece = [&](int stage, int k) {
        return reinterpret_cast<char*>(ring) + ((stage * Ring::kPieces + k) * kThreads + ty * bx + tx) * 16;
    };
    const bool gate = d.z.data;
    for (int64_t at = t.t0; at < t.t1;) {
        const SeqAt s = part_at(a, t.row, at, t.t1);
        for (int p = tx; p < all; p += bx) {
            const int64_t g = t.group0 + p / packs, c = (int64_t)t.group0 * a.cg + p * VEC;
            const float mean = a.mean[s.q * d.groups + g], rstd = a.rstd[s.q * d.groups + g];
            float s1 = 0.f, s2 = 0.f;
            if (BWD) s1 = a.sums[(s.q * d.groups + g) * 2], s2 = a.sums[(s.q * d.groups + g) * 2 + 1];
            Channel<T, VEC> ch;
            ch.load(d, c, true);
            const T* x = static_cast<const T*>(d.x.data) + t.row * d.x.seq_stride + c;
            const T* z = static_cast<const T*>(d.z.data) + t.row * d.z.seq_stride + c;
            const T* go = BWD ? static_cast<const T*>(a.dout.data) + t.row * a.dout.seq_stride + c : nullptr;
            T* out = static_cast<T*>(a.out.data) + t.row * a.out.seq_stride + c;
            T* dz = BWD ? static_cast<T*>(a.dz.data) + t.row * a.dz.seq_stride + c : nullptr;
            auto finish = [&](const Pack<T, VEC>& px, const Pack<T, VEC>& pz, const Pack<T, VEC>& pg, int64_t i) {
                Values<VEC> n = unpack<T, VEC>(px), y, dzv, zv = unpack<T, VEC>(pz), gv = unpack<T, VEC>(pg);
#pragma unroll
                for (int k = 0; k < n.N; ++k) {
                    n.v[k] = mul2(add2(n.v[k], minus(mean)), splat(rstd));
                    y.v[k] = fma2(n.v[k], ch.w.v[k], ch.b.v[k]);
                }
                if constexpr (BWD) {
                    reaches<VEC>(d, y, zv, gv, dzv);
#pragma unroll
                    for (int k = 0; k < n.N; ++k)
                        y.v[k] = mul2(fma2(y.v[k], ch.w.v[k], fma2(n.v[k], minus(s2), minus(s1))), splat(rstd));
                    if (gate) st_pack<VEC>(dz + i * a.dz.tok_stride, rounded<T, VEC>(dzv));
                } else {
                    outcome<VEC>(d, y, zv);
                }
                st_pack<VEC>(out + i * a.out.tok_stride, rounded<T, VEC>(y));
            };
            if constexpr (RING) {
                // rows ahead wait in shared memory, where a thread reads only what it has copied itself
                int64_t from = s.begin + ty;
                auto fetch = [&](int stage) {
                    const bool in = from < s.end;
                    copy16(piece(stage, 0), in ? x + from * d.x.tok_stride : x, in);
                    if (gate) copy16(piece(stage, 1), in ? z + from * d.z.tok_stride : z, in);
                    if (BWD) copy16(piece(stage, 2), in ? go + from * a.dout.tok_stride : go, in);
                    copy_commit();
                    from += by;
                };
                for (int k = 0; k < AHEAD - 1; ++k) fetch(k);
                int stage = 0;
                for (int64_t i = s.begin + ty; i < s.end; i += by) {
                    fetch((stage + AHEAD - 1) % AHEAD);
                    copy_wait<AHEAD - 1>();
                    Pack<T, VEC> pz = {}, pg = {};
                    const Pack<T, VEC> px = *reinterpret_cast<const Pack<T, VEC>*>(piece(stage, 0));
                    if (gate) pz = *reinterpret_cast<const Pack<T, VEC>*>(piece(stage, 1));
                    if (BWD) pg = *reinterpret_cast<const Pack<T, VEC>*>(piece(stage, 2));
                    finish(px, pz, pg, i);
                    stage = (stage + 1) % AHEAD;
                }
                copy_wait<0>();
            } else {
                constexpr int DEEP = 4;
                const int64_t first = s.begin + ty, hx = by * d.x.tok_stride, hz = by * d.z.tok_stride,
                              hg = by * a.dout.tok_stride;
                const T *xp = x + first * d.x.tok_stride, *zp = z + first * d.z.tok_stride,
                        *gp = go + first * a.dout.tok_stride;
                const int count = s.end > first ? (int)((s.end - first + by - 1) / by) : 0;
                for (int i0 = 0; i0 < count; i0 += DEEP) {
                    Pack<T, VEC> px[DEEP], pz[DEEP], pg[DEEP];
#pragma unroll
                    for (int u = 0; u < DEEP; ++u) {
                        const bool in = i0 + u < count;
                        px[u] = load<T, VEC>(xp, in);
                        pz[u] = load<T, VEC>(zp, in && gate);
                        pg[u] = load<T, VEC>(gp, in && BWD);
                        xp += hx;
                        if (gate) zp += hz;
                        if (BWD) gp += hg;
                    }
#pragma unroll
                    for (int u = 0; u < DEEP; ++u)
                        if (i0 + u < count) finish(px[u], pz[u], pg[u], first + (i0 + u) * by);
                }
            }
        }
        at = s.end;
    }
}

// First pass of the gradients: sums of w and w n of every part, of dy n and dy of every channel.  A block
// takes a set's tiles at a stride and leaves one row of channel sums for all of them.
template <class T, int VEC>
__global__ void __launch_bounds__(kThreads, VEC > 1 ? 2 : 4) k_gn_sums(const GnArgs a) {
    __shared__ float red[2][kThreads];
    extern __shared__ float chans[];  // [2][ty][tx * VEC]
    const fft_gnorm_desc& d = a.d;
    const int set = (int)(blockIdx.x % (unsigned)a.sets);
    const int64_t walk = blockIdx.x / (unsigned)a.sets, all_tiles = a.rows * a.tiles;
    const int64_t c0 = (int64_t)set * a.each * a.cg;
    const int tx = (int)threadIdx.x, ty = (int)threadIdx.y, bx = (int)blockDim.x, by = (int)blockDim.y;
    const int packs = a.cg / VEC, all = packs * tile_of_set(a, set, 0).groups, tid = ty * bx + tx;
    const bool gate = d.z.data;
    // packs outermost, since a channel's sums run over all parts; with several rounds of packs (a
    // set of one group of many channels) the parts' sums go on from what is there
    for (int p0 = 0; p0 < all; p0 += bx) {
        const int p = p0 + tx;
        const bool in = p < all;
        const int64_t c = c0 + p * VEC;
        Channel<T, VEC> ch;
        ch.load(d, c, in);
        Values<VEC> dw, db;
#pragma unroll
        for (int k = 0; k < dw.N; ++k) dw.v[k] = db.v[k] = splat(0.f);
        for (int64_t n = walk; n < all_tiles; n += a.walks) {
            const TileAt t = tile_of_set(a, set, n);
            for (int64_t at = t.t0; at < t.t1;) {
                const SeqAt s = part_at(a, t.row, at, t.t1);
                float s1 = 0.f, s2 = 0.f;
                if (in) {
                    const int64_t g = t.group0 + p / packs;
                    const float mean = a.mean[s.q * d.groups + g], rstd = a.rstd[s.q * d.groups + g];
                    const T* x = static_cast<const T*>(d.x.data) + t.row * d.x.seq_stride + c;
                    const T* z = static_cast<const T*>(d.z.data) + t.row * d.z.seq_stride + c;
                    const T* go = static_cast<const T*>(a.dout.data) + t.row * a.dout.seq_stride + c;
                    float2 p1 = splat(0.f), p2 = splat(0.f);
                    constexpr int DEEP = VEC == 1 ? 4 : 2;  // tokens loaded before the first of them is used
                    const int64_t first = s.begin + ty, hx = by * d.x.tok_stride, hz = by * d.z.tok_stride,
                                  hg = by * a.dout.tok_stride;
                    x += first * d.x.tok_stride, go += first * a.dout.tok_stride;
                    if (gate) z += first * d.z.tok_stride;
                    const int count = s.end > first ? (int)((s.end - first + by - 1) / by) : 0;
                    for (int i0 = 0; i0 < count; i0 += DEEP) {
                        Pack<T, VEC> px[DEEP], pz[DEEP], pg[DEEP];
#pragma unroll
                        for (int u = 0; u < DEEP; ++u) {
                            const bool in = i0 + u < count;
                            px[u] = load<T, VEC>(x, in);
                            pg[u] = load<T, VEC>(go, in);
                            pz[u] = load<T, VEC>(z, in && gate);
                            x += hx, go += hg;
                            if (gate) z += hz;
                        }
#pragma unroll
                        for (int u = 0; u < DEEP; ++u) {
                            Values<VEC> n = unpack<T, VEC>(px[u]), y, dzv, zv = unpack<T, VEC>(pz[u]), gv = unpack<T, VEC>(pg[u]);
#pragma unroll
                            for (int k = 0; k < n.N; ++k) {
                                n.v[k] = mul2(add2(n.v[k], minus(mean)), splat(rstd));
                                if (VEC == 1) n.v[k].y = 0.f;
                                y.v[k] = fma2(n.v[k], ch.w.v[k], ch.b.v[k]);
                            }
                            reaches<VEC>(d, y, zv, gv, dzv);
#pragma unroll
                            for (int k = 0; k < n.N; ++k) {
                                if (i0 + u >= count) break;  // (a statistic that is no number times 0 is none)
                                const float2 dn = mul2(y.v[k], n.v[k]);
                                dw.v[k] = add2(dw.v[k], dn);
                                db.v[k] = add2(db.v[k], y.v[k]);
                                p1 = fma2(y.v[k], ch.w.v[k], p1);
                                p2 = fma2(dn, ch.w.v[k], p2);
                            }
                        }
                    }
                    s1 = p1.x + p1.y, s2 = p2.x + p2.y;
                }
                red[0][tid] = s1, red[1][tid] = s2;
                __syncthreads();
                by_group(t.groups, packs, a.each == 1, [&](int g, int lane, int first, int count) {
                    float v1 = 0.f, v2 = 0.f;
                    for (int i = lane; i < count * by; i += 32) {
                        const int at2 = i / count * bx + first + i % count;
                        v1 += red[0][at2], v2 += red[1][at2];
                    }
#pragma unroll
                    for (int o = 16; o; o >>= 1) v1 += __shfl_xor_sync(0xffffffffu, v1, o), v2 += __shfl_xor_sync(0xffffffffu, v2, o);
                    if (lane == 0) {
                        float* r = a.records + (record_of(a, t.row, t.tile, s.q) * d.groups + t.group0 + g) * 3;
                        r[0] = p0 ? r[0] + v1 : v1;
                        r[1] = p0 ? r[1] + v2 : v2;
                    }
                });
                __syncthreads();
                at = s.end;
            }
        }
        if (!a.parts) continue;
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
            chans[tid * VEC + k] = k & 1 ? dw.v[k / 2].y : dw.v[k / 2].x;
            chans[(bx * by + tid) * VEC + k] = k & 1 ? db.v[k / 2].y : db.v[k / 2].x;
        }
        __syncthreads();
        float* out = a.parts + walk * 2 * d.channels + c0 + (int64_t)p0 * VEC;
        const int width = (all - p0 < bx ? all - p0 : bx) * VEC;
        for (int i = tid; i < 2 * width; i += bx * by) {
            const int which = i / width, k = i % width;
            float v = 0.f;
            for (int r = 0; r < by; ++r) v += chans[(which * by + r) * bx * VEC + k];
            out[which * d.channels + k] = v;
        }
        __syncthreads();
    }
}

// ---- host -----------------------------------------------------------------------------------

constexpr int64_t kMaxElements = INT64_C(1) << 58, kMaxTokStride = INT64_C(1) << 26;

int status(cudaError_t e) {
    return e == cudaSuccess ? FFT_OK : (e == cudaErrorInvalidValue ? FFT_ERR_UNSUPPORTED_SIZE : FFT_ERR_CUDA);
}

#define TRY(x)                         \
    do {                               \
        const int rc_ = (x);           \
        if (rc_ != FFT_OK) return rc_; \
    } while (0)

int check_rows(const fft_seq& s, const fft_gnorm_desc& d, bool output) {
    if (!s.data) return d.length == 0 ? FFT_OK : FFT_ERR_INVALID_ARG;
    if (s.tok_stride < 0 || s.seq_stride < 0) return FFT_ERR_INVALID_ARG;
    if (s.tok_stride > kMaxTokStride || (!d.offsets && s.seq_stride > kMaxElements / (d.nseq + 1)))
        return FFT_ERR_UNSUPPORTED_SIZE;
    if (output && d.length > 1 && s.tok_stride < d.channels) return FFT_ERR_INVALID_ARG;
    if (output && !d.offsets && d.nseq > 1 && d.length > 0 && s.seq_stride < d.channels) return FFT_ERR_INVALID_ARG;
    return aligned_to(s.data, dtype_size(d.dtype)) ? FFT_OK : FFT_ERR_MISALIGNED;
}
int check_gnorm(const fft_gnorm_desc* d, bool pointers) {
    if (!d || d->dtype < FFT_F32 || d->dtype > FFT_F16 || (d->silu != 0 && d->silu != 1) ||
        (d->param_dtype != FFT_F32 && d->param_dtype != d->dtype))
        return FFT_ERR_INVALID_ARG;
    if (d->nseq < 1 || d->length < 0 || d->channels < 1 || d->groups < 1 || d->channels % d->groups)
        return FFT_ERR_INVALID_ARG;
    if (!(d->eps >= 0.f)) return FFT_ERR_INVALID_ARG;
    if (d->nseq > INT32_MAX || d->length > INT32_MAX - 65536 || d->channels > FFT_GNORM_MAX_CHANNELS)
        return FFT_ERR_UNSUPPORTED_SIZE;
    if (!aligned_to(d->offsets, 8)) return FFT_ERR_MISALIGNED;
    if (!pointers) return FFT_OK;
    const size_t p = dtype_size(d->param_dtype);
    if (!aligned_to(d->weight, p) || !aligned_to(d->bias, p)) return FFT_ERR_MISALIGNED;
    TRY(check_rows(d->x, *d, false));
    return d->z.data ? check_rows(d->z, *d, false) : FFT_OK;
}

int64_t up16(int64_t bytes) { return (bytes + 15) / 16 * 16; }
bool by_token(const fft_gnorm_desc& d) {  // sequences of one token whose groups fit their lanes
    return !d.offsets && d.length == 1 && d.channels / d.groups <= 32 * kTokenValues;
}
// Lanes that share a group of the token kernel: a pack of one value each, two longer ones (fewer
// steps of their sums), up to a warp.
int token_lanes(int64_t packs, bool wide) {
    int lanes = 1;
    while (lanes < 32 && lanes * (wide ? 2 : 1) < packs) lanes *= 2;
    return lanes;
}
// Rows that the token kernel's threads start at: as many as the SMs hold, at three blocks each where
// every start leaves a row of partial sums.
int64_t token_step(const fft_gnorm_desc& d, int lanes, bool backward) {
    const int64_t subs = (int64_t)num_sms() * (backward ? 3 : 6) * (kThreads / lanes);
    const int64_t step = subs / d.groups;
    return step < 1 ? 1 : (step > d.nseq ? d.nseq : step);
}
// Tokens of a tile: as many as leave every SM eight blocks of 512 channels, 16 to 128.  Measured: 8 x 4096
// tokens of 1024 channels 94 us with tiles of 16 and 72 us with tiles of 32 (and a first pass of 26 us).
int64_t tile_of(const fft_gnorm_desc& d) {
    const int64_t rows = d.offsets ? 1 : d.nseq, wide = (d.channels + 511) / 512;
    int64_t tile = 128;
    while (tile > 16 && rows * ((d.length + tile - 1) / tile) * wide < (int64_t)num_sms() * 8) tile /= 2;
    return tile;
}
// Groups of a block and blocks for all of them, of like size, with packs of `vec` values.
void gnorm_sets(const fft_gnorm_desc& d, int64_t vec, GnArgs* a) {
    const int64_t packs = d.channels / d.groups / vec;
    int64_t each = packs >= kThreads ? 1 : kThreads / packs;
    if (each > d.groups) each = d.groups;
    a->sets = (int)((d.groups + each - 1) / each);
    a->each = (int)((d.groups + a->sets - 1) / a->sets);
    // Walks of the gradients' sums, each of which leaves two rows of channels: eight blocks for every SM (fewer
    // where a block takes its channels in several rounds, one at least), and no more than 65536 tokens for a
    // walk, whose threads' sums are float32.  One for every tile instead left rows of four times the bytes of
    // x where sequences are short (16384 rows of 4096 channels in 4 groups: 538 MB of workspace, 21 MB now).
    const int64_t rounds = (packs + kThreads - 1) / kThreads, tokens = a->rows * d.length;
    const int64_t most = a->rows * a->tiles, sms = num_sms();
    int64_t walks = sms * 8 / (a->sets * rounds);
    if (walks < sms / a->sets) walks = sms / a->sets;
    if (walks < tokens / 65536) walks = tokens / 65536;
    a->walks = walks < 1 ? 1 : (walks < most ? walks : most);
}
int64_t gnorm_layout(const fft_gnorm_desc& d, bool backward, GnArgs* a, char* w) {
    int64_t at = 0;
    auto take = [&](int64_t floats) {
        float* p = reinterpret_cast<float*>(w ? w + at : nullptr);
        at += up16(floats * 4);
        return p;
    };
    a->rows = d.offsets ? 1 : d.nseq;
    a->cg = (int)(d.channels / d.groups);
    if (by_token(d)) {
        // packs of one value, where rows are off 16-byte boundaries, have no fewer lanes
        const int64_t vec = 16 / (int64_t)dtype_size(d.dtype);
        if (backward) a->parts = take(token_step(d, token_lanes((a->cg + vec - 1) / vec, true), true) * 2 * d.channels);
        return at;
    }
    a->tile = tile_of(d);
    a->tiles = (d.length + a->tile - 1) / a->tile;
    a->records = take((a->rows * a->tiles + (d.offsets ? d.nseq : 0)) * d.groups * 3);
    if (backward) {
        a->sums = take(d.nseq * d.groups * 2);
        // rows off 16-byte boundaries go value by value, which makes no fewer sets and so no more walks
        const int64_t vec = 16 / (int64_t)dtype_size(d.dtype);
        gnorm_sets(d, a->cg % vec ? 1 : vec, a);
        a->parts = take(a->walks * 2 * d.channels);
    }
    return at;
}

bool vec_rows(const fft_seq& s, const fft_gnorm_desc& d, int64_t vec) {
    return !s.data || (aligned_to(s.data, 16) && (d.length < 2 || s.tok_stride % vec == 0) &&
                       (d.offsets || d.nseq < 2 || s.seq_stride % vec == 0));
}

template <class T, int VEC, int NV, bool BWD>
cudaError_t launch_token(const GnArgs& a, unsigned blocks, int lanes, int64_t step, cudaStream_t s) {
    constexpr size_t bytes = VEC > 1 ? (size_t)kGnAhead * NV * (BWD ? 3 : 2) * 16 * kThreads : 0;
    if constexpr (bytes > 0) {
        static LaunchCache cache;
        LaunchGeom g;
        const cudaError_t e = cache.get(
            [](int dev, LaunchGeom* out) {
                return setup_persistent(k_gn_token<T, VEC, NV, BWD>, kThreads, bytes, dev, out);
            },
            &g);
        if (e != cudaSuccess) return e;
    }
    k_gn_token<T, VEC, NV, BWD><<<blocks, kThreads, bytes, s>>>(a, lanes, step);
    return cudaGetLastError();
}
template <class T, int VEC, bool BWD>
cudaError_t run_token(const GnArgs& a, int64_t* parts, cudaStream_t s) {
    const int packs = a.cg / VEC, lanes = token_lanes(packs, VEC > 1);
    const int nv = (packs + lanes - 1) / lanes;
    const int64_t step = token_step(a.d, lanes, BWD);
    const int64_t blocks = (step * a.d.groups * lanes + kThreads - 1) / kThreads;
    if (blocks > INT32_MAX) return cudaErrorInvalidValue;
    *parts = step;
    const unsigned n = (unsigned)blocks;
    constexpr int MOST = kTokenValues / VEC;
    if (nv <= 1) return launch_token<T, VEC, 1, BWD>(a, n, lanes, step, s);
    if (nv <= 2 || MOST == 2) return launch_token<T, VEC, 2, BWD>(a, n, lanes, step, s);
    if constexpr (MOST >= 4) {
        if (nv <= 4 || MOST == 4) return launch_token<T, VEC, 4, BWD>(a, n, lanes, step, s);
        if constexpr (MOST >= 16) {
            if (nv <= 8) return launch_token<T, VEC, 8, BWD>(a, n, lanes, step, s);
            return launch_token<T, VEC, 16, BWD>(a, n, lanes, step, s);
        }
    }
    return cudaGetLastError();
}

template <class T, int VEC, bool BWD>
cudaError_t run_tiles(GnArgs a, int64_t* parts, cudaStream_t s) {
    const int packs = a.cg / VEC;
    gnorm_sets(a.d, VEC, &a);
    const int all = packs * a.each;
    int bx = 1;  // whole warps: a power of two, or a multiple of 32
    while (bx < 32 && bx < all) bx *= 2;
    if (all > 32) bx = all < kThreads ? (all + 31) / 32 * 32 : kThreads;
    const int by = kThreads / bx;
    const int64_t blocks = a.rows * a.tiles * a.sets, joins = (a.d.nseq * a.d.groups + 7) / 8;
    if (blocks > INT32_MAX || joins > INT32_MAX) return cudaErrorInvalidValue;
    *parts = a.walks;
    const dim3 threads((unsigned)bx, (unsigned)by);
    const unsigned n = (unsigned)blocks;
    if constexpr (BWD)
        k_gn_sums<T, VEC><<<(unsigned)(a.walks * a.sets), threads, 2 * bx * by * VEC * sizeof(float), s>>>(a);
    else
        k_gn_moments<T, VEC><<<n, threads, 0, s>>>(a);
    k_gn_join<BWD><<<(unsigned)joins, kThreads, 0, s>>>(a);
    constexpr size_t bytes = GnRing<T, VEC, BWD>::kBytes;
    if constexpr (bytes > 0) {
        static LaunchCache cache;
        LaunchGeom g;
        const cudaError_t e = cache.get(
            [](int dev, LaunchGeom* out) {
                return setup_persistent(k_gn_apply<T, VEC, BWD>, kThreads, bytes, dev, out);
            },
            &g);
        if (e != cudaSuccess) return e;
    }
    k_gn_apply<T, VEC, BWD><<<n, threads, bytes, s>>>(a);
    return cudaGetLastError();
}

template <class T, bool BWD>
cudaError_t run_gnorm(const GnArgs& a, int64_t* parts, cudaStream_t s) {
    constexpr int V = 16 / sizeof(T);
    bool vec = a.cg % V == 0;
    for (const fft_seq* q : {&a.d.x, &a.d.z, &a.out, &a.dout, &a.dz}) vec = vec && vec_rows(*q, a.d, V);
    if (by_token(a.d))
        return vec ? run_token<T, V, BWD>(a, parts, s) : run_token<T, 1, BWD>(a, parts, s);
    return vec ? run_tiles<T, V, BWD>(a, parts, s) : run_tiles<T, 1, BWD>(a, parts, s);
}

// Sequences without tokens.
__global__ void k_gn_blank(float* mean, float* rstd, int64_t n, float eps) {
    const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (i < n) mean[i] = 0.f, rstd[i] = 1.f / sqrtf(eps);
}

}  // namespace
}  // namespace gbfft

using namespace gbfft;

extern "C" int fft_gnorm_workspace(const fft_gnorm_desc* d, int backward, size_t* bytes) {
    if (!bytes || (backward != 0 && backward != 1)) return FFT_ERR_INVALID_ARG;
    TRY(check_gnorm(d, false));
    GnArgs a = {};
    *bytes = d->length < 1 ? 0 : (size_t)gnorm_layout(*d, backward, &a, nullptr);
    return FFT_OK;
}

extern "C" int fft_gnorm_forward(const fft_gnorm_desc* d, const fft_seq* out, float* mean, float* rstd,
                                 void* workspace, size_t workspace_bytes, void* stream) {
    TRY(check_gnorm(d, true));
    if (!out || !mean || !rstd) return FFT_ERR_INVALID_ARG;
    TRY(check_rows(*out, *d, true));
    if (!aligned_to(mean, 4) || !aligned_to(rstd, 4) || !aligned_to(workspace, 16)) return FFT_ERR_MISALIGNED;
    for (const fft_seq* in : {&d->x, &d->z})  // a value is read where it is written, by the same thread
        if (!seqs_same(*out, *in, d->nseq, d->length, d->offsets) &&
            seqs_meet(*out, *in, d->channels, d->channels, d->nseq, d->length, d->offsets, dtype_size(d->dtype)))
            return FFT_ERR_INVALID_ARG;
    cudaStream_t s = (cudaStream_t)stream;
    if (d->length < 1) {
        const int64_t n = d->nseq * d->groups;
        if ((n + 255) / 256 > INT32_MAX) return FFT_ERR_UNSUPPORTED_SIZE;
        k_gn_blank<<<(unsigned)((n + 255) / 256), 256, 0, s>>>(mean, rstd, n, d->eps);
        return status(cudaGetLastError());
    }
    GnArgs a = {};
    const int64_t need = gnorm_layout(*d, false, &a, static_cast<char*>(workspace));
    if (need > 0 && (!workspace || workspace_bytes < (size_t)need)) return FFT_ERR_INVALID_ARG;
    a.d = *d;
    a.out = *out;
    a.mean = mean;
    a.rstd = rstd;
    int64_t parts;
    return status(d->dtype == FFT_F32 ? run_gnorm<float, false>(a, &parts, s)
                                      : (d->dtype == FFT_BF16 ? run_gnorm<__nv_bfloat16, false>(a, &parts, s)
                                                              : run_gnorm<__half, false>(a, &parts, s)));
}

extern "C" int fft_gnorm_backward(const fft_gnorm_desc* d, const fft_gnorm_grads* g, void* workspace,
                                  size_t workspace_bytes, void* stream) {
    TRY(check_gnorm(d, true));
    if (!g || !g->mean || !g->rstd || (g->dz.data == nullptr) != (d->z.data == nullptr)) return FFT_ERR_INVALID_ARG;
    TRY(check_rows(g->dout, *d, false));
    TRY(check_rows(g->dx, *d, true));
    if (g->dz.data) TRY(check_rows(g->dz, *d, true));
    if (!aligned_to(g->mean, 4) || !aligned_to(g->rstd, 4) || !aligned_to(g->dweight, 4) || !aligned_to(g->dbias, 4) ||
        !aligned_to(workspace, 16))
        return FFT_ERR_MISALIGNED;
    for (const fft_seq* o : {&g->dx, &g->dz})
        for (const fft_seq* in : {&d->x, &d->z, &g->dout})
            if (seqs_meet(*o, *in, d->channels, d->channels, d->nseq, d->length, d->offsets, dtype_size(d->dtype)))
                return FFT_ERR_INVALID_ARG;
    cudaStream_t s = (cudaStream_t)stream;
    GnArgs a = {};
    int64_t parts = 0;
    cudaError_t e = cudaSuccess;
    if (d->length > 0) {
        const int64_t need = gnorm_layout(*d, true, &a, static_cast<char*>(workspace));
        if (!workspace || workspace_bytes < (size_t)need) return FFT_ERR_INVALID_ARG;
        a.d = *d;
        a.out = g->dx;
        a.dout = g->dout;
        a.dz = g->dz;
        a.mean = const_cast<float*>(g->mean);
        a.rstd = const_cast<float*>(g->rstd);
        if (!g->dweight && !g->dbias) a.parts = nullptr;
        e = d->dtype == FFT_F32 ? run_gnorm<float, true>(a, &parts, s)
                                : (d->dtype == FFT_BF16 ? run_gnorm<__nv_bfloat16, true>(a, &parts, s)
                                                        : run_gnorm<__half, true>(a, &parts, s));
    }
    const int64_t c = d->channels;
    if (g->dweight && g->dbias == g->dweight + c) {  // one behind the other, as in the partial rows
        if (e == cudaSuccess) e = run_sum_parts(a.parts, parts, 2 * c, 2 * c, g->dweight, 2 * c, 1, s);
        return status(e);
    }
    if (e == cudaSuccess && g->dweight) e = run_sum_parts(a.parts, parts, 2 * c, c, g->dweight, c, 1, s);
    if (e == cudaSuccess && g->dbias) e = run_sum_parts(a.parts ? a.parts + c : nullptr, parts, 2 * c, c, g->dbias, c, 1, s);
    return status(e);
}
