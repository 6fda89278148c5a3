// Group norm, channels last, with SiLU and a gate (fft_gnorm_forward, fft_gnorm_backward):
//   n = (x - mean) rstd over a sequence's tokens and a group's channels, y = n weight + bias,
//   p = y or y sigmoid(y),  out = p or p z sigmoid(z)
// and its gradients, with dy what reaches y and w = weight dy:
//   dx = rstd (w - mean(w) - n mean(w n)),  dweight = sum dy n,  dbias = sum dy.
// A few operations per element: bound by HBM.
//
// Sequences of one token (what follows the heads of an attention) are read once: the lanes that
// share a group hold its values in registers, keep their channels' weights there too and take rows
// at a stride.  Longer sequences are read twice, by blocks of a tile of tokens and whole groups: the
// first pass leaves mean and sum of squares of every tile, joined by counts (Chan, Golub and
// LeVeque's update), the second one runs through the tiles from the last one on, which the first
// has left in L2.  Its sums are taken about one of the group's own values, so that groups far from
// zero lose nothing.
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
    float* records;        // tiles' origin, sum and squares, or sums of w and w n: [record][group][3]
    float* sums;           // [sequence][group][2]: mean(w) and mean(w n)
    float* parts;          // [part][2][channels]: dweight, dbias
    int64_t rows, tile, tiles;
    int cg, each, sets;    // channels of a group; groups of a block, blocks for all groups
    int backward;
};

__device__ __forceinline__ float silu(float y) { return y * sigmoid(y); }

// A thread's channels: weight and bias in registers.
template <class T, int VEC>
struct Channel {
    float w[VEC], b[VEC];
    __device__ __forceinline__ void load(const fft_gnorm_desc& d, int64_t c, bool in) {
        const int f32 = d.param_dtype == FFT_F32;
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
            w[k] = in ? (d.weight ? ld_param<T>(d.weight, c + k, f32) : 1.f) : 0.f;
            b[k] = in && d.bias ? ld_param<T>(d.bias, c + k, f32) : 0.f;
        }
    }
};
template <class T, int VEC>
__device__ __forceinline__ Pack<T, VEC> load(const fft_seq& s, int64_t at, bool in) {
    Pack<T, VEC> p = {};
    if (in) p = ld_pack<VEC>(static_cast<const T*>(s.data) + at);
    return p;
}

// What an output is of y and the gate, and (gradients) what of g reaches y and the gate: a pack's values,
// asked once what there is.
template <class T, int VEC>
__device__ __forceinline__ void outcome(const fft_gnorm_desc& d, float (&y)[VEC], const Pack<T, VEC>& z) {
    if (d.silu) {
#pragma unroll
        for (int k = 0; k < VEC; ++k) y[k] = silu(y[k]);
    }
    if (d.z.data) {
#pragma unroll
        for (int k = 0; k < VEC; ++k) y[k] *= silu(to_f(z.v[k]));
    }
}
// y becomes what reaches it.
template <class T, int VEC>
__device__ __forceinline__ void reaches(const fft_gnorm_desc& d, float (&y)[VEC], const Pack<T, VEC>& z, const Pack<T, VEC>& g,
                                        float (&dz)[VEC]) {
    float f[VEC];
#pragma unroll
    for (int k = 0; k < VEC; ++k) f[k] = to_f(g.v[k]);
    if (d.z.data) {
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
            const float zk = to_f(z.v[k]), s = sigmoid(zk);
            dz[k] = f[k] * (s * fmaf(zk, 1.f - s, 1.f));
            f[k] *= zk * s;
        }
    }
    if (d.silu) {
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
            const float s = sigmoid(y[k]);
            dz[k] *= y[k] * s;
            y[k] = f[k] * (s * fmaf(y[k], 1.f - s, 1.f));
        }
    } else {
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
            dz[k] *= y[k];
            y[k] = f[k];
        }
    }
}
template <class T, int VEC>
__device__ __forceinline__ Pack<T, VEC> rounded(const float (&v)[VEC]) {
    Pack<T, VEC> o;
    if constexpr (VEC == 1) {
        o.v[0] = from_f<T>(v[0]);
    } else {
#pragma unroll
        for (int k = 0; k < VEC; k += 2) {
            const Pack<T, 2> p = from_f2<T>(make_float2(v[k], v[k + 1]));
            o.v[k] = p.v[0];
            o.v[k + 1] = p.v[1];
        }
    }
    return o;
}

// ---- sequences of one token -----------------------------------------------------------------

__device__ __forceinline__ float lanes_sum(float v, int lanes, unsigned mask) {
    for (int o = lanes / 2; o; o >>= 1) v += __shfl_xor_sync(mask, v, o);
    return v;
}

// `lanes` threads hold a group: NV packs of VEC values each.  They take the rows row0, row0 + step,
// ... , the next row's values under way.
template <class T, int VEC, int NV, bool BWD>
__global__ void __launch_bounds__(kThreads) k_gn_token(const GnArgs a, int lanes, int64_t step) {
    const fft_gnorm_desc& d = a.d;
    const int tid = (int)threadIdx.x, lane = tid & (lanes - 1);
    const unsigned mask = lanes == 32 ? 0xffffffffu : ((1u << lanes) - 1u) << ((tid & 31) & ~(lanes - 1));
    const int64_t sub = ((int64_t)blockIdx.x * kThreads + tid) / lanes;
    const int64_t group = sub % d.groups, row0 = sub / d.groups;
    if (row0 >= step) return;
    Channel<T, VEC> ch[NV];
    int64_t at[NV];
    bool in[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int c = (lane + j * lanes) * VEC;
        in[j] = c < a.cg;
        at[j] = group * a.cg + c;
        ch[j].load(d, at[j], in[j]);
    }
    float dw[BWD ? NV : 1][VEC] = {}, db[BWD ? NV : 1][VEC] = {};
    Pack<T, VEC> nx[NV], nz[NV], ng[BWD ? NV : 1];
    float nmean = 0.f, nrstd = 0.f;
    auto fetch = [&](int64_t row) {
        const bool live = row < a.rows;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            nx[j] = load<T, VEC>(d.x, row * d.x.seq_stride + at[j], live && in[j]);
            if (d.z.data) nz[j] = load<T, VEC>(d.z, row * d.z.seq_stride + at[j], live && in[j]);
            if (BWD) ng[j] = load<T, VEC>(a.dout, row * a.dout.seq_stride + at[j], live && in[j]);
        }
        if (BWD && live) nmean = a.mean[row * d.groups + group], nrstd = a.rstd[row * d.groups + group];
    };
    fetch(row0);
    const float inv = 1.f / (float)a.cg;
    for (int64_t row = row0; row < a.rows; row += step) {
        Pack<T, VEC> px[NV], pz[NV], pg[BWD ? NV : 1];
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            px[j] = nx[j];
            if (d.z.data) pz[j] = nz[j];
            if (BWD) pg[j] = ng[j];
        }
        float mean = nmean, rstd = nrstd;
        fetch(row + step);
        float x[NV][VEC];
        if constexpr (!BWD) {
            float sum = 0.f, sq = 0.f;
#pragma unroll
            for (int j = 0; j < NV; ++j)
#pragma unroll
                for (int k = 0; k < VEC; ++k) x[j][k] = to_f(px[j].v[k]), sum += x[j][k];
            mean = lanes_sum(sum, lanes, mask) * inv;
#pragma unroll
            for (int j = 0; j < NV; ++j)
#pragma unroll
                for (int k = 0; k < VEC; ++k) {
                    x[j][k] = in[j] ? x[j][k] - mean : 0.f;
                    sq = fmaf(x[j][k], x[j][k], sq);
                }
            rstd = rsqrtf(fmaf(lanes_sum(sq, lanes, mask), inv, d.eps));
            if (lane == 0) {
                a.mean[row * d.groups + group] = mean;
                a.rstd[row * d.groups + group] = rstd;
            }
#pragma unroll
            for (int j = 0; j < NV; ++j) {
#pragma unroll
                for (int k = 0; k < VEC; ++k) x[j][k] = fmaf(x[j][k] * rstd, ch[j].w[k], ch[j].b[k]);
                outcome<T, VEC>(d, x[j], pz[j]);
                if (in[j])
                    st_pack<VEC>(static_cast<T*>(a.out.data) + row * a.out.seq_stride + at[j], rounded<T, VEC>(x[j]));
            }
        } else {
            float w[NV][VEC], s1 = 0.f, s2 = 0.f;
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                float dz[VEC] = {};
#pragma unroll
                for (int k = 0; k < VEC; ++k) {
                    x[j][k] = (to_f(px[j].v[k]) - mean) * rstd;
                    w[j][k] = fmaf(x[j][k], ch[j].w[k], ch[j].b[k]);
                }
                reaches<T, VEC>(d, w[j], pz[j], pg[j], dz);
#pragma unroll
                for (int k = 0; k < VEC; ++k) {
                    dw[j][k] = fmaf(w[j][k], x[j][k], dw[j][k]);
                    db[j][k] += w[j][k];
                    w[j][k] = in[j] ? w[j][k] * ch[j].w[k] : 0.f;
                    s1 += w[j][k];
                    s2 = fmaf(w[j][k], x[j][k], s2);
                }
                if (in[j] && d.z.data)
                    st_pack<VEC>(static_cast<T*>(a.dz.data) + row * a.dz.seq_stride + at[j], rounded<T, VEC>(dz));
            }
            s1 = lanes_sum(s1, lanes, mask) * inv;
            s2 = lanes_sum(s2, lanes, mask) * inv;
#pragma unroll
            for (int j = 0; j < NV; ++j) {
#pragma unroll
                for (int k = 0; k < VEC; ++k) w[j][k] = (w[j][k] - fmaf(x[j][k], s2, s1)) * rstd;
                if (in[j])
                    st_pack<VEC>(static_cast<T*>(a.out.data) + row * a.out.seq_stride + at[j], rounded<T, VEC>(w[j]));
            }
        }
    }
    if constexpr (BWD) {
        if (!a.parts) return;
        float* p = a.parts + row0 * 2 * d.channels;
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int k = 0; k < VEC; ++k)
                if (in[j]) p[at[j] + k] = dw[j][k], p[d.channels + at[j] + k] = db[j][k];
    }
}

// ---- longer sequences -----------------------------------------------------------------------

// The block's part of the grid: a tile of tokens, a set of whole groups.  Thread (tx, ty) takes the
// packs tx, tx + blockDim.x, ... of the set's channels and every blockDim.y-th token.
struct TileAt {
    int64_t row, tile, t0, t1;
    int group0, groups;
};
__device__ __forceinline__ TileAt tile_at(const GnArgs& a, bool last_first) {
    int64_t b = last_first ? (int64_t)gridDim.x - 1 - blockIdx.x : blockIdx.x;
    TileAt t;
    t.group0 = (int)(b % a.sets) * a.each;
    b /= a.sets;
    t.tile = b % a.tiles;
    t.row = b / a.tiles;
    t.t0 = t.tile * a.tile;
    t.t1 = t.t0 + a.tile < a.d.length ? t.t0 + a.tile : a.d.length;
    t.groups = (int)a.d.groups - t.group0 < a.each ? (int)a.d.groups - t.group0 : a.each;
    return t;
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

template <class T, int VEC>
__global__ void __launch_bounds__(kThreads) k_gn_moments(const GnArgs a) {
    __shared__ float red[2][kThreads];
    const fft_gnorm_desc& d = a.d;
    const TileAt t = tile_at(a, false);
    const int tx = (int)threadIdx.x, ty = (int)threadIdx.y, bx = (int)blockDim.x, by = (int)blockDim.y;
    const int packs = a.cg / VEC, all = packs * t.groups;
    const T* base = static_cast<const T*>(d.x.data) + t.row * d.x.seq_stride + (int64_t)t.group0 * a.cg;
    for (int64_t at = t.t0; at < t.t1;) {
        const SeqAt s = part_at(a, t.row, at, t.t1);
        float s1 = 0.f, s2 = 0.f;
        for (int p = tx; p < all; p += bx) {
            const T* x = base + p * VEC;
            const float shift = to_f(base[s.begin * d.x.tok_stride + p / packs * a.cg]);
            float v1[VEC] = {}, v2[VEC] = {};
#pragma unroll 8
            for (int64_t i = s.begin + ty; i < s.end; i += by) {
                const Pack<T, VEC> v = ld_pack<VEC>(x + i * d.x.tok_stride);
#pragma unroll
                for (int k = 0; k < VEC; ++k) {
                    const float e = to_f(v.v[k]) - shift;
                    v1[k] += e;
                    v2[k] = fmaf(e, e, v2[k]);
                }
            }
#pragma unroll
            for (int k = 0; k < VEC; ++k) s1 += v1[k], s2 += v2[k];
        }
        red[0][ty * bx + tx] = s1, red[1][ty * bx + tx] = s2;
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
                r[0] = to_f(base[s.begin * d.x.tok_stride + g * a.cg]);  // what the sums are counted from
                r[1] = v1;
                r[2] = v2;
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
    double n = 0.0, mean = 0.0, m2 = 0.0;
    if (end > begin) {
        const int64_t first = begin / a.tile, last = (end - 1) / a.tile;
        for (int64_t k = first + lane; k <= last; k += 32) {
            const float* r = a.records + (record_of(a, q, k, q) * d.groups + g) * 3;
            if constexpr (BWD) {
                mean += r[0];
                m2 += r[1];
            } else {
                const int64_t lo = k * a.tile > begin ? k * a.tile : begin,
                              hi = (k + 1) * a.tile < end ? (k + 1) * a.tile : end;
                const double c = (double)(hi - lo) * a.cg, all = n + c, own = (double)r[1] / c,
                             delta = (double)r[0] + own - mean;
                mean += delta * (c / all);
                m2 += ((double)r[2] - own * (double)r[1]) + delta * delta * (n * c / all);
                n = all;
            }
        }
    }
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const double bn = __shfl_xor_sync(0xffffffffu, n, o), bm = __shfl_xor_sync(0xffffffffu, mean, o),
                     b2 = __shfl_xor_sync(0xffffffffu, m2, o);
        if constexpr (BWD) {
            mean += bm;
            m2 += b2;
        } else {
            const double all = n + bn, delta = bm - mean;
            if (all > 0.0) {
                m2 += b2 + delta * delta * (n * bn / all);
                mean += delta * (bn / all);
            }
            n = all;
        }
    }
    if (lane) return;
    const double count = end > begin ? (double)(end - begin) * a.cg : 1.0;
    if constexpr (BWD) {
        a.sums[i * 2] = (float)(mean / count);
        a.sums[i * 2 + 1] = (float)(m2 / count);
    } else {
        a.mean[i] = (float)mean;
        a.rstd[i] = (float)(1.0 / sqrt((m2 < 0.0 ? 0.0 : m2) / count + (double)d.eps));
    }
}

// Second pass: outputs, or (backward) gradients of x and z.
template <class T, int VEC, bool BWD>
__global__ void __launch_bounds__(kThreads) k_gn_apply(const GnArgs a) {
    const fft_gnorm_desc& d = a.d;
    const TileAt t = tile_at(a, true);
    const int tx = (int)threadIdx.x, ty = (int)threadIdx.y, bx = (int)blockDim.x, by = (int)blockDim.y;
    const int packs = a.cg / VEC, all = packs * t.groups;
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
            // the rows of four tokens before the first of them is stored (out may be x or z)
            constexpr int DEEP = 4;
            for (int64_t i0 = s.begin + ty; i0 < s.end; i0 += DEEP * by) {
                Pack<T, VEC> px[DEEP], pz[DEEP], pg[DEEP];
#pragma unroll
                for (int u = 0; u < DEEP; ++u) {
                    const int64_t i = i0 + u * by;
                    const bool in = i < s.end;
                    px[u] = pz[u] = pg[u] = Pack<T, VEC>{};
                    if (in) px[u] = ld_pack<VEC>(x + i * d.x.tok_stride);
                    if (in && d.z.data) pz[u] = ld_pack<VEC>(z + i * d.z.tok_stride);
                    if (BWD && in) pg[u] = ld_pack<VEC>(go + i * a.dout.tok_stride);
                }
#pragma unroll
                for (int u = 0; u < DEEP; ++u) {
                    const int64_t i = i0 + u * by;
                    if (i >= s.end) break;
                    float n[VEC], y[VEC], dzv[VEC] = {};
#pragma unroll
                    for (int k = 0; k < VEC; ++k) {
                        n[k] = (to_f(px[u].v[k]) - mean) * rstd;
                        y[k] = fmaf(n[k], ch.w[k], ch.b[k]);
                    }
                    if constexpr (BWD) {
                        reaches<T, VEC>(d, y, pz[u], pg[u], dzv);
#pragma unroll
                        for (int k = 0; k < VEC; ++k) y[k] = (y[k] * ch.w[k] - fmaf(n[k], s2, s1)) * rstd;
                    } else {
                        outcome<T, VEC>(d, y, pz[u]);
                    }
                    st_pack<VEC>(out + i * a.out.tok_stride, rounded<T, VEC>(y));
                    if (BWD && d.z.data) st_pack<VEC>(dz + i * a.dz.tok_stride, rounded<T, VEC>(dzv));
                }
            }
        }
        at = s.end;
    }
}

// First pass of the gradients: sums of w and w n of every part, of dy n and dy of every channel.
template <class T, int VEC>
__global__ void __launch_bounds__(kThreads) k_gn_sums(const GnArgs a) {
    __shared__ float red[2][kThreads];
    extern __shared__ float chans[];  // [2][ty][tx * VEC]
    const fft_gnorm_desc& d = a.d;
    const TileAt t = tile_at(a, false);
    const int tx = (int)threadIdx.x, ty = (int)threadIdx.y, bx = (int)blockDim.x, by = (int)blockDim.y;
    const int packs = a.cg / VEC, all = packs * t.groups, tid = ty * bx + tx;
    // packs outermost, since a channel's sums run over all parts; with several rounds of packs (a
    // set of one group of many channels) the parts' sums go on from what is there
    for (int p0 = 0; p0 < all; p0 += bx) {
        const int p = p0 + tx;
        const bool in = p < all;
        const int64_t c = (int64_t)t.group0 * a.cg + p * VEC;
        Channel<T, VEC> ch;
        ch.load(d, c, in);
        float dw[VEC] = {}, db[VEC] = {};
        for (int64_t at = t.t0; at < t.t1;) {
            const SeqAt s = part_at(a, t.row, at, t.t1);
            float s1 = 0.f, s2 = 0.f;
            if (in) {
                const int64_t g = t.group0 + p / packs;
                const float mean = a.mean[s.q * d.groups + g], rstd = a.rstd[s.q * d.groups + g];
                const T* x = static_cast<const T*>(d.x.data) + t.row * d.x.seq_stride + c;
                const T* z = static_cast<const T*>(d.z.data) + t.row * d.z.seq_stride + c;
                const T* go = static_cast<const T*>(a.dout.data) + t.row * a.dout.seq_stride + c;
#pragma unroll 4
                for (int64_t i = s.begin + ty; i < s.end; i += by) {
                    const Pack<T, VEC> px = ld_pack<VEC>(x + i * d.x.tok_stride);
                    Pack<T, VEC> pz = {};
                    if (d.z.data) pz = ld_pack<VEC>(z + i * d.z.tok_stride);
                    const Pack<T, VEC> pg = ld_pack<VEC>(go + i * a.dout.tok_stride);
                    float n[VEC], y[VEC], dzv[VEC] = {};
#pragma unroll
                    for (int k = 0; k < VEC; ++k) {
                        n[k] = (to_f(px.v[k]) - mean) * rstd;
                        y[k] = fmaf(n[k], ch.w[k], ch.b[k]);
                    }
                    reaches<T, VEC>(d, y, pz, pg, dzv);
#pragma unroll
                    for (int k = 0; k < VEC; ++k) {
                        const float dn = y[k] * n[k];
                        dw[k] += dn;
                        db[k] += y[k];
                        s1 = fmaf(y[k], ch.w[k], s1);
                        s2 = fmaf(dn, ch.w[k], s2);
                    }
                }
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
        if (!a.parts) continue;
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
            chans[tid * VEC + k] = dw[k];
            chans[(bx * by + tid) * VEC + k] = db[k];
        }
        __syncthreads();
        float* out = a.parts + (t.row * a.tiles + t.tile) * 2 * d.channels + (int64_t)t.group0 * a.cg + (int64_t)p0 * VEC;
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
// Lanes that share a group of the token kernel: a pack each, up to a warp.
int token_lanes(int64_t packs) {
    int lanes = 1;
    while (lanes < 32 && lanes < packs) lanes *= 2;
    return lanes;
}
// Rows that the token kernel's threads start at: as many as the SMs hold, at three blocks each where
// every start leaves a row of partial sums.
int64_t token_step(const fft_gnorm_desc& d, int lanes, bool backward) {
    const int64_t subs = (int64_t)num_sms() * (backward ? 3 : 6) * (kThreads / lanes);
    const int64_t step = subs / d.groups;
    return step < 1 ? 1 : (step > d.nseq ? d.nseq : step);
}
// Tokens of a tile: as many as leave every SM four blocks, 16 to 128.
int64_t tile_of(const fft_gnorm_desc& d) {
    const int64_t rows = d.offsets ? 1 : d.nseq;
    int64_t tile = 128;
    while (tile > 16 && rows * ((d.length + tile - 1) / tile) * ((d.channels + 2047) / 2048) < (int64_t)num_sms() * 4) tile /= 2;
    return tile;
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
        if (backward) a->parts = take(token_step(d, token_lanes((a->cg + vec - 1) / vec), true) * 2 * d.channels);
        return at;
    }
    a->tile = tile_of(d);
    a->tiles = (d.length + a->tile - 1) / a->tile;
    a->records = take((a->rows * a->tiles + (d.offsets ? d.nseq : 0)) * d.groups * 3);
    if (backward) {
        a->sums = take(d.nseq * d.groups * 2);
        a->parts = take(a->rows * a->tiles * 2 * d.channels);
    }
    return at;
}

bool vec_rows(const fft_seq& s, const fft_gnorm_desc& d, int64_t vec) {
    return !s.data || (aligned_to(s.data, 16) && (d.length < 2 || s.tok_stride % vec == 0) &&
                       (d.offsets || d.nseq < 2 || s.seq_stride % vec == 0));
}

template <class T, int VEC, bool BWD>
cudaError_t run_token(const GnArgs& a, int64_t* parts, cudaStream_t s) {
    const int packs = a.cg / VEC, lanes = token_lanes(packs);
    const int nv = (packs + lanes - 1) / lanes;
    const int64_t step = token_step(a.d, lanes, BWD);
    const int64_t blocks = (step * a.d.groups * lanes + kThreads - 1) / kThreads;
    if (blocks > INT32_MAX) return cudaErrorInvalidValue;
    *parts = step;
    const unsigned n = (unsigned)blocks;
    constexpr int MOST = kTokenValues / VEC;
    if (nv <= 1) k_gn_token<T, VEC, 1, BWD><<<n, kThreads, 0, s>>>(a, lanes, step);
    else if (nv <= 2 || MOST == 2) k_gn_token<T, VEC, 2, BWD><<<n, kThreads, 0, s>>>(a, lanes, step);
    else if constexpr (MOST >= 4) {
        if (nv <= 4 || MOST == 4) k_gn_token<T, VEC, 4, BWD><<<n, kThreads, 0, s>>>(a, lanes, step);
        else if constexpr (MOST >= 16) {
            if (nv <= 8) k_gn_token<T, VEC, 8, BWD><<<n, kThreads, 0, s>>>(a, lanes, step);
            else k_gn_token<T, VEC, 16, BWD><<<n, kThreads, 0, s>>>(a, lanes, step);
        }
    }
    return cudaGetLastError();
}

template <class T, int VEC, bool BWD>
cudaError_t run_tiles(GnArgs a, int64_t* parts, cudaStream_t s) {
    const int packs = a.cg / VEC;
    a.each = packs >= kThreads ? 1 : kThreads / packs;
    if (a.each > a.d.groups) a.each = (int)a.d.groups;
    a.sets = (int)((a.d.groups + a.each - 1) / a.each);
    a.each = (int)((a.d.groups + a.sets - 1) / a.sets);  // of like size
    const int all = packs * a.each;
    int bx = 1;  // whole warps: a power of two, or a multiple of 32
    while (bx < 32 && bx < all) bx *= 2;
    if (all > 32) bx = all < kThreads ? (all + 31) / 32 * 32 : kThreads;
    const int by = kThreads / bx;
    const int64_t blocks = a.rows * a.tiles * a.sets, joins = (a.d.nseq * a.d.groups + 7) / 8;
    if (blocks > INT32_MAX || joins > INT32_MAX) return cudaErrorInvalidValue;
    *parts = a.rows * a.tiles;
    const dim3 threads((unsigned)bx, (unsigned)by);
    const unsigned n = (unsigned)blocks;
    if constexpr (BWD)
        k_gn_sums<T, VEC><<<n, threads, 2 * bx * by * VEC * sizeof(float), s>>>(a);
    else
        k_gn_moments<T, VEC><<<n, threads, 0, s>>>(a);
    k_gn_join<BWD><<<(unsigned)joins, kThreads, 0, s>>>(a);
    k_gn_apply<T, VEC, BWD><<<n, threads, 0, s>>>(a);
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
        a.backward = 1;
        if (!g->dweight && !g->dbias) a.parts = nullptr;
        e = d->dtype == FFT_F32 ? run_gnorm<float, true>(a, &parts, s)
                                : (d->dtype == FFT_BF16 ? run_gnorm<__nv_bfloat16, true>(a, &parts, s)
                                                        : run_gnorm<__half, true>(a, &parts, s));
    }
    const int64_t c = d->channels;
    if (e == cudaSuccess && g->dweight) e = run_sum_parts(a.parts, parts, 2 * c, c, g->dweight, c, 1, s);
    if (e == cudaSuccess && g->dbias) e = run_sum_parts(a.parts ? a.parts + c : nullptr, parts, 2 * c, c, g->dbias, c, 1, s);
    return status(e);
}
