// C entry points of linear attention: checks on the host, cuts of time, workspace layout, and the
// kernels around k_linattn (gradients of the decay and of shared heads, states of sequences without
// tokens, single tokens).  Declared in include/gbfft.h.
#include <atomic>
#include <mutex>

#include "linattn.h"
#include "seq_overlap.h"
#include "tma.cuh"

namespace gbfft {
namespace {

// ---- single tokens --------------------------------------------------------------------------

constexpr int kStepThreads = 128, kStepCols = 32;

struct AttnStepArgs {
    fft_linattn_desc d;
    fft_heads out;
    float* state;
    const int64_t* slots;
    const int64_t* slots_out;
    int64_t pool;
    int ctiles;
};

// exp(g) of a decay, g at most 0 (a NaN stays), to within 1.6 units of 2^-24 of itself and without a
// lean: the approximate exponential lies 0.3 units low on average, which a state that is kept for a thousand
// tokens collects a thousand times.  g log2(e) in two floats is a whole number n and f in [-1/2, 1/2]; 2^f is
// the Taylor series of exp(f ln 2), whose 1 is added last, and 2^n comes in two factors, since n may be below
// -126.
__device__ __forceinline__ float step_decay(float g) {
    const Two d = log2_decay(g < -104.f ? -104.f : g);  // exp(-104) is below half of the smallest number
    const float n = rintf(d.hi), t = ((d.hi - n) + d.lo) * kLn2;
    float p = 1.f / 5040.f;
    p = fmaf(p, t, 1.f / 720.f);
    p = fmaf(p, t, 1.f / 120.f);
    p = fmaf(p, t, 1.f / 24.f);
    p = fmaf(p, t, 1.f / 6.f);
    p = fmaf(p, t, 0.5f);
    const float v = 1.f + fmaf(t * t, p, t);
    const int whole = (int)n, half = whole / 2;  // (0 of a NaN)
    return v * __int_as_float((127 + half) << 23) * __int_as_float((127 + whole - half) << 23);
}

// A block takes 32 columns of one head's state: VEC columns per thread, so 32 / VEC lanes hold a row
// and the rows are dealt to groups of lanes, eight loads of each under way at once.  Bound by the
// states' bytes for many sequences and by latency for one; queries and keys go through shared memory,
// which leaves registers for eight blocks to an SM.  Measured: 128 sequences of 16 heads of 128 x 128 47 us,
// 5.7 TB/s (84% of the copy rate; 81 us with queries and keys in registers, four blocks); one sequence of 32
// heads of 64 x 64 15 to 17 us with the host side of the call, the kernel 6 us of it (cold, profiled).
template <class T, int VEC>
__global__ void __launch_bounds__(kStepThreads, 8) k_linattn_step(const AttnStepArgs a) {
    constexpr int LANES = kStepCols / VEC, GROUPS = kStepThreads / LANES, DEEP = 8;
    __shared__ float red[GROUPS][kStepCols + 1], qk[2][kAttnMaxDim];
    const int lane = (int)threadIdx.x % LANES, group = (int)threadIdx.x / LANES;
    unsigned b = blockIdx.x;
    const int ct = (int)(b % (unsigned)a.ctiles);
    b /= (unsigned)a.ctiles;
    const int64_t h = b % (unsigned)a.d.heads, q = b / (unsigned)a.d.heads, g = h / (a.d.heads / a.d.groups);
    const int dk = (int)a.d.dk, dv = (int)a.d.dv, c = ct * kStepCols + lane * VEC;
    const bool in = c < dv;
    const int64_t from = a.slots ? a.slots[q] : q, to = a.slots_out ? a.slots_out[q] : from;
    const bool live = from >= 0 && from < a.pool && to >= 0 && to < a.pool;
    const T* qp = static_cast<const T*>(a.d.q.data) + q * a.d.q.seq_stride + g * a.d.q.head_stride;
    const T* kp = static_cast<const T*>(a.d.k.data) + q * a.d.k.seq_stride + g * a.d.k.head_stride;
    const T* vp = static_cast<const T*>(a.d.v.data) + q * a.d.v.seq_stride + h * a.d.v.head_stride + c;
    const float gl = to_f(static_cast<const T*>(a.d.decay.data)[q * a.d.decay.seq_stride + h]);
    const int64_t per = (int64_t)dk * dv;
    const float* src = a.state + (live ? (from * a.d.heads + h) * per + c : 0);
    float* dst = a.state + (live ? (to * a.d.heads + h) * per + c : 0);
    Pack<float, VEC> s[DEEP];
    auto fetch = [&](int r0) {
#pragma unroll
        for (int i = 0; i < DEEP; ++i)
            if (live && in && r0 + i * GROUPS < dk) s[i] = ld_pack<VEC>(src + (r0 + i * GROUPS) * dv);
    };
    fetch(group);
    for (int i = (int)threadIdx.x; i < dk; i += kStepThreads) qk[0][i] = to_f(qp[i]), qk[1][i] = to_f(kp[i]);
    float v[VEC], y[VEC] = {};
#pragma unroll
    for (int k = 0; k < VEC; ++k) v[k] = in ? to_f(vp[k]) : 0.f;
    const float e = step_decay(gl);
    __syncthreads();
    for (int r0 = group; r0 < dk; r0 += GROUPS * DEEP) {
        if (r0 != group) fetch(r0);
#pragma unroll
        for (int i = 0; i < DEEP; ++i) {
            const int r = r0 + i * GROUPS;
            if (live && in && r < dk) {
#pragma unroll
                for (int k = 0; k < VEC; ++k) {
                    s[i].v[k] = fmaf(e, s[i].v[k], qk[1][r] * v[k]);
                    y[k] = fmaf(qk[0][r], s[i].v[k], y[k]);
                }
                st_pack<VEC>(dst + r * dv, s[i]);
            }
        }
    }
#pragma unroll
    for (int k = 0; k < VEC; ++k) red[group][lane * VEC + k] = y[k];
    __syncthreads();
    const int t = (int)threadIdx.x;
    if (t < kStepCols && ct * kStepCols + t < dv) {
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < GROUPS; ++i) sum += red[i][t];
        static_cast<T*>(a.out.data)[q * a.out.seq_stride + h * a.out.head_stride + ct * kStepCols + t] =
            from_f<T>(live ? sum * a.d.scale : 0.f);
    }
}

template <class T>
cudaError_t attn_step(AttnStepArgs a, cudaStream_t s) {
    a.ctiles = (int)((a.d.dv + kStepCols - 1) / kStepCols);
    const int64_t blocks = a.d.nseq * a.d.heads * a.ctiles;
    if (blocks > INT32_MAX) return cudaErrorInvalidValue;
    if (a.d.dv % 4 == 0 && aligned_to(a.state, 16))
        k_linattn_step<T, 4><<<(unsigned)blocks, kStepThreads, 0, s>>>(a);
    else
        k_linattn_step<T, 1><<<(unsigned)blocks, kStepThreads, 0, s>>>(a);
    return cudaGetLastError();
}

// ---- around the kernel of whole sequences ---------------------------------------------------

// Turns what every segment adds into the state that it begins with: one thread for four values.
__global__ void k_linattn_carry(const AttnArgs a, int64_t quads) {
    const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (i >= quads) return;
    const int64_t head = blockIdx.y, row = blockIdx.z;
    float4* p = reinterpret_cast<float4*>(a.carry) + ((row * a.nsegments * a.heads) + head) * quads + i;
    const int64_t step = a.heads * quads;
    const float* gone = a.carry_decay + row * a.nsegments * a.heads + head;
    const int* reset = a.carry_reset + row * a.nsegments * a.heads + head;
    float4 c = make_float4(0.f, 0.f, 0.f, 0.f);
    constexpr int DEEP = 8;  // segments loaded before the first of them is stored
    for (int64_t k0 = 0; k0 < a.nsegments; k0 += DEEP) {
        float4 own[DEEP];
        float f[DEEP];
        bool r[DEEP];
#pragma unroll
        for (int u = 0; u < DEEP; ++u) {
            if (k0 + u >= a.nsegments) break;
            const int64_t s = a.reverse ? a.nsegments - 1 - k0 - u : k0 + u;
            own[u] = p[s * step];
            r[u] = reset[s * a.heads];
            f[u] = ex2(gone[s * a.heads]);
        }
#pragma unroll
        for (int u = 0; u < DEEP; ++u) {
            if (k0 + u >= a.nsegments) break;
            const int64_t s = a.reverse ? a.nsegments - 1 - k0 - u : k0 + u;
            p[s * step] = c;
            c.x = r[u] ? own[u].x : fmaf(f[u], c.x, own[u].x);
            c.y = r[u] ? own[u].y : fmaf(f[u], c.y, own[u].y);
            c.z = r[u] ? own[u].z : fmaf(f[u], c.z, own[u].z);
            c.w = r[u] ? own[u].w : fmaf(f[u], c.w, own[u].w);
        }
    }
}

// States of sequences without tokens: what they begin with.
__global__ void k_linattn_empty(const int64_t* offsets, const float* from, float* to, int64_t per) {
    const int64_t q = blockIdx.x;
    if (offsets[q + 1] > offsets[q]) return;
    for (int64_t i = threadIdx.x; i < per; i += blockDim.x) to[q * per + i] = from ? from[q * per + i] : 0.f;
}

// Sums over the heads that share queries or keys.
template <class T>
__global__ void k_linattn_shared(const float* parts, fft_heads out, int64_t length, int64_t groups, int64_t share,
                                 int64_t dim, int64_t total) {
    const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (i >= total) return;
    const int64_t d = i % dim, g = i / dim % groups, t = i / (dim * groups);
    const float* p = parts + (t * groups * share + g * share) * dim + d;
    float v = 0.f;
    for (int64_t h = 0; h < share; ++h) v += p[h * dim];
    static_cast<T*>(out.data)[t / length * out.seq_stride + t % length * out.tok_stride + g * out.head_stride + d] =
        from_f<T>(v);
}

struct DecayGradArgs {
    fft_seq decay, ddecay;
    const int64_t* offsets;
    int64_t nseq, length, rows, heads, segment, nsegments;
    int64_t ztiles, final_tiles;  // that the sums of rows, of states, come in
    int initial;  // sequences have initial states
    // [ztile][head][row * length + t]: of the rows of dq and dk, between chunks and altogether
    const float* q_inter;
    const float* q_all;
    const float* k_inter;
    const float* k_all;
    const float* final_dots;  // [ztile][sequence][head], or null
    double* carry;            // [row][segment][head]
    int* stops;
};

__device__ __forceinline__ float tiles_sum(const float* p, int64_t tiles, int64_t step) {
    float v = 0.f;
    for (int64_t z = 0; z < tiles; ++z) v += p[z * step];
    return v;
}

// Pairs (j, i) of tokens j < t <= i weigh w[j,i] = scale decay(j, i) (q[i] k[j]) (dout[i] v[j]), and
// the gradient of decay t is the sum of them all (initial and final states count as tokens before and
// behind the sequence).  With X the sum over the pairs that cross a chunk's first token,
//   dg[t] = X - sum_{i < t} qi[i] + sum_{j < t} ki[j] + sum_{i >= t} (qa[i] - ka[i])
// over the chunk's tokens, where qi and ki are those rows' pairs with tokens of other chunks and qa,
// ka those within the chunk; X in turn is that of the next chunk and what the rows between change.
// Only between chunks do such sums run on, over terms that were formed from states in two or three
// pieces, so that what cancels within a chunk is not carried along.  (Terms that are not finite cancel
// nothing: they may reach any token of their sequence and head, and none of another one.)
// One block per segment and head; a warp takes every eighth chunk.
constexpr int kDgWarps = 8, kDgBatch = 64;

// What the tokens of a segment's first sequence change (X at the segment's start less that at its
// end), and whether that sequence ends there.
__global__ void __launch_bounds__(kDgWarps * 32) k_decay_sums(const DecayGradArgs a) {
    __shared__ double red[kDgWarps];
    const int64_t head = blockIdx.x % a.heads, seg = blockIdx.x / a.heads % a.nsegments,
                  row = blockIdx.x / (a.heads * a.nsegments);
    const int64_t t0 = seg * a.segment, t1 = t0 + a.segment < a.length ? t0 + a.segment : a.length;
    const SeqAt s = seq_at(a.offsets, a.nseq, a.length, row, t0);
    const int64_t end = s.end > t1 || s.end <= t0 ? t1 : s.end;
    const int64_t step = a.heads * a.rows * a.length, at = (head * a.rows + row) * a.length;
    double v = 0.0;
    for (int64_t t = t0 + threadIdx.x; t < end; t += kDgWarps * 32)
        v += (double)tiles_sum(a.q_inter + at + t, a.ztiles, step) - (double)tiles_sum(a.k_inter + at + t, a.ztiles, step);
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x / 32] = v;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < kDgWarps; ++w) v += red[w];
        a.carry[blockIdx.x] = v;
        a.stops[blockIdx.x] = s.end <= t1;
    }
}

// PER: tokens of a chunk per lane.
template <class T, int PER>
__global__ void __launch_bounds__(kDgWarps * 32) k_decay_grads(const DecayGradArgs a) {
    constexpr int C = 32 * PER;
    __shared__ double change[kDgBatch], cross[kDgBatch];
    const int64_t head = blockIdx.x % a.heads, seg = blockIdx.x / a.heads % a.nsegments,
                  row = blockIdx.x / (a.heads * a.nsegments);
    const int64_t t0 = seg * a.segment, t1 = t0 + a.segment < a.length ? t0 + a.segment : a.length;
    const int64_t step = a.heads * a.rows * a.length, at = (head * a.rows + row) * a.length;
    const int lane = (int)threadIdx.x & 31, warp = (int)threadIdx.x >> 5;
    auto sums = [&](const float* p, int64_t t, int64_t end, float (&v)[PER]) {
#pragma unroll
        for (int k = 0; k < PER; ++k) v[k] = t + k < end ? tiles_sum(p + at + t + k, a.ztiles, step) : 0.f;
    };
    for (int64_t stop = t1; stop > t0;) {
        const SeqAt s = seq_at(a.offsets, a.nseq, a.length, row, stop - 1);
        const int64_t begin = s.begin > stop - 1 ? stop - 1 : (s.begin < t0 ? t0 : s.begin), end = stop;
        double X = 0.0;  // at `end`
        if (!(s.end <= end || end == a.length)) {
            for (int64_t k = seg + 1; k < a.nsegments; ++k) {
                const int64_t i = (row * a.nsegments + k) * a.heads + head;
                X += a.carry[i];
                if (a.stops[i]) break;
            }
        }
        if (a.final_dots)
            for (int64_t z = 0; z < a.final_tiles; ++z) X += a.final_dots[(z * a.nseq + s.q) * a.heads + head];
        const int64_t chunks = (end - begin + C - 1) / C;
        for (int64_t c1 = chunks; c1 > 0; c1 -= kDgBatch) {
            const int64_t c0 = c1 > kDgBatch ? c1 - kDgBatch : 0;
            for (int64_t c = c0 + warp; c < c1; c += kDgWarps) {
                const int64_t t = begin + c * C + PER * lane;
                float qi[PER], ki[PER];
                sums(a.q_inter, t, end, qi);
                sums(a.k_inter, t, end, ki);
                double v = 0.0;
#pragma unroll
                for (int k = 0; k < PER; ++k) v += (double)qi[k] - ki[k];
#pragma unroll
                for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
                if (lane == 0) change[c - c0] = v;
            }
            __syncthreads();
            if (threadIdx.x == 0)
                for (int64_t c = c1 - 1; c >= c0; --c) cross[c - c0] = X += change[c - c0];
            __syncthreads();
            X = cross[0];
            // nothing crosses a sequence's first token but its initial state
            const bool zero = c0 == 0 && !a.initial && (begin == 0 || s.begin == begin);
            for (int64_t c = c0 + warp; c < c1; c += kDgWarps) {
                const int64_t t = begin + c * C + PER * lane;
                float qi[PER], ki[PER], w[PER], ka[PER];
                sums(a.q_inter, t, end, qi);
                sums(a.k_inter, t, end, ki);
                sums(a.q_all, t, end, w);
                sums(a.k_all, t, end, ka);
                // between chunks: what tokens before t have, from the left; within the chunk, from the right
                float left = 0.f, right = 0.f;
#pragma unroll
                for (int k = 0; k < PER; ++k) {
                    w[k] = (w[k] - qi[k]) - (ka[k] - ki[k]);
                    ki[k] -= qi[k];
                    left += ki[k];
                    right += w[k];
                }
#pragma unroll
                for (int o = 1; o < 32; o *= 2) {
                    const float l = __shfl_up_sync(0xffffffffu, left, o), r = __shfl_down_sync(0xffffffffu, right, o);
                    if (lane >= o) left += l;
                    if (lane + o < 32) right += r;
                }
                left = __shfl_up_sync(0xffffffffu, left, 1);
                right = __shfl_down_sync(0xffffffffu, right, 1);
                if (lane == 0) left = 0.f;
                if (lane == 31) right = 0.f;
                float tail[PER];
#pragma unroll
                for (int k = PER - 1; k >= 0; --k) tail[k] = right += w[k];
                const float base = zero && c == 0 ? 0.f : (float)cross[c - c0];
#pragma unroll
                for (int k = 0; k < PER; ++k) {
                    const float dg = base + left + tail[k];
                    left += ki[k];
                    if (t + k >= end) continue;
                    const float g = to_f(static_cast<const T*>(a.decay.data)[row * a.decay.seq_stride +
                                                                           (t + k) * a.decay.tok_stride + head]);
                    // above 0 the decay is 0 whatever its value, below -104 its exponential is
                    static_cast<T*>(a.ddecay.data)[row * a.ddecay.seq_stride + (t + k) * a.ddecay.tok_stride + head] =
                        from_f<T>(g > 0.f || g < -104.f ? 0.f : dg);
                }
            }
            __syncthreads();
        }
        stop = begin;
    }
}

}  // namespace

cudaError_t attn_carry_pass(const AttnArgs& a, int64_t quads, cudaStream_t s) {
    if (a.heads > 65535) return cudaErrorInvalidValue;
    for (int64_t r = 0; r < a.rows; r += 65535) {
        AttnArgs c = a;
        const int64_t n = a.rows - r < 65535 ? a.rows - r : 65535;
        c.carry += r * a.nsegments * a.heads * quads * 4;
        c.carry_decay += r * a.nsegments * a.heads;
        c.carry_reset += r * a.nsegments * a.heads;
        k_linattn_carry<<<dim3((unsigned)((quads + 127) / 128), (unsigned)a.heads, (unsigned)n), 128, 0, s>>>(c, quads);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

namespace {

// ---- checks and plans -----------------------------------------------------------------------

constexpr int64_t kMaxElements = INT64_C(1) << 58, kMaxTokStride = INT64_C(1) << 26;

int status(cudaError_t e) {
    return e == cudaSuccess ? FFT_OK : (e == cudaErrorInvalidValue ? FFT_ERR_UNSUPPORTED_SIZE : FFT_ERR_CUDA);
}

#define TRY(x)                         \
    do {                               \
        const int rc_ = (x);           \
        if (rc_ != FFT_OK) return rc_; \
    } while (0)

// Rows of an output must lie apart: from the axis of the smallest stride on, each stride is beyond
// what the axes before it take.
bool rows_apart(const fft_heads& t, int64_t dim, int64_t heads, int64_t nseq, int64_t length) {
    int64_t stride[3] = {t.head_stride, t.tok_stride, t.seq_stride}, count[3] = {heads, length, nseq};
    for (int i = 0; i < 2; ++i)
        for (int j = 0; j < 2 - i; ++j)
            if (stride[j] > stride[j + 1]) {
                int64_t v = stride[j];
                stride[j] = stride[j + 1], stride[j + 1] = v;
                v = count[j], count[j] = count[j + 1], count[j + 1] = v;
            }
    int64_t span = dim;
    for (int i = 0; i < 3; ++i) {
        if (count[i] < 2) continue;
        if (stride[i] < span) return false;
        span += (count[i] - 1) * stride[i];
    }
    return true;
}

int check_heads(const fft_heads& t, int64_t dim, int64_t heads, const fft_linattn_desc& d, bool output) {
    if (!t.data) return d.length == 0 ? FFT_OK : FFT_ERR_INVALID_ARG;
    if (t.tok_stride < 0 || t.seq_stride < 0 || t.head_stride < 0) return FFT_ERR_INVALID_ARG;
    if (t.tok_stride > kMaxTokStride || t.head_stride > kMaxElements / (heads + 1) ||
        (!d.offsets && t.seq_stride > kMaxElements / (d.nseq + 1)))
        return FFT_ERR_UNSUPPORTED_SIZE;
    if (output && d.length > 0 && !rows_apart(t, dim, heads, d.offsets ? 1 : d.nseq, d.length))
        return FFT_ERR_INVALID_ARG;
    return aligned_to(t.data, dtype_size(d.dtype)) ? FFT_OK : FFT_ERR_MISALIGNED;
}
int check_decay(const fft_seq& t, const fft_linattn_desc& d, bool output) {
    const fft_heads h = {t.data, t.seq_stride, t.tok_stride, 1};
    return check_heads(h, 1, d.heads, d, output);
}

int check_linattn(const fft_linattn_desc* d, bool pointers) {
    if (!d || d->dtype < FFT_F32 || d->dtype > FFT_F16) return FFT_ERR_INVALID_ARG;
    if (d->nseq < 1 || d->length < 0 || d->heads < 1 || d->groups < 1 || d->heads % d->groups || d->dk < 1 ||
        d->dv < 1)
        return FFT_ERR_INVALID_ARG;
    if (d->nseq > INT32_MAX || d->length > INT32_MAX - 65536 || d->heads > FFT_LINATTN_MAX_HEADS ||
        d->dk > FFT_LINATTN_MAX_DIM || d->dv > FFT_LINATTN_MAX_DIM)
        return FFT_ERR_UNSUPPORTED_SIZE;
    if (!aligned_to(d->offsets, 8)) return FFT_ERR_MISALIGNED;
    if (!pointers) return FFT_OK;
    if (!aligned_to(d->initial_state, 4)) return FFT_ERR_MISALIGNED;
    TRY(check_heads(d->q, d->dk, d->groups, *d, false));
    TRY(check_heads(d->k, d->dk, d->groups, *d, false));
    TRY(check_heads(d->v, d->dv, d->heads, *d, false));
    return check_decay(d->decay, *d, false);
}

// Whether an output shares values with what is read: as rows of columns where heads lie back to
// back, by their ranges of addresses otherwise.
struct Place {
    fft_heads t;
    int64_t dim, heads;
};
int64_t place_bytes(const Place& p, const fft_linattn_desc& d) {
    if (!p.t.data || d.length < 1) return 0;
    return ((d.offsets ? 0 : (d.nseq - 1) * p.t.seq_stride) + (d.length - 1) * p.t.tok_stride +
            (p.heads - 1) * p.t.head_stride + p.dim) * (int64_t)dtype_size(d.dtype);
}
bool places_meet(const Place& a, const Place& b, const fft_linattn_desc& d) {
    const size_t e = dtype_size(d.dtype);
    auto together = [](const Place& p) { return p.heads == 1 || p.t.head_stride == p.dim; };
    if (!bytes_meet(a.t.data, place_bytes(a, d), b.t.data, place_bytes(b, d))) return false;
    if (!together(a) || !together(b)) return true;
    const fft_seq x = {a.t.data, a.t.seq_stride, a.t.tok_stride}, y = {b.t.data, b.t.seq_stride, b.t.tok_stride};
    return seqs_meet(x, y, a.dim * a.heads, b.dim * b.heads, d.nseq, d.length, d.offsets, e);
}
Place decay_place(const fft_seq& t, int64_t heads) { return {{t.data, t.seq_stride, t.tok_stride, 1}, 1, heads}; }
bool meets_inputs(const Place& out, const fft_linattn_desc& d) {
    return places_meet(out, {d.q, d.dk, d.groups}, d) || places_meet(out, {d.k, d.dk, d.groups}, d) ||
           places_meet(out, {d.v, d.dv, d.heads}, d) || places_meet(out, decay_place(d.decay, d.heads), d);
}
// Bytes of `count` states (heads, dk and dv are at most 2^32 together), and whether rows reach into them, or
// states into what is read.
int64_t state_bytes(int64_t count, const fft_linattn_desc& d) {
    const int64_t one = d.heads * d.dk * d.dv;
    return (count > kMaxElements / one ? kMaxElements : count * one) * 4;
}
bool meets_states(const Place& p, const float* states, int64_t count, const fft_linattn_desc& d) {
    return bytes_meet(p.t.data, place_bytes(p, d), states, state_bytes(count, d));
}
bool states_meet_inputs(const float* states, const fft_linattn_desc& d) {
    for (const Place& p : {Place{d.q, d.dk, d.groups}, Place{d.k, d.dk, d.groups}, Place{d.v, d.dv, d.heads},
                           decay_place(d.decay, d.heads)})
        if (meets_states(p, states, d.nseq, d)) return true;
    return false;
}

AttnRows rows_of(const fft_heads& t, int64_t dim, int64_t heads, const fft_linattn_desc& d, int share) {
    const int64_t e = (int64_t)dtype_size(d.dtype);
    const int64_t seq = d.offsets || d.nseq == 1 ? 0 : t.seq_stride, tok = d.length > 1 ? t.tok_stride : 0,
                  head = heads > 1 ? t.head_stride : 0;
    AttnRows r = {t.data, seq, tok, head, share, 0};
    for (int v : {16, 4})
        if (!r.vec && aligned_to(t.data, v) && dim * e % v == 0 && seq * e % v == 0 && tok * e % v == 0 && head * e % v == 0)
            r.vec = v;
    return r;
}

int64_t up16(int64_t bytes) { return (bytes + 15) / 16 * 16; }

// One pass of the kernel: shapes, and time cut into as many segments as give the least time, counted
// in rounds of resident blocks times the chunks of a segment, a chunk as 4, `start` more for every block and
// half as much again for the summaries of a cut call, which reads keys and values twice (1.3 to 1.6 times the
// uncut kernel's time in a profile).  Measured at 17 shapes against 1 to 32 segments: within 4% of the best cut in
// 14 of them, within 9% in two (float16 gradients and float32 outputs of 4 x 2048 tokens), and half as long again in
// float16 gradients of 16 heads of 64 x 64, where two blocks fit an SM and the gradients' plan counts one.
void attn_plan(const fft_linattn_desc& d, int64_t dx, int64_t dz, AttnArgs* a) {
    a->offsets = d.offsets;
    a->nseq = d.nseq;
    a->length = d.length;
    a->rows = d.offsets ? 1 : d.nseq;
    a->heads = d.heads;
    a->dx = dx;
    a->dz = dz;
    const int64_t zt = attn_ztile(d.dtype, dx, dz);
    a->ztiles = (dz + zt - 1) / zt;
}
// Whether sizes and type are the tcgen05 kernel's; rows have to lie on 16-byte boundaries too.
bool tc_sizes(const fft_linattn_desc& d, bool backward) {
    return d.dtype == FFT_BF16 && d.dk <= 128 && (!backward || d.dv <= 128);
}
int64_t attn_segment(const fft_linattn_desc& d, int64_t ztiles, int64_t resident, int64_t chunk, int64_t start) {
    const int64_t rows = d.offsets ? 1 : d.nseq, blocks = rows * d.heads * ztiles;
    int64_t segment = (d.length + chunk - 1) / chunk * chunk, best = INT64_MAX;
    for (int64_t k = 1; k <= 256; ++k) {
        int64_t size = (d.length + k - 1) / k;
        size = (size + chunk - 1) / chunk * chunk;
        const int64_t n = (d.length + size - 1) / size;
        const int64_t cost = (blocks * n + resident - 1) / resident * (size / chunk * (n > 1 ? 6 : 4) + start) + (n > 1 ? 2 * start : 0);
        if (cost < best) best = cost, segment = size;
        if (size <= chunk) break;
    }
    return segment < 1 ? chunk : segment;
}
void attn_cut(AttnArgs* a, int64_t segment) {
    a->segment = segment;
    a->nsegments = (a->length + segment - 1) / segment;
}

struct Taker {
    char* w;
    int64_t at = 0;
    template <class P>
    P* take(int64_t count) {
        P* p = reinterpret_cast<P*>(w ? w + at : nullptr);
        at += up16(count * (int64_t)sizeof(P));
        return p;
    }
};
void take_carry(AttnArgs* a, int dtype, Taker* t) {
    if (a->nsegments < 2) return;
    const int64_t n = a->rows * a->nsegments * a->heads;
    a->carry = t->take<float>(n * a->ztiles * attn_carry(dtype, a->dx, a->dz));
    a->carry_decay = t->take<float>(n);
    a->carry_reset = t->take<int>(n);
}

int64_t forward_layout(const fft_linattn_desc& d, AttnArgs* a, char* w) {
    attn_plan(d, d.dk, d.dv, a);
    const bool tc = tc_sizes(d, false);
    const int64_t resident = (int64_t)num_sms() * (!tc && attn_warps(d.dtype, d.dk, d.dv) == 4 ? 2 : 1);
    attn_cut(a, attn_segment(d, a->ztiles, resident, tc ? kTcChunk : kAttnChunk, 8));
    Taker t = {w};
    take_carry(a, d.dtype, &t);
    return t.at;
}

// The three passes of the gradients share their cuts, so that chunks are the same ones.
struct BackwardPlan {
    AttnArgs q, k, v;  // passes for dq, dk, dv
    DecayGradArgs g;
    float *dq_parts, *dk_parts;
};
int64_t backward_layout(const fft_linattn_desc& d, const fft_linattn_grads* gr, BackwardPlan* p, char* w) {
    attn_plan(d, d.dv, d.dk, &p->q);
    attn_plan(d, d.dv, d.dk, &p->k);
    attn_plan(d, d.dk, d.dv, &p->v);
    const int64_t zk = p->q.ztiles, zv = p->v.ztiles;
    // start: the tcgen05 kernel's chunks take longer than a block's start here (4 x 2048 tokens of 16 heads of
    // 128 x 128, 480 us with 8, uncut, and 454 us with 3, cut in two); 13 packed rows of 4001 tokens of 8 heads in
    // float16 391 us with 8 and 421 us with 3
    const bool tc = tc_sizes(d, true);
    const int64_t segment = attn_segment(d, zk > zv ? zk : zv, (int64_t)num_sms(), tc ? kTcChunk : kAttnChunk, tc ? 3 : 8);
    Taker t = {w};
    for (AttnArgs* a : {&p->q, &p->k, &p->v}) {
        attn_cut(a, segment);
        take_carry(a, d.dtype, &t);
    }
    // the tcgen05 kernel leaves the sums of rows in halves
    const int64_t tokens = p->q.rows * d.length, dots = (tc_sizes(d, true) ? 2 : 1) * zk * d.heads * tokens;
    p->q.dots_inter = t.take<float>(dots);
    p->q.dots_all = t.take<float>(dots);
    p->k.dots_inter = t.take<float>(dots);
    p->k.dots_all = t.take<float>(dots);
    const int64_t n = p->q.rows * p->q.nsegments * d.heads;
    float* final_dots = t.take<float>(zk * d.nseq * d.heads);
    DecayGradArgs& g = p->g;
    g.carry = t.take<double>(n);
    g.stops = t.take<int>(n);
    const bool shared = d.heads > d.groups;
    p->dq_parts = shared ? t.take<float>(tokens * d.heads * d.dk) : nullptr;
    p->dk_parts = shared ? t.take<float>(tokens * d.heads * d.dk) : nullptr;
    if (!w || !gr) return t.at;
    p->q.final_dots = final_dots;
    g.decay = d.decay;
    g.ddecay = gr->ddecay;
    g.offsets = d.offsets;
    g.nseq = d.nseq;
    g.length = d.length;
    g.rows = p->q.rows;
    g.heads = d.heads;
    g.segment = segment;
    g.nsegments = p->q.nsegments;
    g.ztiles = g.final_tiles = zk;
    g.initial = d.initial_state != nullptr;
    g.q_inter = p->q.dots_inter;
    g.q_all = p->q.dots_all;
    g.k_inter = p->k.dots_inter;
    g.k_all = p->k.dots_all;
    g.final_dots = gr->dfinal_state ? final_dots : nullptr;
    return t.at;
}

void set_out(AttnArgs* a, const fft_heads& out, const fft_linattn_desc& d, float* parts) {
    if (parts) {
        a->out = parts;
        a->out_f32 = 1;
        a->out_head = a->dz;
        a->out_tok = d.heads * a->dz;
        a->out_seq = d.length * a->out_tok;
        return;
    }
    a->out = out.data;
    a->out_seq = d.offsets ? 0 : out.seq_stride;
    a->out_tok = out.tok_stride;
    a->out_head = out.head_stride;
    a->out_pair = a->dz % 2 == 0 && aligned_to(out.data, 2 * dtype_size(d.dtype)) && a->out_seq % 2 == 0 &&
                  a->out_tok % 2 == 0 && a->out_head % 2 == 0;
}

template <class F32, class B16, class F16>
cudaError_t by_type(int dtype, F32 f32, B16 b16, F16 f16, const AttnArgs& a, cudaStream_t s) {
    return dtype == FFT_F32 ? f32(a, s) : (dtype == FFT_BF16 ? b16(a, s) : f16(a, s));
}
// The device's error word: set by a wait that has run out; and what a check has taken out of it.
__device__ int g_attn_error, g_attn_taken;
__global__ void k_take_error() { g_attn_taken = atomicExch(&g_attn_error, 0); }
cudaError_t error_word(int** word) {
    return cudaGetSymbolAddress(reinterpret_cast<void**>(word), g_attn_error);
}
// Whether a pass runs on tcgen05: its rows and outputs lie on 16-byte boundaries.
bool tc_rows(const AttnArgs& a) {
    auto even = [](int64_t stride) { return stride % 8 == 0; };
    return a.x.vec == 16 && a.y.vec == 16 && a.z.vec == 16 && (!a.partner.data || a.partner.vec == 16) &&
           aligned_to(a.out, 16) && even(a.out_seq) && even(a.out_tok) && even(a.out_head);
}
std::atomic<uint32_t> g_wait_ns{2000000000u};  // limit of a device-side wait
cudaError_t run_tc(AttnArgs a, bool backward, cudaStream_t s) {
    int* err = nullptr;
    const cudaError_t e = error_word(&err);
    if (e != cudaSuccess) return e;
    a.wait_ns = g_wait_ns.load();
    return backward ? attn_tc_bwd(a, err, s) : attn_tc_fwd(a, err, s);
}
cudaError_t run_forward(const AttnArgs& a, int dtype, cudaStream_t s) {
    return by_type(dtype, attn_f32_fwd, attn_bf16_fwd, attn_f16_fwd, a, s);
}
cudaError_t run_backward(const AttnArgs& a, int dtype, cudaStream_t s) {
    return by_type(dtype, attn_f32_bwd, attn_bf16_bwd, attn_f16_bwd, a, s);
}

cudaError_t fill_empty(const fft_linattn_desc& d, const float* from, float* to, cudaStream_t s) {
    const int64_t per = d.heads * d.dk * d.dv;
    if (!to) return cudaSuccess;
    if (d.offsets && d.length > 0) {
        k_linattn_empty<<<(unsigned)d.nseq, 256, 0, s>>>(d.offsets, from, to, per);
        return cudaGetLastError();
    }
    if (d.length > 0) return cudaSuccess;
    const size_t bytes = (size_t)(d.nseq * per) * sizeof(float);
    return from ? cudaMemcpyAsync(to, from, bytes, cudaMemcpyDeviceToDevice, s) : cudaMemsetAsync(to, 0, bytes, s);
}

template <class T>
cudaError_t run_shared(const float* parts, const fft_heads& out, const fft_linattn_desc& d, cudaStream_t s) {
    const int64_t total = (d.offsets ? 1 : d.nseq) * d.length * d.groups * d.dk;
    const int64_t blocks = (total + 255) / 256;
    if (blocks > INT32_MAX) return cudaErrorInvalidValue;
    k_linattn_shared<T><<<(unsigned)blocks, 256, 0, s>>>(parts, out, d.length, d.groups, d.heads / d.groups, d.dk,
                                                         total);
    return cudaGetLastError();
}

template <class T>
cudaError_t finish_backward(const BackwardPlan& p, const fft_linattn_desc& d, const fft_linattn_grads& g,
                            bool tc, cudaStream_t s) {
    const unsigned blocks = (unsigned)(p.g.rows * p.g.nsegments * p.g.heads);
    if (p.g.nsegments > 1) k_decay_sums<<<blocks, kDgWarps * 32, 0, s>>>(p.g);
    if (tc)
        k_decay_grads<T, kTcChunk / 32><<<blocks, kDgWarps * 32, 0, s>>>(p.g);
    else
        k_decay_grads<T, kAttnChunk / 32><<<blocks, kDgWarps * 32, 0, s>>>(p.g);
    cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess && p.dq_parts) e = run_shared<T>(p.dq_parts, g.dq, d, s);
    if (e == cudaSuccess && p.dk_parts) e = run_shared<T>(p.dk_parts, g.dk, d, s);
    return e;
}

}  // namespace
}  // namespace gbfft

using namespace gbfft;

extern "C" int fft_linattn_workspace(const fft_linattn_desc* d, int backward, size_t* bytes) {
    if (!bytes || (backward != 0 && backward != 1)) return FFT_ERR_INVALID_ARG;
    TRY(check_linattn(d, false));
    AttnArgs a = {};
    BackwardPlan p = {};
    *bytes = d->length < 1 ? 0 : (size_t)(backward ? backward_layout(*d, nullptr, &p, nullptr)
                                                  : forward_layout(*d, &a, nullptr));
    return FFT_OK;
}

extern "C" int fft_linattn_forward(const fft_linattn_desc* d, const fft_heads* out, float* final_state,
                                   void* workspace, size_t workspace_bytes, void* stream) {
    TRY(check_linattn(d, true));
    if (!out) return FFT_ERR_INVALID_ARG;
    TRY(check_heads(*out, d->dv, d->heads, *d, true));
    if (!aligned_to(final_state, 4) || !aligned_to(workspace, 16)) return FFT_ERR_MISALIGNED;
    const int64_t states = state_bytes(d->nseq, *d);
    const Place place = {*out, d->dv, d->heads};
    if (meets_inputs(place, *d) || meets_states(place, d->initial_state, d->nseq, *d) ||
        meets_states(place, final_state, d->nseq, *d) || states_meet_inputs(final_state, *d) ||
        bytes_meet(final_state, states, d->initial_state, states))
        return FFT_ERR_INVALID_ARG;
    cudaStream_t s = (cudaStream_t)stream;
    if (d->length > 0) {
        AttnArgs a = {};
        const int64_t need = forward_layout(*d, &a, static_cast<char*>(workspace));
        if (need > 0 && (!workspace || workspace_bytes < (size_t)need)) return FFT_ERR_INVALID_ARG;
        const int share = (int)(d->heads / d->groups);
        a.x = rows_of(d->q, d->dk, d->groups, *d, share);
        a.y = rows_of(d->k, d->dk, d->groups, *d, share);
        a.z = rows_of(d->v, d->dv, d->heads, *d, 1);
        a.decay = d->decay;
        a.scale_pair = a.scale_inter = d->scale;
        a.scale_update = 1.f;
        a.initial = d->initial_state;
        a.final_state = final_state;
        a.state_x = d->dv;
        a.state_z = 1;
        set_out(&a, *out, *d, nullptr);
        TRY(status(tc_sizes(*d, false) && tc_rows(a) ? run_tc(a, false, s) : run_forward(a, d->dtype, s)));
    }
    return status(fill_empty(*d, d->initial_state, final_state, s));
}

extern "C" int fft_linattn_backward(const fft_linattn_desc* d, const fft_linattn_grads* g, void* workspace,
                                    size_t workspace_bytes, void* stream) {
    TRY(check_linattn(d, true));
    if (!g) return FFT_ERR_INVALID_ARG;
    TRY(check_heads(g->dout, d->dv, d->heads, *d, false));
    TRY(check_heads(g->dq, d->dk, d->groups, *d, true));
    TRY(check_heads(g->dk, d->dk, d->groups, *d, true));
    TRY(check_heads(g->dv, d->dv, d->heads, *d, true));
    TRY(check_decay(g->ddecay, *d, true));
    if (!aligned_to(g->dfinal_state, 4) || !aligned_to(g->dinitial_state, 4) || !aligned_to(workspace, 16))
        return FFT_ERR_MISALIGNED;
    const int64_t states = state_bytes(d->nseq, *d);
    const Place dout = {g->dout, d->dv, d->heads};
    for (const Place& o : {Place{g->dq, d->dk, d->groups}, Place{g->dk, d->dk, d->groups},
                           Place{g->dv, d->dv, d->heads}, decay_place(g->ddecay, d->heads)})
        if (meets_inputs(o, *d) || places_meet(o, dout, *d) || meets_states(o, d->initial_state, d->nseq, *d) ||
            meets_states(o, g->dfinal_state, d->nseq, *d) || meets_states(o, g->dinitial_state, d->nseq, *d))
            return FFT_ERR_INVALID_ARG;
    if (states_meet_inputs(g->dinitial_state, *d) || meets_states(dout, g->dinitial_state, d->nseq, *d) ||
        bytes_meet(g->dinitial_state, states, d->initial_state, states) ||
        bytes_meet(g->dinitial_state, states, g->dfinal_state, states))
        return FFT_ERR_INVALID_ARG;
    cudaStream_t s = (cudaStream_t)stream;
    if (d->length > 0) {
        BackwardPlan p = {};
        const int64_t need = backward_layout(*d, g, &p, static_cast<char*>(workspace));
        if (!workspace || workspace_bytes < (size_t)need) return FFT_ERR_INVALID_ARG;
        const int share = (int)(d->heads / d->groups);
        const AttnRows q = rows_of(d->q, d->dk, d->groups, *d, share), k = rows_of(d->k, d->dk, d->groups, *d, share),
                       v = rows_of(d->v, d->dv, d->heads, *d, 1), o = rows_of(g->dout, d->dv, d->heads, *d, 1);
        AttnArgs& a = p.q;  // dq[i] = sum over j <= i of (dout[i] v[j]) k[j]
        a.x = o, a.y = v, a.z = k, a.partner = q;
        a.initial = d->initial_state;
        a.scale_pair = a.scale_inter = d->scale;
        a.scale_update = 1.f;
        a.state_x = 1, a.state_z = d->dv;
        a.final_dot = g->dfinal_state;
        set_out(&a, g->dq, *d, p.dq_parts);
        AttnArgs& b = p.k;  // dk[j] = sum over i >= j of (v[j] dout[i]) q[i]
        b.x = v, b.y = o, b.z = q, b.partner = k;
        b.state_x = 1, b.state_z = d->dv;
        set_out(&b, g->dk, *d, p.dk_parts);
        AttnArgs& c = p.v;  // dv[j] = sum over i >= j of (k[j] q[i]) dout[i]
        c.x = k, c.y = q, c.z = o;
        c.state_x = d->dv, c.state_z = 1;
        c.final_state = g->dinitial_state;
        set_out(&c, g->dv, *d, nullptr);
        for (AttnArgs* r : {&b, &c}) {
            r->reverse = 1;
            r->initial = g->dfinal_state;
            r->scale_pair = r->scale_update = d->scale;
            r->scale_inter = 1.f;
        }
        a.decay = b.decay = c.decay = d->decay;
        // all three on the same kernel: the decay's gradient takes their sums by chunks
        const bool tc = tc_sizes(*d, true) && tc_rows(a) && tc_rows(b) && tc_rows(c);
        for (const AttnArgs* r : {&a, &b, &c}) TRY(status(tc ? run_tc(*r, true, s) : run_backward(*r, d->dtype, s)));
        if (tc) p.g.ztiles *= 2;
        TRY(status(d->dtype == FFT_F32 ? finish_backward<float>(p, *d, *g, tc, s)
                                       : (d->dtype == FFT_BF16 ? finish_backward<__nv_bfloat16>(p, *d, *g, tc, s)
                                                               : finish_backward<__half>(p, *d, *g, tc, s))));
    }
    return status(fill_empty(*d, g->dfinal_state, g->dinitial_state, s));
}

extern "C" int fft_linattn_check(void* stream) {
    // read and cleared in one operation, by one thread at a time: no error between the two is lost
    static std::mutex one;
    std::lock_guard<std::mutex> lock(one);
    cudaStream_t s = (cudaStream_t)stream;
    void* taken = nullptr;
    int h = 0;
    if (cudaGetSymbolAddress(&taken, g_attn_taken) != cudaSuccess) return FFT_ERR_CUDA;
    k_take_error<<<1, 1, 0, s>>>();
    if (cudaGetLastError() != cudaSuccess ||
        cudaMemcpyAsync(&h, taken, sizeof(int), cudaMemcpyDeviceToHost, s) != cudaSuccess ||
        cudaStreamSynchronize(s) != cudaSuccess)
        return FFT_ERR_CUDA;
    return kerr_status(h);
}

extern "C" int fft_linattn_set_wait_timeout(uint64_t ns) {
    g_wait_ns.store(ns < 4000000000u ? (uint32_t)ns : 4000000000u);
    return FFT_OK;
}

extern "C" int fft_linattn_step(const fft_linattn_desc* d, const fft_heads* out, float* state, int64_t pool,
                                const int64_t* slots, const int64_t* slots_out, void* stream) {
    TRY(check_linattn(d, true));
    if (!out || d->length != 1 || d->offsets || pool < 0) return FFT_ERR_INVALID_ARG;
    if ((pool > 0 && !state) || (!slots && pool < d->nseq)) return FFT_ERR_INVALID_ARG;
    if (!aligned_to(slots, 8) || !aligned_to(slots_out, 8) || !aligned_to(state, 4)) return FFT_ERR_MISALIGNED;
    TRY(check_heads(*out, d->dv, d->heads, *d, true));
    const Place place = {*out, d->dv, d->heads};
    if (meets_inputs(place, *d) || meets_states(place, state, pool, *d)) return FFT_ERR_INVALID_ARG;
    const AttnStepArgs a = {*d, *out, state, slots, slots_out, pool, 0};
    cudaStream_t s = (cudaStream_t)stream;
    return status(d->dtype == FFT_F32 ? attn_step<float>(a, s)
                                      : (d->dtype == FFT_BF16 ? attn_step<__nv_bfloat16>(a, s) : attn_step<__half>(a, s)));
}
