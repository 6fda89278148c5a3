// Root-mean-square norm with the residual's addition (fft_norm_forward, fft_norm_backward):
//   r = x + residual;  y = r * rstd * weight,  rstd = 1 / sqrt(mean(r^2) + eps)
// in the inputs' type or in e4m3 with one scale per row or group of columns, and its gradient
//   dr = rstd (w dy) - r rstd^3 mean(w dy r) + dresidual,  dweight = sum_rows dy r rstd.
// A dozen operations per element: bound by HBM.  Each row is read once into registers (up to 16
// values per thread), reduced across its threads, and written once.  Measured with inputs that
// change from call to call: 16384 rows of 4096 bfloat16 with a bfloat16 residual to e4m3 82 us,
// 5.7 TB/s (84% of the copy rate; 69 us from a clean L2); gradients of 8192 x 2560 bfloat16 with a
// float32 residual 79 us, 4.2 TB/s, where five tensors per row leave room for two rows on their
// way.  What carried it: weights in registers (reading them for every row filled the L1 port), a
// ring of later rows in shared memory instead of registers (130 -> 81 us), sums over the warps of
// a row by one shuffle tree instead of a loop.  Rows off 16-byte boundaries, which are loaded value by
// value when they are needed, are far from that: 16384 x 4095 347 us, to e4m3 356, with a scale per
// 128 columns 772 (an atomic maximum for every value).
#include <cuda_fp8.h>

#include "launch_cache.cuh"
#include "seq_common.cuh"
#include "seq_overlap.h"

namespace gbfft {
namespace {

constexpr int kMaxWarps = 32;
constexpr int kNormResident = 1024;  // threads of an SM: 64 registers each

struct NormArgs {
    const void* x;
    const void* residual;  // may be null
    void* out;
    float* scale;
    void* sum;  // may be null
    const void* weight;
    int64_t x_stride, residual_stride, out_stride, sum_stride;
    int64_t rows;
    int columns, wf32, wvec, group;
    float fcolumns, eps;
};

// The values of a thread are kept as pairs, two float32 operations to an instruction: value
// i * VEC + k is element k of its pack i.
template <int E>
struct Values {
    float2 v[E / 2];
    __device__ __forceinline__ float& operator[](int e) { return e & 1 ? v[e / 2].y : v[e / 2].x; }
};
template <class T, int VEC, int E>
__device__ __forceinline__ void unpack(const Pack<T, VEC>& p, int i, bool in, Values<E>& x) {
#pragma unroll
    for (int k = 0; k < VEC; ++k) x[i * VEC + k] = in ? to_f(p.v[k]) : 0.f;
}
template <class T, int VEC, int E>
__device__ __forceinline__ Pack<T, VEC> pack(Values<E>& x, int i) {
    Pack<T, VEC> p;
    if constexpr (VEC == 1) {
        p.v[0] = from_f<T>(x[i]);
    } else {
#pragma unroll
        for (int k = 0; k < VEC; k += 2) {
            const Pack<T, 2> y = from_f2<T>(x.v[(i * VEC + k) / 2]);
            p.v[k] = y.v[0];
            p.v[k + 1] = y.v[1];
        }
    }
    return p;
}

// The weights of pack i at column c, 0 beyond the row; wvec: they are on a 16-byte boundary.
template <class T, int VEC, int E, class A>
__device__ __forceinline__ void load_weight(const A& a, int i, int c, Values<E>& w) {
    const bool in = c < a.columns;
    if (a.wf32 && a.wvec) {
        Pack<float, VEC> p = {};
        if (in) p = ld_pack<VEC>(static_cast<const float*>(a.weight) + c);
        unpack<float, VEC, E>(p, i, true, w);
    } else if (a.wvec) {
        Pack<T, VEC> p;
        if (in) p = ld_pack<VEC>(static_cast<const T*>(a.weight) + c);
        unpack<T, VEC, E>(p, i, in, w);
    } else {
#pragma unroll
        for (int k = 0; k < VEC; ++k) w[i * VEC + k] = in ? ld_param<T>(a.weight, c + k, a.wf32) : 0.f;
    }
}

// Sums over a warp, then over the warps that share a row, side by side.
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
__device__ __forceinline__ float warps_sum(const float* red, int warps) {
    const int lane = (int)threadIdx.x & 31;
    return warp_sum(lane < warps ? red[lane] : 0.f);
}
__device__ __forceinline__ float max_abs_nan(float m, float v) {  // a NaN stays
    return max_nan(m, fabsf(v));
}

// 448 / m, for t = r * weight and m = max |t|: with q = t * (448 / m) rstd cancels, and m * rstd is
// max |y|.  0 where y is 0 all over the group; a NaN stays.  Below kTiny the quotient is beyond
// float32: m counts raised by kRaise there, and so have the values to be.
constexpr float kTiny = 0x1p-119f, kRaise = 0x1p64f;
__device__ __forceinline__ float e4m3_inv(float m, float my) {
    if (my == 0.f) return 0.f;
    return 448.f / (m < kTiny ? m * kRaise : m);
}

// Rows ahead of the present one wait in shared memory: a thread copies the 16-byte pieces of its
// own columns asynchronously and reads only those, so a ring of rows needs no barrier and no
// registers.  PIECES per thread and row; as many rows, up to four, as two blocks of an SM have room
// for (one block of 1024 threads).  Less than two, or rows of single values: no ring, the row is
// loaded when it is needed.
template <int PIECES, int MAXT>
struct Ring {
    static constexpr int kFit = (MAXT > 512 ? 200 : 100) * 1024 / (PIECES * 16 * MAXT);
    static constexpr int kDepth = kFit > 4 ? 4 : kFit;
    char* base;
    __device__ __forceinline__ void* at(int stage, int piece) const {
        return base + ((stage * PIECES + piece) * (int)blockDim.x + (int)threadIdx.x) * 16;
    }
    static size_t bytes(int threads) { return (size_t)kDepth * PIECES * 16 * threads; }
};

// Threads: tpr per row, blockDim.x / tpr rows per block; thread j of a row holds the packs
// j, j + tpr, ... (NV of VEC columns) and their weights, and its block takes rows at a stride of
// the grid.  OUT: 0 = type T, 1 = e4m3 with one scale per row, 2 = e4m3 with a scale per `group`
// columns (32, 64 or 128).  Blocks of more than 512 threads (MAXT 1024) have no registers for the
// weights: they load them for every row.
template <class T, class R, int VEC, int NV, int OUT, int MAXT>
__global__ void __launch_bounds__(MAXT, kNormResident / MAXT) k_norm_fwd(const NormArgs a, int tpr) {
    constexpr int E = NV * VEC, RP = VEC > 1 ? VEC * (int)sizeof(R) / 16 : 0;
    using Rows = Ring<NV * (1 + RP), MAXT>;
    constexpr bool KEEP = MAXT <= 512, AHEAD = VEC > 1 && Rows::kDepth > 1;
    extern __shared__ uint4 dynamic[];
    unsigned* group_max = reinterpret_cast<unsigned*>(dynamic);  // VEC 1, OUT 2: [row][group]
    Rows ring{reinterpret_cast<char*>(dynamic)};
    __shared__ float red[2][kMaxWarps], redm[2][kMaxWarps];
    const int local = (int)threadIdx.x / tpr, j = (int)threadIdx.x - local * tpr;
    const int lane = (int)threadIdx.x & 31, warp = (int)threadIdx.x >> 5;
    const int warp0 = local * (tpr >> 5), warps = tpr >> 5, rpb = (int)blockDim.x / tpr;
    const int groups = OUT == 2 ? (a.columns + a.group - 1) / a.group : 1;
    Values<E> w;
    auto weights = [&]() {
#pragma unroll
        for (int i = 0; i < NV; ++i) load_weight<T, VEC, E>(a, i, (i * tpr + j) * VEC, w);
    };
    if (KEEP) weights();
    auto ahead = [&](int64_t row, int stage) {
        const T* x = static_cast<const T*>(a.x) + row * a.x_stride;
        const R* res = static_cast<const R*>(a.residual) + row * a.residual_stride;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * tpr + j) * VEC;
            const bool in = row < a.rows && c < a.columns;
            copy16(ring.at(stage, i), in ? x + c : a.x, in);
            if (a.residual) {
#pragma unroll
                for (int k = 0; k < RP; ++k)
                    copy16(ring.at(stage, NV + i * RP + k), in ? res + c + k * 16 / (int)sizeof(R) : a.residual, in);
            }
        }
        copy_commit();
    };
    const int64_t step = (int64_t)gridDim.x * rpb;
    int buf = 0;
    int stage = 0;
    if constexpr (AHEAD) {
#pragma unroll
        for (int k = 0; k < Rows::kDepth - 1; ++k) ahead((int64_t)blockIdx.x * rpb + local + k * step, k);
    }
    for (int64_t base = (int64_t)blockIdx.x * rpb; base < a.rows; base += step, buf ^= 1) {
        const int64_t row = base + local;
        const bool live = row < a.rows;
        Values<E> v;
        if constexpr (AHEAD) {
            ahead(row + (Rows::kDepth - 1) * step, stage ? stage - 1 : Rows::kDepth - 1);
            copy_wait<Rows::kDepth - 1>();
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                unpack<T, VEC, E>(ld_pack<VEC>(static_cast<const T*>(ring.at(stage, i))), i, true, v);
                if (a.residual) {
                    Values<E> r;
                    Pack<R, VEC> p;
#pragma unroll
                    for (int k = 0; k < RP; ++k)
                        reinterpret_cast<uint4*>(&p)[k] =
                            *static_cast<const uint4*>(ring.at(stage, NV + i * RP + k));
                    unpack<R, VEC, E>(p, i, true, r);
#pragma unroll
                    for (int e = i * VEC / 2; e < (i + 1) * VEC / 2; ++e) v.v[e] = add2(v.v[e], r.v[e]);
                }
            }
            stage = stage + 1 < Rows::kDepth ? stage + 1 : 0;
        } else {
            const T* x = static_cast<const T*>(a.x) + row * a.x_stride;
            const R* res = static_cast<const R*>(a.residual) + row * a.residual_stride;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = (i * tpr + j) * VEC;
                const bool in = live && c < a.columns;
                Pack<T, VEC> p;
                Pack<R, VEC> q;
                if (in) p = ld_pack<VEC>(x + c);
                if (in && a.residual) q = ld_pack<VEC>(res + c);
                unpack<T, VEC, E>(p, i, in, v);
#pragma unroll
                for (int k = 0; k < VEC; ++k)
                    if (in && a.residual) v[i * VEC + k] += to_f(q.v[k]);
            }
        }
        float2 ss2 = splat(0.f);
#pragma unroll
        for (int e = 0; e < E / 2; ++e) ss2 = fma2(v.v[e], v.v[e], ss2);
        float ss = warp_sum(ss2.x + ss2.y);
        if (lane == 0) red[buf][warp] = ss;
        if (a.sum) {
            R* sum = static_cast<R*>(a.sum) + row * a.sum_stride;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = (i * tpr + j) * VEC;
                if (live && c < a.columns) st_pack<VEC>(sum + c, pack<R, VEC, E>(v, i));
            }
        }
        if (!KEEP) weights();
        if constexpr (OUT != 0) {
#pragma unroll
            for (int e = 0; e < E / 2; ++e) v.v[e] = mul2(v.v[e], w.v[e]);
        }
        // with one scale per row its maximum needs no rstd and shares the barrier; bit patterns of
        // |t| are ordered like the values, with NaN above infinity
        float m = 0.f;
        if constexpr (OUT == 1) {
#pragma unroll
            for (int e = 0; e < E; ++e) m = max_abs_nan(m, v[e]);
            m = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m)));
            if (lane == 0) redm[buf][warp] = m;
        }
        if constexpr (OUT == 2 && VEC == 1) {
            for (int i = (int)threadIdx.x; i < groups * rpb; i += (int)blockDim.x) group_max[i] = 0;
        }
        __syncthreads();  // the other buffers are written before the next one
        ss = warps_sum(red[buf] + warp0, warps);
        const float rstd = rsqrtf(ss / a.fcolumns + a.eps);
        if constexpr (OUT == 0) {
            T* out = static_cast<T*>(a.out) + row * a.out_stride;
#pragma unroll
            for (int e = 0; e < E / 2; ++e) v.v[e] = mul2(mul2(v.v[e], splat(rstd)), w.v[e]);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = (i * tpr + j) * VEC;
                if (live && c < a.columns) st_pack<VEC>(out + c, pack<T, VEC, E>(v, i));
            }
        } else {
            if constexpr (OUT == 1)
                m = __uint_as_float(__reduce_max_sync(
                    0xffffffffu, lane < warps ? __float_as_uint(redm[buf][warp0 + lane]) : 0u));
            if constexpr (OUT == 2 && VEC == 1) {
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    const int c = i * tpr + j;
                    if (live && c < a.columns)
                        atomicMax(&group_max[local * groups + c / a.group],
                                  __float_as_uint(v[i]) & 0x7fffffffu);
                }
                __syncthreads();
            }
            uint8_t* out = static_cast<uint8_t*>(a.out) + row * a.out_stride;
            float inv = OUT == 1 ? e4m3_inv(m, m * rstd) : 0.f;
            if (OUT == 1 && live && j == 0) a.scale[row] = m * rstd / 448.f;
            if (OUT == 1 && m < kTiny) {
#pragma unroll
                for (int e = 0; e < E / 2; ++e) v.v[e] = mul2(v.v[e], splat(kRaise));
            }
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = (i * tpr + j) * VEC;
                const bool in = live && c < a.columns;
                if constexpr (OUT == 2) {
                    if constexpr (VEC == 1) {
                        m = in ? __uint_as_float(group_max[local * groups + c / a.group]) : 0.f;
                    } else {  // the group's packs are held by neighbouring lanes
                        m = 0.f;
#pragma unroll
                        for (int k = 0; k < VEC; ++k) m = max_abs_nan(m, v[i * VEC + k]);
                        for (int o = a.group / VEC / 2; o; o >>= 1)
                            m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
                    }
                    inv = e4m3_inv(m, m * rstd);
                    if (m < kTiny) {
#pragma unroll
                        for (int k = 0; k < VEC; ++k) v[i * VEC + k] *= kRaise;
                    }
                    if (in && c % a.group == 0) a.scale[row * groups + c / a.group] = m * rstd / 448.f;
                }
                if constexpr (VEC == 1) {
                    const uint8_t b = __nv_cvt_float_to_fp8(v[i] * inv, __NV_SATFINITE, __NV_E4M3);
                    if (in) out[c] = b;
                } else {
                    Pack<uint16_t, VEC / 2> p;
#pragma unroll
                    for (int k = 0; k < VEC; k += 2)
                        p.v[k / 2] = __nv_cvt_float2_to_fp8x2(mul2(v.v[(i * VEC + k) / 2], splat(inv)),
                                                              __NV_SATFINITE, __NV_E4M3);
                    if (in) st_pack<VEC / 2>(reinterpret_cast<uint16_t*>(out + c), p);
                }
            }
            // the next row clears the maxima
            if constexpr (OUT == 2 && VEC == 1) __syncthreads();
        }
    }
    if constexpr (AHEAD) copy_wait<0>();  // rows beyond the last: zeros on their way to shared memory
}

struct NormBwdArgs {
    const void* dout;
    const void* r;
    const void* dres;  // may be null
    void* dsum;        // may be null
    void* dx;          // may be null
    const void* weight;
    float* parts;  // [blocks][columns], null: no dweight
    int64_t dout_stride, r_stride, dres_stride, dsum_stride, dx_stride;
    int64_t rows;
    int columns, wf32, wvec;
    float fcolumns, eps;
};

// One row per block at a time, rows blockIdx.x, + gridDim.x, ..., later ones on their way.  Every
// thread keeps its columns, so dweight is summed in registers and leaves as one partial row per
// block.  MAXT as above.
template <class T, class R, int VEC, int NV, int MAXT>
__global__ void __launch_bounds__(MAXT) k_norm_bwd(const NormBwdArgs a) {
    constexpr int E = NV * VEC, RP = VEC > 1 ? VEC * (int)sizeof(R) / 16 : 0;
    using Rows = Ring<NV * (1 + 2 * RP), MAXT>;
    constexpr bool KEEP = MAXT <= 512, AHEAD = VEC > 1 && Rows::kDepth > 1;
    extern __shared__ uint4 dynamic[];
    Rows ring{reinterpret_cast<char*>(dynamic)};
    __shared__ float red[2][2][kMaxWarps];
    const int j = (int)threadIdx.x, tpr = (int)blockDim.x, warps = tpr >> 5;
    const int lane = j & 31, warp = j >> 5;
    Values<E> dw, w;
#pragma unroll
    for (int e = 0; e < E / 2; ++e) dw.v[e] = splat(0.f);
    auto weights = [&]() {
#pragma unroll
        for (int i = 0; i < NV; ++i) load_weight<T, VEC, E>(a, i, (i * tpr + j) * VEC, w);
    };
    if (KEEP) weights();
    auto ahead = [&](int64_t row, int stage) {
        const R* r = static_cast<const R*>(a.r) + row * a.r_stride;
        const T* g = static_cast<const T*>(a.dout) + row * a.dout_stride;
        const R* d = static_cast<const R*>(a.dres) + row * a.dres_stride;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * tpr + j) * VEC;
            const bool in = row < a.rows && c < a.columns;
            copy16(ring.at(stage, i), in ? g + c : a.dout, in);
#pragma unroll
            for (int k = 0; k < RP; ++k) {
                const int at = c + k * 16 / (int)sizeof(R);
                copy16(ring.at(stage, NV + i * RP + k), in ? r + at : a.r, in);
                if (a.dres) copy16(ring.at(stage, NV * (1 + RP) + i * RP + k), in ? d + at : a.dres, in);
            }
        }
        copy_commit();
    };
    int buf = 0, stage = 0;
    if constexpr (AHEAD) {
#pragma unroll
        for (int k = 0; k < Rows::kDepth - 1; ++k) ahead(blockIdx.x + (int64_t)k * gridDim.x, k);
    }
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, buf ^= 1) {
        if (!KEEP) weights();
        Values<E> r, g, d;  // d: dresidual, then the result
        if constexpr (AHEAD) {
            ahead(row + (int64_t)(Rows::kDepth - 1) * gridDim.x, stage ? stage - 1 : Rows::kDepth - 1);
            copy_wait<Rows::kDepth - 1>();
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                unpack<T, VEC, E>(ld_pack<VEC>(static_cast<const T*>(ring.at(stage, i))), i, true, g);
                Pack<R, VEC> p, q = {};
#pragma unroll
                for (int k = 0; k < RP; ++k) {
                    reinterpret_cast<uint4*>(&p)[k] =
                        *static_cast<const uint4*>(ring.at(stage, NV + i * RP + k));
                    if (a.dres)
                        reinterpret_cast<uint4*>(&q)[k] =
                            *static_cast<const uint4*>(ring.at(stage, NV * (1 + RP) + i * RP + k));
                }
                unpack<R, VEC, E>(p, i, true, r);
                unpack<R, VEC, E>(q, i, a.dres != nullptr, d);
            }
            stage = stage + 1 < Rows::kDepth ? stage + 1 : 0;
        } else {
            const R* rr = static_cast<const R*>(a.r) + row * a.r_stride;
            const T* gg = static_cast<const T*>(a.dout) + row * a.dout_stride;
            const R* dd = static_cast<const R*>(a.dres) + row * a.dres_stride;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = (i * tpr + j) * VEC;
                const bool in = c < a.columns;
                Pack<R, VEC> p, q;
                Pack<T, VEC> o;
                if (in) {
                    p = ld_pack<VEC>(rr + c);
                    o = ld_pack<VEC>(gg + c);
                    if (a.dres) q = ld_pack<VEC>(dd + c);
                }
                unpack<R, VEC, E>(p, i, in, r);
                unpack<T, VEC, E>(o, i, in, g);
                unpack<R, VEC, E>(q, i, in && a.dres, d);
            }
        }
        float2 ss2 = splat(0.f), sg2 = splat(0.f);
#pragma unroll
        for (int e = 0; e < E / 2; ++e) {
            ss2 = fma2(r.v[e], r.v[e], ss2);
            sg2 = fma2(r.v[e], mul2(g.v[e], w.v[e]), sg2);
        }
        float ss = warp_sum(ss2.x + ss2.y), sg = warp_sum(sg2.x + sg2.y);
        if (lane == 0) {
            red[buf][0][warp] = ss;
            red[buf][1][warp] = sg;
        }
        __syncthreads();  // the other buffer is written before the next one
        ss = warps_sum(red[buf][0], warps);
        sg = warps_sum(red[buf][1], warps);
        const float rstd = rsqrtf(ss / a.fcolumns + a.eps);
        const float2 back = splat(-rstd * rstd * rstd * (sg / a.fcolumns)), rs = splat(rstd);
#pragma unroll
        for (int e = 0; e < E / 2; ++e) {
            const float2 gs = mul2(g.v[e], rs);
            dw.v[e] = fma2(gs, r.v[e], dw.v[e]);
            d.v[e] = add2(fma2(gs, w.v[e], mul2(r.v[e], back)), d.v[e]);
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * tpr + j) * VEC;
            if (c < a.columns) {
                if (a.dsum)
                    st_pack<VEC>(static_cast<R*>(a.dsum) + row * a.dsum_stride + c, pack<R, VEC, E>(d, i));
                if (a.dx)
                    st_pack<VEC>(static_cast<T*>(a.dx) + row * a.dx_stride + c, pack<T, VEC, E>(d, i));
            }
        }
    }
    if constexpr (AHEAD) copy_wait<0>();  // rows beyond the last: zeros on their way to shared memory
    if (a.parts) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * tpr + j) * VEC;
#pragma unroll
            for (int k = 0; k < VEC; ++k)
                if (c + k < a.columns) a.parts[(int64_t)blockIdx.x * a.columns + c + k] = dw[i * VEC + k];
        }
    }
}

// Column sums over the parts: 32 columns a block, 32 groups of parts summed side by side and
// then in order.
__global__ void __launch_bounds__(1024)
    k_sum_parts(const float* parts, int64_t nparts, int64_t stride, int64_t cols, float* out,
                int64_t chan, int64_t wide) {
    __shared__ float s[32][33];
    const int64_t col = (int64_t)blockIdx.x * 32 + threadIdx.x;
    float v = 0.f;
    if (col < cols)
        for (int64_t p = threadIdx.y; p < nparts; p += 32) v += parts[p * stride + col];
    s[threadIdx.y][threadIdx.x] = v;
    __syncthreads();
    if (threadIdx.y == 0 && col < cols) {
        v = 0.f;
#pragma unroll
        for (int i = 0; i < 32; ++i) v += s[i][threadIdx.x];
        const int64_t k = col / chan, c = col - k * chan;
        out[c * wide + k] = v;
    }
}

// 8 values per thread (one pack of 16-bit values, two of 32-bit ones) up to 4096 columns; longer
// rows take 16.
int values_per_thread(int64_t columns) { return columns <= 4096 ? 8 : 16; }
int threads_per_row(int64_t columns, int per_thread) {
    const int64_t t = (columns + per_thread - 1) / per_thread;
    return (int)((t + 31) / 32 * 32);
}

template <class T, class R, int VEC, int NV, int MAXT, int OUT>
cudaError_t launch_fwd(const NormArgs& a, cudaStream_t s) {
    const int tpr = threads_per_row(a.columns, VEC * NV), rpb = tpr >= 256 ? 1 : 256 / tpr;
    const int groups = OUT == 2 ? (a.columns + a.group - 1) / a.group : 1;
    using Rows = Ring<NV * (1 + (VEC > 1 ? VEC * (int)sizeof(R) / 16 : 0)), MAXT>;
    constexpr bool AHEAD = VEC > 1 && Rows::kDepth > 1;
    const size_t smem =
        AHEAD ? Rows::bytes(rpb * tpr) : (OUT == 2 && VEC == 1 ? rpb * groups * sizeof(unsigned) : 0);
    static LaunchCache cache;
    LaunchGeom geo;
    const cudaError_t e = cache.get([](int dev, LaunchGeom* g) {
        return setup_persistent(k_norm_fwd<T, R, VEC, NV, OUT, MAXT>, MAXT, AHEAD ? Rows::bytes(MAXT) : 16384, dev,
                                g);
    }, &geo);
    if (e != cudaSuccess) return e;
    const int64_t cap = (int64_t)geo.num_sms * (kNormResident / (rpb * tpr));
    const int64_t blocks = (a.rows + rpb - 1) / rpb;
    k_norm_fwd<T, R, VEC, NV, OUT, MAXT>
        <<<(unsigned)(blocks < cap ? blocks : cap), (unsigned)(rpb * tpr), smem, s>>>(a, tpr);
    return cudaGetLastError();
}
template <class T, class R, int VEC, int NV, int MAXT>
cudaError_t launch_fwd_out(const fft_norm_desc& d, const NormArgs& a, cudaStream_t s) {
    if (d.out_dtype != FFT_E4M3) return launch_fwd<T, R, VEC, NV, MAXT, 0>(a, s);
    return a.group == 0 ? launch_fwd<T, R, VEC, NV, MAXT, 1>(a, s)
                        : launch_fwd<T, R, VEC, NV, MAXT, 2>(a, s);
}

template <class T, class R>
cudaError_t norm_fwd(const fft_norm_desc& d, const NormArgs& a, cudaStream_t s) {
    constexpr int V = 16 / sizeof(T);
    const int64_t osz = d.out_dtype == FFT_E4M3 ? 1 : sizeof(T);
    auto rows16 = [&](const void* p, int64_t stride, int64_t size, int64_t al) {
        return !p || (aligned_to(p, al) && (a.rows == 1 || stride * size % al == 0));
    };
    const bool vec = a.columns % V == 0 && rows16(a.x, a.x_stride, sizeof(T), 16) &&
                     rows16(a.residual, a.residual_stride, sizeof(R), 16) &&
                     rows16(a.sum, a.sum_stride, sizeof(R), 16) &&
                     rows16(a.out, a.out_stride, osz, osz * V);
    if (!vec) {
        if (a.columns <= 4096) return launch_fwd_out<T, R, 1, 8, 512>(d, a, s);
        return a.columns <= 8192 ? launch_fwd_out<T, R, 1, 16, 512>(d, a, s)
                                 : launch_fwd_out<T, R, 1, 16, 1024>(d, a, s);
    }
    if (a.columns <= 4096) return launch_fwd_out<T, R, V, 8 / V, 512>(d, a, s);
    return a.columns <= 8192 ? launch_fwd_out<T, R, V, 16 / V, 512>(d, a, s)
                             : launch_fwd_out<T, R, V, 16 / V, 1024>(d, a, s);
}

template <class T, class R, int VEC, int NV, int MAXT>
cudaError_t launch_bwd(const NormBwdArgs& a, int64_t blocks, cudaStream_t s) {
    using Rows = Ring<NV * (1 + (VEC > 1 ? 2 * VEC * (int)sizeof(R) / 16 : 0)), MAXT>;
    constexpr bool AHEAD = VEC > 1 && Rows::kDepth > 1;
    const int threads = threads_per_row(a.columns, VEC * NV);
    static LaunchCache cache;
    LaunchGeom geo;
    const cudaError_t e = cache.get([](int dev, LaunchGeom* g) {
        return setup_persistent(k_norm_bwd<T, R, VEC, NV, MAXT>, MAXT, AHEAD ? Rows::bytes(MAXT) : 0, dev, g);
    }, &geo);
    if (e != cudaSuccess) return e;
    k_norm_bwd<T, R, VEC, NV, MAXT>
        <<<(unsigned)blocks, threads, AHEAD ? Rows::bytes(threads) : 0, s>>>(a);
    return cudaGetLastError();
}
template <class T, class R>
cudaError_t norm_bwd(const NormBwdArgs& a, int64_t blocks, cudaStream_t s) {
    constexpr int V = 16 / sizeof(T);
    auto rows16 = [&](const void* p, int64_t stride, int64_t size) {
        return !p || (aligned_to(p, 16) && (a.rows == 1 || stride * size % 16 == 0));
    };
    const bool vec = a.columns % V == 0 && rows16(a.dout, a.dout_stride, sizeof(T)) &&
                     rows16(a.r, a.r_stride, sizeof(R)) && rows16(a.dres, a.dres_stride, sizeof(R)) &&
                     rows16(a.dsum, a.dsum_stride, sizeof(R)) && rows16(a.dx, a.dx_stride, sizeof(T));
    if (!vec) {
        if (a.columns <= 4096) return launch_bwd<T, R, 1, 8, 512>(a, blocks, s);
        return a.columns <= 8192 ? launch_bwd<T, R, 1, 16, 512>(a, blocks, s)
                                 : launch_bwd<T, R, 1, 16, 1024>(a, blocks, s);
    }
    if (a.columns <= 8 * 384) return launch_bwd<T, R, V, 8 / V, 384>(a, blocks, s);
    if (a.columns <= 4096) return launch_bwd<T, R, V, 8 / V, 512>(a, blocks, s);
    return a.columns <= 8192 ? launch_bwd<T, R, V, 16 / V, 512>(a, blocks, s)
                             : launch_bwd<T, R, V, 16 / V, 1024>(a, blocks, s);
}

// Blocks of the backward pass: as many rows in flight as the SMs hold, and no more partial rows
// than that.
int64_t bwd_blocks(int64_t rows, int64_t columns) {
    const int t = threads_per_row(columns, values_per_thread(columns));
    const int64_t cap = (int64_t)num_sms() * (768 / t > 0 ? 768 / t : 1);
    return rows < cap ? rows : cap;
}

bool norm_types_ok(const fft_norm_desc& d) {
    if (d.dtype < FFT_F32 || d.dtype > FFT_F16) return false;
    if (d.res_dtype != d.dtype && d.res_dtype != FFT_F32) return false;
    return d.param_dtype == d.dtype || d.param_dtype == FFT_F32;
}
int norm_sizes(const fft_norm_desc* d) {
    if (!d || !norm_types_ok(*d) || !d->weight || d->rows < 0 || d->columns < 1 || !(d->eps >= 0.f))
        return FFT_ERR_INVALID_ARG;
    if (d->columns > FFT_NORM_MAX_COLUMNS || d->rows > INT32_MAX) return FFT_ERR_UNSUPPORTED_SIZE;
    return FFT_OK;
}
bool stride_ok(const void* p, int64_t stride, const fft_norm_desc* d) {
    return !p || stride >= d->columns || (d->rows <= 1 && stride >= 0);
}

// Whether rows that are written lie over rows that are read without being the same ones: a thread
// reads what it writes, and later rows are copied ahead.
bool rows_clash(const void* out, int64_t out_stride, size_t out_size, const void* in, int64_t in_stride,
                size_t in_size, const fft_norm_desc* d) {
    if (!out || !in || (out == in && out_size == in_size && (out_stride == in_stride || d->rows == 1)))
        return false;
    const fft_seq a = {const_cast<void*>(out), 0, out_stride * (int64_t)out_size};
    const fft_seq b = {const_cast<void*>(in), 0, in_stride * (int64_t)in_size};
    return seqs_meet(a, b, d->columns * (int64_t)out_size, d->columns * (int64_t)in_size, 1, d->rows,
                     false, 1);
}

}  // namespace

cudaError_t run_sum_parts(const float* parts, int64_t nparts, int64_t stride, int64_t cols,
                          float* out, int64_t chan, int64_t wide, cudaStream_t s) {
    k_sum_parts<<<(unsigned)((cols + 31) / 32), dim3(32, 32), 0, s>>>(parts, nparts, stride, cols,
                                                                     out, chan, wide);
    return cudaGetLastError();
}

}  // namespace gbfft

using namespace gbfft;

extern "C" int fft_norm_forward(const fft_norm_desc* d, const void* x, int64_t x_stride,
                                const void* residual, int64_t residual_stride, void* out,
                                int64_t out_stride, float* scale, void* sum, int64_t sum_stride,
                                void* stream) {
    int rc = norm_sizes(d);
    if (rc != FFT_OK) return rc;
    const bool q = d->out_dtype == FFT_E4M3;
    if (!q && d->out_dtype != d->dtype) return FFT_ERR_INVALID_ARG;
    const bool rows = d->rows > 0;  // tensors without rows may have no address
    if (q ? ((rows && !scale) || (d->group != 0 && d->group != 32 && d->group != 64 && d->group != 128))
          : d->group != 0)
        return FFT_ERR_INVALID_ARG;
    if ((rows && (!x || !out)) || !stride_ok(x, x_stride, d) || !stride_ok(residual, residual_stride, d) ||
        !stride_ok(out, out_stride, d) || !stride_ok(sum, sum_stride, d))
        return FFT_ERR_INVALID_ARG;
    const size_t e = dtype_size(d->dtype), r = dtype_size(d->res_dtype);
    if (!aligned_to(x, e) || !aligned_to(residual, r) || !aligned_to(sum, r) ||
        !aligned_to(out, dtype_size(d->out_dtype)) || !aligned_to(scale, 4) ||
        !aligned_to(d->weight, dtype_size(d->param_dtype)))
        return FFT_ERR_MISALIGNED;
    if (!rows) return FFT_OK;
    const size_t o = dtype_size(d->out_dtype);
    if (rows_clash(out, out_stride, o, x, x_stride, e, d) ||
        rows_clash(out, out_stride, o, residual, residual_stride, r, d) ||
        rows_clash(sum, sum_stride, r, x, x_stride, e, d) ||
        rows_clash(sum, sum_stride, r, residual, residual_stride, r, d))
        return FFT_ERR_INVALID_ARG;
    const NormArgs a = {x, residual, out, scale, sum, d->weight, x_stride, residual_stride,
                        out_stride, sum_stride, d->rows, (int)d->columns, d->param_dtype == FFT_F32,
                        aligned_to(d->weight, 16), (int)d->group, (float)d->columns, d->eps};
    cudaStream_t s = (cudaStream_t)stream;
    const bool r32 = d->res_dtype == FFT_F32;
    cudaError_t e2;
    if (d->dtype == FFT_F32)
        e2 = norm_fwd<float, float>(*d, a, s);
    else if (d->dtype == FFT_BF16)
        e2 = r32 ? norm_fwd<__nv_bfloat16, float>(*d, a, s)
                 : norm_fwd<__nv_bfloat16, __nv_bfloat16>(*d, a, s);
    else
        e2 = r32 ? norm_fwd<__half, float>(*d, a, s) : norm_fwd<__half, __half>(*d, a, s);
    return e2 == cudaSuccess ? FFT_OK : FFT_ERR_CUDA;
}

extern "C" int fft_norm_workspace(const fft_norm_desc* d, size_t* bytes) {
    if (!bytes) return FFT_ERR_INVALID_ARG;
    const int rc = norm_sizes(d);
    if (rc != FFT_OK) return rc;
    *bytes = (size_t)(bwd_blocks(d->rows, d->columns) * d->columns) * sizeof(float);
    return FFT_OK;
}

extern "C" int fft_norm_backward(const fft_norm_desc* d, const void* dout, int64_t dout_stride,
                                 const void* r, int64_t r_stride, const void* dresidual,
                                 int64_t dresidual_stride, void* dsum, int64_t dsum_stride,
                                 void* dx, int64_t dx_stride, float* dweight, void* workspace,
                                 size_t workspace_bytes, void* stream) {
    int rc = norm_sizes(d);
    if (rc != FFT_OK) return rc;
    const bool none = d->rows == 0;  // tensors without rows may have no address
    if ((!none && (!dout || !r || (!dsum && !dx && !dweight))) || !stride_ok(dout, dout_stride, d) ||
        !stride_ok(r, r_stride, d) || !stride_ok(dresidual, dresidual_stride, d) ||
        !stride_ok(dsum, dsum_stride, d) || !stride_ok(dx, dx_stride, d))
        return FFT_ERR_INVALID_ARG;
    const int64_t blocks = bwd_blocks(d->rows, d->columns);
    if (dweight && !none &&
        (!workspace || workspace_bytes < (size_t)(blocks * d->columns) * sizeof(float)))
        return FFT_ERR_INVALID_ARG;
    const size_t e = dtype_size(d->dtype), rs = dtype_size(d->res_dtype);
    if (!aligned_to(dout, e) || !aligned_to(dx, e) || !aligned_to(r, rs) ||
        !aligned_to(dresidual, rs) || !aligned_to(dsum, rs) || !aligned_to(dweight, 4) ||
        !aligned_to(workspace, 16) || !aligned_to(d->weight, dtype_size(d->param_dtype)))
        return FFT_ERR_MISALIGNED;
    cudaStream_t s = (cudaStream_t)stream;
    if (none) {
        if (dweight && cudaMemsetAsync(dweight, 0, (size_t)d->columns * 4, s) != cudaSuccess)
            return FFT_ERR_CUDA;
        return FFT_OK;
    }
    const NormBwdArgs a = {dout, r, dresidual, dsum, dx, d->weight,
                           dweight ? static_cast<float*>(workspace) : nullptr, dout_stride, r_stride,
                           dresidual_stride, dsum_stride, dx_stride, d->rows, (int)d->columns,
                           d->param_dtype == FFT_F32, aligned_to(d->weight, 16),
                           (float)d->columns, d->eps};
    const bool r32 = d->res_dtype == FFT_F32;
    cudaError_t e2;
    if (d->dtype == FFT_F32)
        e2 = norm_bwd<float, float>(a, blocks, s);
    else if (d->dtype == FFT_BF16)
        e2 = r32 ? norm_bwd<__nv_bfloat16, float>(a, blocks, s)
                 : norm_bwd<__nv_bfloat16, __nv_bfloat16>(a, blocks, s);
    else
        e2 = r32 ? norm_bwd<__half, float>(a, blocks, s) : norm_bwd<__half, __half>(a, blocks, s);
    if (e2 == cudaSuccess && dweight)
        e2 = run_sum_parts(a.parts, blocks, d->columns, d->columns, dweight, d->columns, 1, s);
    return e2 == cudaSuccess ? FFT_OK : FFT_ERR_CUDA;
}
