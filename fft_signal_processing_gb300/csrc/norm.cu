// Root-mean-square norm with the residual's addition (fft_norm_forward, fft_norm_backward):
//   r = x + residual;  y = r * rstd * weight,  rstd = 1 / sqrt(mean(r^2) + eps)
// in the inputs' type or in e4m3 with one scale per row or group of columns, and its gradient
//   dr = rstd (w dy) - r rstd^3 mean(w dy r) + dresidual,  dweight = sum_rows dy r rstd.
// A dozen operations per element: bound by HBM.  Each row is read once into registers (up to 16
// values per thread), reduced across its threads, and written once.
#include <cuda_fp8.h>
#include <float.h>

#include "seq_common.cuh"

namespace gbfft {
namespace {

constexpr int kMaxWarps = 32;

struct NormArgs {
    const void* x;
    const void* residual;  // may be null
    void* out;
    float* scale;
    void* sum;  // may be null
    const void* weight;
    int64_t x_stride, residual_stride, out_stride, sum_stride;
    int64_t rows, columns;
    int wf32, group;
    float eps;
};

// Sum over the tpr threads (whole warps) that share a row; `red` is double buffered by the caller.
__device__ __forceinline__ float row_sum(float v, float* red, int warp0, int warps) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.f;
    for (int w = 0; w < warps; ++w) v += red[warp0 + w];
    return v;
}
// Largest bit pattern of |v| over a row: ordered like the values, with NaN above infinity.
__device__ __forceinline__ unsigned row_max(unsigned v, unsigned* red, int warp0, int warps) {
    v = __reduce_max_sync(0xffffffffu, v);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0;
    for (int w = 0; w < warps; ++w) v = max(v, red[warp0 + w]);
    return v;
}
__device__ __forceinline__ unsigned abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// 448 / m, held finite for tiny m; 0 for m = 0; NaN stays.
__device__ __forceinline__ float e4m3_inv(float m) {
    if (m == 0.f) return 0.f;
    const float inv = 448.f / m;
    return inv > FLT_MAX ? FLT_MAX : inv;
}

// Threads: tpr per row, blockDim.x / tpr rows per block; thread j of a row holds the packs
// j, j + tpr, ... (NV of VEC columns).  OUT: 0 = type T, 1 = e4m3 with one scale per row,
// 2 = e4m3 with a scale per `group` columns (32, 64 or 128).
template <class T, class R, int VEC, int NV, int OUT>
__global__ void __launch_bounds__(1024) k_norm_fwd(const NormArgs a, int tpr) {
    extern __shared__ unsigned group_max[];  // OUT 2 with VEC 1: [rows per block][groups]
    __shared__ float red[kMaxWarps];
    __shared__ unsigned redm[kMaxWarps];
    const int local = (int)threadIdx.x / tpr, j = (int)threadIdx.x - local * tpr;
    const int warp0 = local * (tpr >> 5), warps = tpr >> 5;
    const int64_t row = (int64_t)blockIdx.x * (blockDim.x / tpr) + local;
    const bool live = row < a.rows;
    const T* x = static_cast<const T*>(a.x) + row * a.x_stride;
    const R* res = static_cast<const R*>(a.residual) + row * a.residual_stride;
    float v[NV][VEC];
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int64_t c = ((int64_t)i * tpr + j) * VEC;
        if (live && c < a.columns) {
            const Pack<T, VEC> px = ld_pack<VEC>(x + c);
#pragma unroll
            for (int k = 0; k < VEC; ++k) v[i][k] = to_f(px.v[k]);
            if (a.residual) {
                const Pack<R, VEC> pr = ld_pack<VEC>(res + c);
#pragma unroll
                for (int k = 0; k < VEC; ++k) v[i][k] += to_f(pr.v[k]);
            }
        } else {
#pragma unroll
            for (int k = 0; k < VEC; ++k) v[i][k] = 0.f;
        }
#pragma unroll
        for (int k = 0; k < VEC; ++k) ss += v[i][k] * v[i][k];
    }
    ss = row_sum(ss, red, warp0, warps);
    const float rstd = rsqrtf(ss / (float)a.columns + a.eps);
    const int64_t groups = OUT == 2 ? (a.columns + a.group - 1) / a.group : 1;
    if constexpr (OUT == 2 && VEC == 1) {
        for (int i = (int)threadIdx.x; i < (int)groups * (int)(blockDim.x / tpr); i += blockDim.x)
            group_max[i] = 0;
        __syncthreads();
    }
    R* sum = static_cast<R*>(a.sum) + row * a.sum_stride;
    unsigned m = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int64_t c = ((int64_t)i * tpr + j) * VEC;
        const bool in = live && c < a.columns;
        if (in && a.sum) {
            Pack<R, VEC> p;
#pragma unroll
            for (int k = 0; k < VEC; ++k) p.v[k] = from_f<R>(v[i][k]);
            st_pack<VEC>(sum + c, p);
        }
        if (in) {
#pragma unroll
            for (int k = 0; k < VEC; ++k) {
                v[i][k] = v[i][k] * rstd * ld_param<T>(a.weight, c + k, a.wf32);
                if (OUT == 1) m = max(m, abs_bits(v[i][k]));
            }
        }
        if constexpr (OUT == 0) {
            if (in) {
                Pack<T, VEC> p;
#pragma unroll
                for (int k = 0; k < VEC; ++k) p.v[k] = from_f<T>(v[i][k]);
                st_pack<VEC>(static_cast<T*>(a.out) + row * a.out_stride + c, p);
            }
        }
        if constexpr (OUT == 2 && VEC == 1)
            if (in) atomicMax(&group_max[local * groups + c / a.group], abs_bits(v[i][0]));
    }
    if constexpr (OUT != 0) {
        if constexpr (OUT == 1) m = row_max(m, redm, warp0, warps);
        if constexpr (OUT == 2 && VEC == 1) __syncthreads();
        uint8_t* out = static_cast<uint8_t*>(a.out) + row * a.out_stride;
        if (OUT == 1 && live && j == 0) a.scale[row] = __uint_as_float(m) / 448.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int64_t c = ((int64_t)i * tpr + j) * VEC;
            const bool in = live && c < a.columns;
            if constexpr (OUT == 2) {
                if constexpr (VEC == 1) {
                    m = in ? group_max[local * groups + c / a.group] : 0;
                } else {  // the group's packs are held by neighbouring lanes
                    m = 0;
                    if (in) {
#pragma unroll
                        for (int k = 0; k < VEC; ++k) m = max(m, abs_bits(v[i][k]));
                    }
                    for (int o = a.group / VEC / 2; o; o >>= 1)
                        m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
                }
                if (in && c % a.group == 0)
                    a.scale[row * groups + c / a.group] = __uint_as_float(m) / 448.f;
            }
            if (!in) continue;
            const float inv = e4m3_inv(__uint_as_float(m));
            if constexpr (VEC == 1) {
                out[c] = __nv_cvt_float_to_fp8(v[i][0] * inv, __NV_SATFINITE, __NV_E4M3);
            } else {
                Pack<uint16_t, VEC / 2> p;
#pragma unroll
                for (int k = 0; k < VEC; k += 2)
                    p.v[k / 2] = __nv_cvt_float2_to_fp8x2(
                        make_float2(v[i][k] * inv, v[i][k + 1] * inv), __NV_SATFINITE, __NV_E4M3);
                st_pack<VEC / 2>(reinterpret_cast<uint16_t*>(out + c), p);
            }
        }
    }
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
    int64_t rows, columns;
    int wf32;
    float eps;
};

// One row per block at a time, rows blockIdx.x, + gridDim.x, ...: every thread keeps its columns,
// so dweight is summed in registers and leaves as one partial row per block.
template <class T, class R, int VEC, int NV>
__global__ void __launch_bounds__(1024) k_norm_bwd(const NormBwdArgs a) {
    __shared__ float red[2][2 * kMaxWarps];
    const int j = (int)threadIdx.x, tpr = (int)blockDim.x, warps = tpr >> 5;
    float dw[NV][VEC] = {};
    int buf = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const T* dout = static_cast<const T*>(a.dout) + row * a.dout_stride;
        const R* rr = static_cast<const R*>(a.r) + row * a.r_stride;
        const R* dres = static_cast<const R*>(a.dres) + row * a.dres_stride;
        float r[NV][VEC], g[NV][VEC];
        float ss = 0.f, sg = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int64_t c = ((int64_t)i * tpr + j) * VEC;
            if (c < a.columns) {
                const Pack<R, VEC> pr = ld_pack<VEC>(rr + c);
                const Pack<T, VEC> pg = ld_pack<VEC>(dout + c);
#pragma unroll
                for (int k = 0; k < VEC; ++k) {
                    r[i][k] = to_f(pr.v[k]);
                    g[i][k] = to_f(pg.v[k]);
                    ss += r[i][k] * r[i][k];
                    sg += r[i][k] * (g[i][k] * ld_param<T>(a.weight, c + k, a.wf32));
                }
            }
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            ss += __shfl_xor_sync(0xffffffffu, ss, o);
            sg += __shfl_xor_sync(0xffffffffu, sg, o);
        }
        if ((j & 31) == 0) {
            red[buf][j >> 5] = ss;
            red[buf][kMaxWarps + (j >> 5)] = sg;
        }
        __syncthreads();  // the other buffer is written before the next one
        ss = sg = 0.f;
        for (int w = 0; w < warps; ++w) {
            ss += red[buf][w];
            sg += red[buf][kMaxWarps + w];
        }
        buf ^= 1;
        const float rstd = rsqrtf(ss / (float)a.columns + a.eps);
        const float back = rstd * rstd * rstd * (sg / (float)a.columns);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int64_t c = ((int64_t)i * tpr + j) * VEC;
            if (c < a.columns) {
                Pack<R, VEC> ps, pd;
                Pack<T, VEC> px;
                if (a.dres) pd = ld_pack<VEC>(dres + c);
#pragma unroll
                for (int k = 0; k < VEC; ++k) {
                    dw[i][k] += g[i][k] * r[i][k] * rstd;
                    float d = rstd * (g[i][k] * ld_param<T>(a.weight, c + k, a.wf32)) -
                              r[i][k] * back;
                    if (a.dres) d += to_f(pd.v[k]);
                    ps.v[k] = from_f<R>(d);
                    px.v[k] = from_f<T>(d);
                }
                if (a.dsum) st_pack<VEC>(static_cast<R*>(a.dsum) + row * a.dsum_stride + c, ps);
                if (a.dx) st_pack<VEC>(static_cast<T*>(a.dx) + row * a.dx_stride + c, px);
            }
        }
    }
    if (a.parts) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int64_t c = ((int64_t)i * tpr + j) * VEC;
            if (c < a.columns) {
#pragma unroll
                for (int k = 0; k < VEC; ++k)
                    a.parts[(int64_t)blockIdx.x * a.columns + c + k] = dw[i][k];
            }
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

// Values per thread: 8 (one pack of 16-bit values, two of 32-bit ones) keeps the most rows in
// flight; rows above 8192 columns need 16 to fit a block of 1024 threads.
int threads_per_row(int64_t columns, int per_thread) {
    const int64_t t = (columns + per_thread - 1) / per_thread;
    return (int)((t + 31) / 32 * 32);
}

template <class T, class R, int VEC, int NV>
cudaError_t launch_fwd(const fft_norm_desc& d, const NormArgs& a, cudaStream_t s) {
    const int tpr = threads_per_row(a.columns, VEC * NV);
    const int rpb = tpr >= 256 ? 1 : 256 / tpr;
    const unsigned grid = (unsigned)((a.rows + rpb - 1) / rpb);
    const unsigned threads = (unsigned)(rpb * tpr);
    if (d.out_dtype != FFT_E4M3)
        k_norm_fwd<T, R, VEC, NV, 0><<<grid, threads, 0, s>>>(a, tpr);
    else if (a.group == 0)
        k_norm_fwd<T, R, VEC, NV, 1><<<grid, threads, 0, s>>>(a, tpr);
    else
        k_norm_fwd<T, R, VEC, NV, 2><<<grid, threads,
            VEC == 1 ? rpb * ((a.columns + a.group - 1) / a.group) * sizeof(unsigned) : 0, s>>>(a, tpr);
    return cudaGetLastError();
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
    if (!vec) return a.columns <= 8192 ? launch_fwd<T, R, 1, 8>(d, a, s) : launch_fwd<T, R, 1, 16>(d, a, s);
    if (a.columns <= 8192) return launch_fwd<T, R, V, 8 / V>(d, a, s);
    return launch_fwd<T, R, V, 16 / V>(d, a, s);
}

template <class T, class R, int VEC, int NV>
cudaError_t launch_bwd(const NormBwdArgs& a, int64_t blocks, cudaStream_t s) {
    k_norm_bwd<T, R, VEC, NV><<<(unsigned)blocks, threads_per_row(a.columns, VEC * NV), 0, s>>>(a);
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
    if (!vec) return a.columns <= 8192 ? launch_bwd<T, R, 1, 8>(a, blocks, s) : launch_bwd<T, R, 1, 16>(a, blocks, s);
    if (a.columns <= 8192) return launch_bwd<T, R, V, 8 / V>(a, blocks, s);
    return launch_bwd<T, R, V, 16 / V>(a, blocks, s);
}

// Blocks of the backward pass: as many rows in flight as the SMs hold (blocks of up to 1024
// threads at two 1024-thread blocks per SM), and no more partial rows than that.
int64_t bwd_blocks(int64_t rows, int64_t columns) {
    const int t = threads_per_row(columns, columns <= 8192 ? 8 : 16);
    const int64_t cap = (int64_t)num_sms() * (t >= 1024 ? 2 : 2048 / t);
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
    if (q ? (!scale || (d->group != 0 && d->group != 32 && d->group != 64 && d->group != 128))
          : d->group != 0)
        return FFT_ERR_INVALID_ARG;
    if (!x || !out || !stride_ok(x, x_stride, d) || !stride_ok(residual, residual_stride, d) ||
        !stride_ok(out, out_stride, d) || !stride_ok(sum, sum_stride, d))
        return FFT_ERR_INVALID_ARG;
    const size_t e = dtype_size(d->dtype), r = dtype_size(d->res_dtype);
    if (!aligned_to(x, e) || !aligned_to(residual, r) || !aligned_to(sum, r) ||
        !aligned_to(out, dtype_size(d->out_dtype)) || !aligned_to(scale, 4) ||
        !aligned_to(d->weight, dtype_size(d->param_dtype)))
        return FFT_ERR_MISALIGNED;
    if (d->rows == 0) return FFT_OK;
    const NormArgs a = {x, residual, out, scale, sum, d->weight, x_stride, residual_stride,
                        out_stride, sum_stride, d->rows, d->columns, d->param_dtype == FFT_F32,
                        (int)d->group, d->eps};
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
    if (!dout || !r || (!dsum && !dx && !dweight) || !stride_ok(dout, dout_stride, d) ||
        !stride_ok(r, r_stride, d) || !stride_ok(dresidual, dresidual_stride, d) ||
        !stride_ok(dsum, dsum_stride, d) || !stride_ok(dx, dx_stride, d))
        return FFT_ERR_INVALID_ARG;
    const int64_t blocks = bwd_blocks(d->rows, d->columns);
    if (dweight && d->rows > 0 &&
        (!workspace || workspace_bytes < (size_t)(blocks * d->columns) * sizeof(float)))
        return FFT_ERR_INVALID_ARG;
    const size_t e = dtype_size(d->dtype), rs = dtype_size(d->res_dtype);
    if (!aligned_to(dout, e) || !aligned_to(dx, e) || !aligned_to(r, rs) ||
        !aligned_to(dresidual, rs) || !aligned_to(dsum, rs) || !aligned_to(dweight, 4) ||
        !aligned_to(workspace, 16) || !aligned_to(d->weight, dtype_size(d->param_dtype)))
        return FFT_ERR_MISALIGNED;
    cudaStream_t s = (cudaStream_t)stream;
    if (d->rows == 0) {
        if (dweight && cudaMemsetAsync(dweight, 0, (size_t)d->columns * 4, s) != cudaSuccess)
            return FFT_ERR_CUDA;
        return FFT_OK;
    }
    const NormBwdArgs a = {dout, r, dresidual, dsum, dx, d->weight,
                           dweight ? static_cast<float*>(workspace) : nullptr, dout_stride, r_stride,
                           dresidual_stride, dsum_stride, dx_stride, d->rows, d->columns,
                           d->param_dtype == FFT_F32, d->eps};
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
