// C entry points of the short causal convolution and the selective scan: checks on the host,
// workspace layout, and the choice of the per-type launcher.  Declared in include/gbfft.h.
#include "conv.h"
#include "scan.h"
#include "scan_bwd.h"
#include "seq_overlap.h"
#include "seq_step.h"

using namespace gbfft;

namespace {

constexpr int64_t kMaxElements = INT64_C(1) << 58;  // offsets stay in 64 bits
constexpr int64_t kMaxTokStride = INT64_C(1) << 26;  // 16 tokens stay in 32 bits

int status(cudaError_t e) {
    return e == cudaSuccess ? FFT_OK
                            : (e == cudaErrorInvalidValue ? FFT_ERR_UNSUPPORTED_SIZE : FFT_ERR_CUDA);
}

// A sequence tensor whose rows hold `width` values.
int check_seq(const fft_seq& s, int64_t width, int64_t nseq, int64_t length, bool packed,
              size_t size, bool output) {
    if (!s.data) return length == 0 ? FFT_OK : FFT_ERR_INVALID_ARG;
    if (s.tok_stride < 0 || s.seq_stride < 0) return FFT_ERR_INVALID_ARG;
    if (output && length > 1 && s.tok_stride < width) return FFT_ERR_INVALID_ARG;
    if (output && !packed && nseq > 1 && length > 0 && s.seq_stride < width) return FFT_ERR_INVALID_ARG;
    if (s.tok_stride > kMaxTokStride ||
        (!packed && s.seq_stride > kMaxElements / (nseq + 1)))
        return FFT_ERR_UNSUPPORTED_SIZE;
    return aligned_to(s.data, size) ? FFT_OK : FFT_ERR_MISALIGNED;
}
int check_sizes(int64_t nseq, int64_t length, int64_t channels, const int64_t* offsets) {
    if (nseq < 1 || length < 0 || channels < 1) return FFT_ERR_INVALID_ARG;
    if (nseq > INT32_MAX || length > INT32_MAX - 65536 || channels > INT32_MAX / 256)
        return FFT_ERR_UNSUPPORTED_SIZE;
    return aligned_to(offsets, 8) ? FFT_OK : FFT_ERR_MISALIGNED;
}

#define TRY(x)                        \
    do {                              \
        const int rc_ = (x);          \
        if (rc_ != FFT_OK) return rc_; \
    } while (0)

int check_conv(const fft_conv_desc* d, bool pointers) {
    if (!d || d->dtype < FFT_F32 || d->dtype > FFT_F16 || (d->silu != 0 && d->silu != 1) ||
        (d->param_dtype != FFT_F32 && d->param_dtype != d->dtype))
        return FFT_ERR_INVALID_ARG;
    if (d->width < 1) return FFT_ERR_INVALID_ARG;
    if (d->width > FFT_CONV_MAX_WIDTH) return FFT_ERR_UNSUPPORTED_SIZE;
    TRY(check_sizes(d->nseq, d->length, d->channels, d->offsets));
    if (!pointers) return FFT_OK;
    if (!d->weight) return FFT_ERR_INVALID_ARG;
    const size_t e = dtype_size(d->dtype), p = dtype_size(d->param_dtype);
    if (!aligned_to(d->weight, p) || !aligned_to(d->bias, p) || !aligned_to(d->initial_state, e))
        return FFT_ERR_MISALIGNED;
    return check_seq(d->x, d->channels, d->nseq, d->length, d->offsets, e, false);
}

int64_t conv_tiles(const fft_conv_desc& d) {
    const int64_t tile = kConvRuns * conv_run_tokens(d, true);
    return (d.offsets ? 1 : d.nseq) * ((d.length + tile - 1) / tile);
}

int check_scan(const fft_scan_desc* d, bool pointers) {
    if (!d || d->dtype < FFT_F32 || d->dtype > FFT_F16 || (d->softplus != 0 && d->softplus != 1))
        return FFT_ERR_INVALID_ARG;
    TRY(check_sizes(d->nseq, d->length, d->channels, d->offsets));
    if (d->groups < 1 || d->channels % d->groups || d->states < 1) return FFT_ERR_INVALID_ARG;
    if (d->states > FFT_SCAN_MAX_STATES) return FFT_ERR_UNSUPPORTED_SIZE;
    if (!pointers) return FFT_OK;
    if (!d->A) return FFT_ERR_INVALID_ARG;
    if (!aligned_to(d->A, 4) || !aligned_to(d->D, 4) || !aligned_to(d->delta_bias, 4) ||
        !aligned_to(d->initial_state, 4))
        return FFT_ERR_MISALIGNED;
    const size_t e = dtype_size(d->dtype);
    const int64_t bc = d->groups * d->states;
    TRY(check_seq(d->u, d->channels, d->nseq, d->length, d->offsets, e, false));
    TRY(check_seq(d->delta, d->channels, d->nseq, d->length, d->offsets, e, false));
    TRY(check_seq(d->B, bc, d->nseq, d->length, d->offsets, e, false));
    TRY(check_seq(d->C, bc, d->nseq, d->length, d->offsets, e, false));
    if (d->z.data) TRY(check_seq(d->z, d->channels, d->nseq, d->length, d->offsets, e, false));
    return FFT_OK;
}

int64_t up16(int64_t bytes) { return (bytes + 15) / 16 * 16; }

// Forward plan and workspace: carry, dsum, reset.
int64_t scan_layout(const fft_scan_desc& d, ScanArgs* a, char* w) {
    ScanArgs b = {};
    if (a) b = *a;
    b.d = d;
    scan_plan(&b);
    int64_t at = 0;
    auto take = [&](int64_t bytes) {
        char* p = w ? w + at : nullptr;
        at += up16(bytes);
        return p;
    };
    if (b.nchunks > 1) {
        const int64_t ch = b.rows * b.nchunks;
        b.carry = reinterpret_cast<float*>(take(ch * d.channels * scan_out_np(d.states) * 4));
        b.dsum = reinterpret_cast<float*>(take(ch * d.channels * 4));
        b.reset = reinterpret_cast<int*>(take(ch * 4));
    }
    if (a) *a = b;
    return at;
}

}  // namespace

namespace gbfft {

void scan_plan(ScanArgs* a) {
    const fft_scan_desc& d = a->d;
    const int np = scan_np(d.states);
    const int64_t dg = d.channels / d.groups;
    a->rows = d.offsets ? 1 : d.nseq;
    auto blocks = [&](int sl) {
        const int ct = scan_channels(sl);
        return a->rows * d.groups * ((dg + ct - 1) / ct);
    };
    a->sl = scan_lanes(np);
    // Uncut with two lanes per channel where that alone gives every SM four blocks or more, else k_scan
    // with time cut into as many chunks as give every SM about six blocks.  Measured, bfloat16, 16
    // states, gated, 2048 tokens, by the SM's blocks of two lanes (us: two lanes uncut / k_scan at its
    // best cut): 3.4 (4 x 4096 channels) 262 / 265, 4.2 (5 x 4096) 325 / 355, 5.1 327 / 373, 6.7 406 /
    // 475; k_scan uncut takes 375 to 379 at all of these, so it is the faster one at 6.7, and with 8
    // states (265 / 235 at 4.2, 313 / 265 at 6.7) the rule is not the best.  Blocks of k_scan to an SM,
    // 2 / 3 / 4 / 5 / 6 / 7 / 8: one sequence of 16384 x 2048 287 326 250 295 250 293 262; 4 of 4096 x
    // 2048 377 327 297 295 262 293 262; 3 of 5000 x 2000 286 289 287 272 241 276 247; one of 4096 x
    // 2048 94 106 87 103 98 106 106.
    const int64_t sms = num_sms();
    int64_t k = 1;
    if ((np == 8 || np == 16) && scan_out_np(d.states) != 12 && blocks(2) >= sms * 4)
        a->sl = 2;
    else
        k = (sms * 6 + blocks(a->sl) / 2) / blocks(a->sl);
    a->ctiles = blocks(a->sl) / (a->rows * d.groups);
    a->chunk = d.length;
    if (k > 1) {
        a->chunk = (d.length + k - 1) / k;
        a->chunk = (a->chunk + 15) / 16 * 16;
    }
    if (a->chunk < 64) a->chunk = 64;
    a->nchunks = (d.length + a->chunk - 1) / a->chunk;
}

int64_t scan_bwd_layout(const fft_scan_desc& d, ScanBwdArgs* a, char* w) {
    const int64_t n = d.states, np = scan_np(n), sl = bwd_sl(n), ct = bwd_channels((int)sl);
    const int64_t dg = d.channels / d.groups, rows = d.offsets ? 1 : d.nseq;
    const int64_t ctiles = (dg + ct - 1) / ct;
    // Chunks: the main kernel holds two blocks on an SM, so the time goes with the rounds of blocks
    // times the tokens of a chunk (and about 16 tokens' time to start a block); the fewest chunks
    // of the best.  Four rows of 2048 tokens and 2048 channels: nine chunks of 240 tokens.
    const int64_t blocks = rows * ctiles * d.groups, resident = (int64_t)num_sms() * 2;
    int64_t chunk = 64, best = INT64_MAX;
    for (int64_t k = 1; k <= 256; ++k) {
        int64_t size = (d.length + k - 1) / k;
        size = (size + 15) / 16 * 16;
        if (size < 64) size = 64;
        const int64_t n = (d.length + size - 1) / size;
        const int64_t cost = (blocks * n + resident - 1) / resident * (size + 16);
        if (cost < best) {
            best = cost;
            chunk = size;
        }
        if (size == 64) break;
    }
    const int64_t nchunks = (d.length + chunk - 1) / chunk;
    const int64_t state_tiles = (d.length + kScanTile - 1) / kScanTile;
    int64_t at = 0;
    auto take = [&](int64_t floats) {
        float* p = reinterpret_cast<float*>(w ? w + at : nullptr);
        at += up16(floats * 4);
        return p;
    };
    const int64_t per = d.channels * np, parts = rows * nchunks;
    const int64_t cuts = (chunk + kScanPart - 1) / kScanPart;
    const int64_t last = d.length - (nchunks - 1) * chunk;  // tokens of a row's last chunk
    ScanBwdArgs b = {};
    if (a) b = *a;
    b.ctiles = ctiles;
    b.f.d = d;
    b.f.rows = rows;
    b.f.chunk = chunk;
    b.f.nchunks = nchunks;
    b.f.sl = scan_lanes((int)np);
    const int64_t fct = scan_channels(b.f.sl);
    b.f.ctiles = (dg + fct - 1) / fct;
    const int64_t bct = np <= 16 ? kScanThreads : kScanThreads * 16 / np;
    b.back_ctiles = (dg + bct - 1) / bct;
    if (nchunks > 1) {
        b.f.carry = take(parts * per);
        b.f.dsum = take(parts * d.channels);
        b.f.reset = reinterpret_cast<int*>(take(parts));
        b.carry = take(parts * per);
    }
    b.f.tiles = take(rows * state_tiles * per);
    b.bc = take(ctiles * rows * d.length * d.groups * 2 * n);
    b.cuts = cuts;
    b.parts = nchunks ? (nchunks - 1) * cuts + (last + kScanPart - 1) / kScanPart : 0;
    b.pA = take(rows * b.parts * d.channels * n);
    b.pD = take(rows * b.parts * d.channels);
    b.pbias = take(rows * b.parts * d.channels);
    if (a) *a = b;
    return at;
}

}  // namespace gbfft

extern "C" int fft_conv_forward(const fft_conv_desc* d, const fft_seq* out, void* final_state,
                                void* stream) {
    TRY(check_conv(d, true));
    if (!out) return FFT_ERR_INVALID_ARG;
    const size_t e = dtype_size(d->dtype);
    TRY(check_seq(*out, d->channels, d->nseq, d->length, d->offsets, e, true));
    if (!aligned_to(final_state, e)) return FFT_ERR_MISALIGNED;
    const int64_t states = d->nseq * (d->width - 1) * d->channels * (int64_t)e;
    if (seqs_meet(*out, d->x, d->channels, d->channels, d->nseq, d->length, d->offsets, e) ||
        bytes_meet(final_state, states, d->initial_state, states))
        return FFT_ERR_INVALID_ARG;
    ConvArgs a = {};
    a.d = *d;
    a.out = *out;
    a.final_state = final_state;
    cudaStream_t s = (cudaStream_t)stream;
    return status(d->dtype == FFT_F32 ? conv_forward_f32(a, s)
                                      : (d->dtype == FFT_BF16 ? conv_forward_bf16(a, s)
                                                              : conv_forward_f16(a, s)));
}

extern "C" int fft_conv_workspace(const fft_conv_desc* d, size_t* bytes) {
    if (!bytes) return FFT_ERR_INVALID_ARG;
    TRY(check_conv(d, false));
    *bytes = (size_t)(conv_tiles(*d) * (d->width + 1) * d->channels) * sizeof(float);
    return FFT_OK;
}

extern "C" int fft_conv_backward(const fft_conv_desc* d, const fft_seq* dout,
                                 const void* dfinal_state, const fft_seq* dx, float* dweight,
                                 float* dbias, void* dinitial_state, void* workspace,
                                 size_t workspace_bytes, void* stream) {
    TRY(check_conv(d, true));
    if (!dout || !dx) return FFT_ERR_INVALID_ARG;
    const size_t e = dtype_size(d->dtype);
    TRY(check_seq(*dout, d->channels, d->nseq, d->length, d->offsets, e, false));
    if (dx->data) TRY(check_seq(*dx, d->channels, d->nseq, d->length, d->offsets, e, true));
    if (!aligned_to(dfinal_state, e) || !aligned_to(dinitial_state, e) || !aligned_to(dweight, 4) ||
        !aligned_to(dbias, 4) || !aligned_to(workspace, 16))
        return FFT_ERR_MISALIGNED;
    const int64_t tiles = conv_tiles(*d), cols = (d->width + 1) * d->channels;
    const bool params = dweight || dbias;
    if (params && tiles > 0 &&
        (!workspace || workspace_bytes < (size_t)(tiles * cols) * sizeof(float)))
        return FFT_ERR_INVALID_ARG;
    const int64_t states = d->nseq * (d->width - 1) * d->channels * (int64_t)e;
    auto meets = [&](const fft_seq& in) {
        return seqs_meet(*dx, in, d->channels, d->channels, d->nseq, d->length, d->offsets, e);
    };
    if (meets(d->x) || meets(*dout) || bytes_meet(dinitial_state, states, d->initial_state, states) ||
        bytes_meet(dinitial_state, states, dfinal_state, states))
        return FFT_ERR_INVALID_ARG;
    ConvArgs a = {};
    a.d = *d;
    a.out = *dx;
    a.dout = *dout;
    a.final_state = const_cast<void*>(dfinal_state);
    a.dinitial = dinitial_state;
    a.parts = params && tiles > 0 ? static_cast<float*>(workspace) : nullptr;
    cudaStream_t s = (cudaStream_t)stream;
    cudaError_t r = d->dtype == FFT_F32 ? conv_backward_f32(a, s)
                                        : (d->dtype == FFT_BF16 ? conv_backward_bf16(a, s)
                                                                : conv_backward_f16(a, s));
    // partial rows are [tiles][width + 1][channels], the bias behind the taps
    if (r == cudaSuccess && dweight)
        r = run_sum_parts(a.parts, tiles, cols, d->width * d->channels, dweight, d->channels,
                          d->width, s);
    if (r == cudaSuccess && dbias)
        r = run_sum_parts(a.parts ? a.parts + d->width * d->channels : nullptr, tiles, cols,
                          d->channels, dbias, d->channels, 1, s);
    return status(r);
}

static int check_step(const fft_seq* out, const void* state, int64_t pool, const int64_t* slots,
                      const int64_t* slots_out, int64_t nseq, int64_t length,
                      const int64_t* offsets, int64_t channels, size_t e, bool needs_state) {
    if (!out || length != 1 || offsets || pool < 0) return FFT_ERR_INVALID_ARG;
    if (needs_state && pool > 0 && !state) return FFT_ERR_INVALID_ARG;
    if (!slots && pool < nseq) return FFT_ERR_INVALID_ARG;
    if (!aligned_to(slots, 8) || !aligned_to(slots_out, 8)) return FFT_ERR_MISALIGNED;
    return check_seq(*out, channels, nseq, 1, false, e, true);
}

extern "C" int fft_conv_step(const fft_conv_desc* d, const fft_seq* out, void* state, int64_t pool,
                             const int64_t* slots, const int64_t* slots_out, void* stream) {
    TRY(check_conv(d, true));
    const size_t e = dtype_size(d->dtype);
    TRY(check_step(out, state, pool, slots, slots_out, d->nseq, d->length, d->offsets, d->channels,
                   e, d->width > 1));
    if (!aligned_to(state, e)) return FFT_ERR_MISALIGNED;
    if (!seqs_same(*out, d->x, d->nseq, 1, false) &&
        seqs_meet(*out, d->x, d->channels, d->channels, d->nseq, 1, false, e))
        return FFT_ERR_INVALID_ARG;
    const ConvStepArgs a = {*d, *out, state, slots, slots_out, pool};
    return status(conv_step_any(a, (cudaStream_t)stream));
}

extern "C" int fft_scan_workspace(const fft_scan_desc* d, int backward, size_t* bytes) {
    if (!bytes || (backward != 0 && backward != 1)) return FFT_ERR_INVALID_ARG;
    TRY(check_scan(d, false));
    *bytes = (size_t)(backward ? scan_bwd_layout(*d, nullptr, nullptr)
                               : scan_layout(*d, nullptr, nullptr));
    return FFT_OK;
}

extern "C" int fft_scan_forward(const fft_scan_desc* d, const fft_seq* out, float* final_state,
                                void* workspace, size_t workspace_bytes, void* stream) {
    TRY(check_scan(d, true));
    if (!out) return FFT_ERR_INVALID_ARG;
    TRY(check_seq(*out, d->channels, d->nseq, d->length, d->offsets, dtype_size(d->dtype), true));
    if (!aligned_to(final_state, 4) || !aligned_to(workspace, 16)) return FFT_ERR_MISALIGNED;
    ScanArgs a = {};
    a.d = *d;
    a.out = *out;
    a.final_state = final_state;
    const int64_t need = scan_layout(*d, &a, static_cast<char*>(workspace));
    if (need > 0 && (!workspace || workspace_bytes < (size_t)need)) return FFT_ERR_INVALID_ARG;
    const int64_t states = d->nseq * d->channels * d->states * 4;
    auto meets = [&](const fft_seq& in, int64_t width) {
        return seqs_meet(*out, in, d->channels, width, d->nseq, d->length, d->offsets, dtype_size(d->dtype));
    };
    for (const fft_seq* in : {&d->u, &d->z})  // read where they are written, by the same thread
        if (!seqs_same(*out, *in, d->nseq, d->length, d->offsets) && meets(*in, d->channels))
            return FFT_ERR_INVALID_ARG;
    if (meets(d->delta, d->channels) || meets(d->B, d->groups * d->states) ||
        meets(d->C, d->groups * d->states) || bytes_meet(final_state, states, d->initial_state, states))
        return FFT_ERR_INVALID_ARG;
    cudaStream_t s = (cudaStream_t)stream;
    return status(d->dtype == FFT_F32 ? scan_forward_f32(a, s)
                                      : (d->dtype == FFT_BF16 ? scan_forward_bf16(a, s)
                                                              : scan_forward_f16(a, s)));
}

extern "C" int fft_scan_step(const fft_scan_desc* d, const fft_seq* out, float* state, int64_t pool,
                             const int64_t* slots, const int64_t* slots_out, void* stream) {
    TRY(check_scan(d, true));
    TRY(check_step(out, state, pool, slots, slots_out, d->nseq, d->length, d->offsets, d->channels,
                   dtype_size(d->dtype), true));
    if (!aligned_to(state, 4)) return FFT_ERR_MISALIGNED;
    const int64_t bc = d->groups * d->states;
    auto meets = [&](const fft_seq& in, int64_t width) {
        return seqs_meet(*out, in, d->channels, width, d->nseq, 1, false, dtype_size(d->dtype));
    };
    for (const fft_seq* in : {&d->u, &d->delta, &d->z})
        if (!seqs_same(*out, *in, d->nseq, 1, false) && meets(*in, d->channels)) return FFT_ERR_INVALID_ARG;
    if (meets(d->B, bc) || meets(d->C, bc)) return FFT_ERR_INVALID_ARG;
    const ScanStepArgs a = {*d, *out, state, slots, slots_out, pool, 0, false};
    return status(scan_step_any(a, (cudaStream_t)stream));
}

extern "C" int fft_scan_backward(const fft_scan_desc* d, const fft_scan_grads* g, void* workspace,
                                 size_t workspace_bytes, void* stream) {
    TRY(check_scan(d, true));
    if (!g || (g->dz.data != nullptr) != (d->z.data != nullptr)) return FFT_ERR_INVALID_ARG;
    const size_t e = dtype_size(d->dtype);
    const int64_t bc = d->groups * d->states;
    TRY(check_seq(g->dout, d->channels, d->nseq, d->length, d->offsets, e, false));
    TRY(check_seq(g->du, d->channels, d->nseq, d->length, d->offsets, e, true));
    TRY(check_seq(g->ddelta, d->channels, d->nseq, d->length, d->offsets, e, true));
    TRY(check_seq(g->dB, bc, d->nseq, d->length, d->offsets, e, true));
    TRY(check_seq(g->dC, bc, d->nseq, d->length, d->offsets, e, true));
    if (g->dz.data) TRY(check_seq(g->dz, d->channels, d->nseq, d->length, d->offsets, e, true));
    if (!aligned_to(g->dfinal_state, 4) || !aligned_to(g->dA, 4) || !aligned_to(g->dD, 4) ||
        !aligned_to(g->ddelta_bias, 4) || !aligned_to(g->dinitial_state, 4) ||
        !aligned_to(workspace, 16))
        return FFT_ERR_MISALIGNED;
    ScanBwdArgs a = {};
    a.d = *d;
    a.g = *g;
    const int64_t need = scan_bwd_layout(*d, &a, static_cast<char*>(workspace));
    if (need > 0 && (!workspace || workspace_bytes < (size_t)need)) return FFT_ERR_INVALID_ARG;
    cudaStream_t s = (cudaStream_t)stream;
    return status(d->dtype == FFT_F32 ? scan_backward_f32(a, s)
                                      : (d->dtype == FFT_BF16 ? scan_backward_bf16(a, s)
                                                              : scan_backward_f16(a, s)));
}
