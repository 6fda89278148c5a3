// Outputs over inputs: whether the rows of two sequence tensors share values (host only).
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "../../include/gbfft.h"

namespace gbfft {

// Bytes that a sequence tensor's rows of `width` values may touch, from its first value on.
inline int64_t seq_span_bytes(const fft_seq& s, int64_t width, int64_t nseq, int64_t length,
                              bool packed, size_t size) {
    if (!s.data || length < 1) return 0;
    return ((packed ? 0 : (nseq - 1) * s.seq_stride) + (length - 1) * s.tok_stride + width) *
           (int64_t)size;
}
inline bool bytes_meet(const void* a, int64_t na, const void* b, int64_t nb) {
    const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
    return a && b && na > 0 && nb > 0 && x < y + nb && y < x + na;
}
// Whether two sequence tensors share values.  Spans may meet without that, as those of two halves of
// one projection do: every row of both starts a multiple of the strides' common divisor after the
// first one of its tensor, so the columns modulo it tell them apart.  Where the strides are the same,
// as those of two ranges of tokens of one buffer, rows of one tensor and the other are compared by
// how many sequences and tokens they lie apart.  Other tensors whose spans meet count as sharing.
inline bool seqs_meet(const fft_seq& a, const fft_seq& b, int64_t width, int64_t bwidth, int64_t nseq,
                      int64_t length, bool packed, size_t size) {
    if (!bytes_meet(a.data, seq_span_bytes(a, width, nseq, length, packed, size), b.data,
                    seq_span_bytes(b, bwidth, nseq, length, packed, size)))
        return false;
    const int64_t seqs = packed ? 1 : nseq;
    const int64_t apart = ((intptr_t)b.data - (intptr_t)a.data) / (int64_t)size;
    int64_t period = 0;
    auto add = [&](int64_t stride) {
        while (stride) {
            const int64_t r = period % stride;
            period = stride;
            stride = r;
        }
    };
    if (length > 1) add(a.tok_stride), add(b.tok_stride);
    if (seqs > 1) add(a.seq_stride), add(b.seq_stride);
    if (!period) return true;
    const int64_t column = (apart % period + period) % period;  // of b's rows, a's being 0
    if (column >= width && column + bwidth <= period) return false;
    const int64_t tok = length > 1 ? a.tok_stride : 0, seq = seqs > 1 ? a.seq_stride : 0;
    if ((length > 1 && b.tok_stride != tok) || (seqs > 1 && b.seq_stride != seq)) return true;
    auto floor_div = [](int64_t x, int64_t y) { return x / y - (x % y < 0 ? 1 : 0); };
    for (int64_t i = 0; i < 2 * seqs - 1; ++i) {  // 0, 1, -1, 2, ... sequences apart
        const int64_t at = apart + (i & 1 ? (i + 1) / 2 : -(i / 2)) * seq;
        // some t in (-length, length) with -bwidth < at + t * tok < width
        if (!tok) {
            if (at > -bwidth && at < width) return true;
            continue;
        }
        int64_t first = floor_div(-bwidth - at, tok) + 1, last = floor_div(width - 1 - at, tok);
        if (first < 1 - length) first = 1 - length;
        if (last > length - 1) last = length - 1;
        if (first <= last) return true;
    }
    return false;
}
inline bool seqs_same(const fft_seq& a, const fft_seq& b, int64_t nseq, int64_t length, bool packed) {
    return a.data == b.data && (length < 2 || a.tok_stride == b.tok_stride) &&
           (packed || nseq < 2 || a.seq_stride == b.seq_stride);
}

}  // namespace gbfft
