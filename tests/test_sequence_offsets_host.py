"""Offsets of packed sequences are device data that no host check sees.  Whatever stands there, the
scan's kernels may touch only the row's own tokens: their walk over the tiles of a chunk, with the
functions of csrc/seq_common.cuh that they call, compiled for the host and followed here (no GPU
needed)."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

WALK = r"""
#include <stdio.h>
#include <stdlib.h>
#include <vector>
#include "seq_common.cuh"
using namespace gbfft;
// length, chunk, tile, nseq, offsets ...: the tokens that are stored, in order
int main(int argc, char** argv) {
    const int64_t length = atoll(argv[1]), chunk = atoll(argv[2]), tile = atoll(argv[3]);
    const int64_t nseq = atoll(argv[4]);
    std::vector<int64_t> o;
    for (int i = 5; i < argc; ++i) o.push_back(atoll(argv[i]));
    const int64_t* offsets = o.data();
    int goes_on = 0;
    for (int64_t t0 = 0; t0 < length; t0 += chunk) {
        const int64_t t1 = t0 + chunk < length ? t0 + chunk : length, len = t1 - t0;
        int64_t below = 0;  // as warp_count_le counts on ascending values
        while (below <= nseq && offsets[below] <= t0) ++below;
        SeqAt sq = seq_span(offsets, nseq, below - 1);
        if (!starts_at(sq, t0)) {  // the chunk goes on from the state that the one before left
            if (t0 == 0) return 3;
            ++goes_on;
        }
        int stop = seq_stop(sq, t0, (int)len);
        for (int64_t t = 0; t < len; t += tile) {
            const int64_t at = t0 + t;
            if (sq.q < 0 || sq.q >= nseq) return 2;
            if (t + tile < stop) {
                for (int64_t j = 0; j < tile; ++j) printf("%lld ", (long long)(at + j));
                continue;
            }
            const int64_t tl = len - t < tile ? len - t : tile;
            int64_t j = 0;
            while (j < tl) {
                if (at + j >= sq.end) {
                    seq_next(offsets, nseq, at + j, &sq);
                    stop = seq_stop(sq, t0, (int)len);
                }
                if (sq.q < 0 || sq.q >= nseq) return 2;
                const int64_t je = sq.end > at + j && sq.end < at + tl ? sq.end - at : tl;
                for (; j < je; ++j) printf("%lld ", (long long)(at + j));
            }
        }
    }
    fprintf(stderr, "%d", goes_on);
    return 0;
}
"""


@pytest.fixture(scope="module")
def walk(tmp_path_factory):
    from fft_signal_processing_gb300 import _build

    at = tmp_path_factory.mktemp("walk")
    src, exe = at / "walk.cu", at / "walk"
    src.write_text(WALK)
    subprocess.run([_build.nvcc(), *_build.ARCH, "-std=c++17", "-I", os.path.join(ROOT, "include"),
                    "-I", _build.CSRC, str(src), "-o", str(exe)], check=True)

    def run(length, chunk, tile, offsets):
        r = subprocess.run([str(exe), *map(str, (length, chunk, tile, len(offsets) - 1, *offsets))],
                           capture_output=True, text=True)
        assert r.returncode == 0
        return [int(v) for v in r.stdout.split()], int(r.stderr)

    return run


OFFSETS = [
    (36, [0, 36]), (36, [0, 5, 5, 36]), (200, [0, 1, 130, 200]),  # as they should be
    (36, [0, 41]), (36, [0, 1000]), (36, [0, 10, 52]), (36, [0, 1 << 40]), (200, [0, 64, 207]),
    (36, [0, 20]), (36, [0, 0]), (36, [7, 36]), (36, [40, 50]), (36, [-9, 36]), (36, [-9, -3, 60]),
    (200, [0, 150, 80, 200]), (200, [0, 300, 80, 200]), (200, [0, 300, 80, 90])]


@pytest.mark.parametrize("length,offsets", OFFSETS, ids=str)
@pytest.mark.parametrize("chunk", [64, 1000])
@pytest.mark.parametrize("tile", [8, 16])
def test_every_token_of_the_row_and_none_beyond(walk, length, offsets, chunk, tile):
    tokens, _ = walk(length, chunk, tile, offsets)
    assert tokens == list(range(length))


@pytest.mark.parametrize("length,offsets", OFFSETS, ids=str)
def test_a_row_that_is_not_cut_reads_no_chunk_state(walk, length, offsets):
    """There is none then: also not where no sequence holds the first token."""
    assert walk(length, 1000, 8, offsets)[1] == 0


def test_chunks_go_on_inside_sequences(walk):
    assert walk(200, 64, 8, [0, 200])[1] == 3
    assert walk(200, 64, 8, [0, 64, 128, 192, 200])[1] == 0
    assert walk(200, 64, 8, [0, 65, 128, 200])[1] == 2
