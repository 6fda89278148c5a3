"""Workspace of the group norm's gradients (no GPU needed): rows of partial sums are left by as many
blocks as the GPU holds, not by every tile of every sequence."""
import ctypes

import pytest

import fft_signal_processing_gb300 as fx
from fft_signal_processing_gb300 import sequence as sq

A, MB = 1 << 20, 1 << 20


@pytest.fixture(scope="module")
def lib():
    from fft_signal_processing_gb300 import _build

    _build.build()
    return fx.lib()


def workspace(lib, nseq, length, channels, groups, dtype=sq.BF16, offsets=0, backward=1):
    d = sq._GNORM.pack(dtype, sq.F32, 0, 1e-5, nseq, length, channels, groups, offsets, 0, 0, 0, 0, 0, 0, 0, 0)
    size = ctypes.c_size_t()
    assert lib.fft_gnorm_workspace(d, backward, size) == fx.FFT_OK
    return size.value


@pytest.mark.parametrize("nseq,length,channels,groups,offsets", [
    (16384, 1, 4096, 4, 0), (16384, 1, 4096, 8, 0), (65536, 1, 4096, 1, 0), (8192, 2, 1024, 8, 0),
    (1 << 20, 1, 1030, 1, 0), (1, 1 << 22, 1024, 8, 0), (4096, 1 << 20, 1024, 8, A), (64, 1000, 65536, 1, 0),
    (64, 1000, 65535, 1, 0), (1000, 30, 7, 7, 0)], ids=str)
@pytest.mark.parametrize("dtype", [sq.F32, sq.BF16])
def test_does_not_grow_with_the_rows(lib, nseq, length, channels, groups, offsets, dtype):
    small = workspace(lib, nseq, length, channels, groups, dtype, offsets)
    twice = workspace(lib, 2 * nseq, length, channels, groups, dtype, offsets)
    # a sequence has two sums for every group, and three numbers for every group and tile of 16 tokens or more
    tiles = 1 if offsets else -(-length // 16)
    assert twice - small <= nseq * groups * (8 + 12 * tiles) + 64
    # what is left by blocks: two rows of their channels by eight blocks of 8 KB of values for every SM
    rows = 1 if offsets else nseq
    records = rows * -(-length // 16) + (nseq if offsets else 0)
    assert small <= groups * (8 * nseq + 12 * records) + 96 * MB


def test_long_rows_of_one_sequence(lib):
    assert workspace(lib, 1, 1 << 22, 1024, 8) <= 64 * MB
    assert workspace(lib, 65536, 1, 4096, 1) <= 64 * MB
