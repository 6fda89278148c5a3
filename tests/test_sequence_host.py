"""Host-side checks of the sequence operators (no GPU needed): descriptor layouts against the
header, refusals before anything is enqueued, and workspace sizes."""
import ctypes
import os
import subprocess

import pytest

import fft_signal_processing_gb300 as fx
from fft_signal_processing_gb300 import sequence as sq

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    from fft_signal_processing_gb300 import _build

    _build.build()
    return fx.lib()


def test_descriptors_match_the_header(tmp_path):
    src = tmp_path / "sizes.c"
    src.write_text('''#include "gbfft.h"
#include <stdio.h>
#define O(t, f) printf(" %zu", offsetof(t, f))
int main(void) {
    printf("%zu %zu %zu %zu %zu", sizeof(fft_seq), sizeof(fft_conv_desc), sizeof(fft_scan_desc),
           sizeof(fft_scan_grads), sizeof(fft_norm_desc));
    O(fft_conv_desc, offsets); O(fft_conv_desc, x); O(fft_scan_desc, A); O(fft_scan_desc, z);
    O(fft_scan_grads, du); O(fft_scan_grads, dA); O(fft_norm_desc, eps); O(fft_norm_desc, weight);
    return 0;
}''')
    exe = tmp_path / "sizes"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = [int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True).stdout.split()]
    sizes = [s.size for s in (sq._SEQ, sq._CONV, sq._SCAN, sq._GRADS, sq._NORM)]
    assert got == sizes + [40, 72, 56, 184, 32, 152, 40, 48]


A = 1 << 20  # an address that is never read: the calls under test are refused on the host


def conv(**k):
    v = dict(dtype=sq.BF16, param=sq.F32, width=4, silu=1, nseq=2, length=8, channels=16, offsets=0,
             weight=A, bias=0, initial=0, x=(A, 128, 16))
    v.update(k)
    x = v.pop("x")
    return sq._CONV.pack(*v.values(), *x)


def scan(**k):
    v = dict(dtype=sq.BF16, softplus=1, nseq=2, length=8, channels=16, groups=1, states=16, offsets=0,
             A=A, D=0, bias=0, initial=0, u=(A, 128, 16), delta=(A, 128, 16), B=(A, 128, 16),
             C=(A, 128, 16), z=(0, 0, 0))
    v.update(k)
    return sq._SCAN.pack(*list(v.values())[:12], *v["u"], *v["delta"], *v["B"], *v["C"], *v["z"])


def norm(**k):
    v = dict(dtype=sq.BF16, res=sq.F32, param=sq.F32, out=sq.BF16, rows=4, columns=64, group=0,
             eps=1e-6, weight=A)
    v.update(k)
    return sq._NORM.pack(*v.values())


OUT = sq._SEQ.pack(A, 128, 16)
INVALID, SIZE, ALIGN = fx.FFT_ERR_INVALID_ARG, fx.FFT_ERR_UNSUPPORTED_SIZE, fx.FFT_ERR_MISALIGNED


@pytest.mark.parametrize("change,status", [
    (dict(dtype=7), INVALID), (dict(dtype=sq.E4M3), INVALID), (dict(param=sq.F16), INVALID),
    (dict(width=0), INVALID), (dict(width=9), SIZE), (dict(silu=2), INVALID), (dict(nseq=0), INVALID),
    (dict(length=-1), INVALID), (dict(channels=0), INVALID), (dict(weight=0), INVALID),
    (dict(weight=A + 2), ALIGN), (dict(initial=A + 1), ALIGN), (dict(offsets=A + 4), ALIGN),
    (dict(x=(0, 128, 16)), INVALID), (dict(x=(A + 1, 128, 16)), ALIGN), (dict(x=(A, -1, 16)), INVALID),
    (dict(x=(A, 128, 1 << 27)), SIZE)], ids=str)
def test_conv_refuses(lib, change, status):
    assert lib.fft_conv_forward(conv(**change), OUT, None, None) == status
    size = ctypes.c_size_t()
    if "x" not in change and "weight" not in change and "initial" not in change:
        assert lib.fft_conv_workspace(conv(**change), size) == status


def test_conv_calls_refuse(lib):
    assert lib.fft_conv_forward(None, OUT, None, None) == INVALID
    assert lib.fft_conv_forward(conv(), None, None, None) == INVALID
    assert lib.fft_conv_forward(conv(), sq._SEQ.pack(A, 128, 8), None, None) == INVALID  # rows overlap
    assert lib.fft_conv_backward(conv(), OUT, None, OUT, A, None, None, None, 0, None) == INVALID
    assert lib.fft_conv_backward(conv(), OUT, None, OUT, A, None, None, A + 8, 1 << 20, None) == ALIGN
    one = conv(length=1)
    assert lib.fft_conv_step(conv(), OUT, A, 4, None, None, None) == INVALID  # more than one token
    assert lib.fft_conv_step(one, OUT, A, 1, None, None, None) == INVALID  # pool below the sequences
    assert lib.fft_conv_step(one, OUT, 0, 4, None, None, None) == INVALID
    assert lib.fft_conv_step(one, OUT, A + 1, 4, None, None, None) == ALIGN
    assert lib.fft_conv_step(one, OUT, A, 4, A + 4, None, None) == ALIGN


@pytest.mark.parametrize("change,status", [
    (dict(dtype=-1), INVALID), (dict(softplus=3), INVALID), (dict(groups=3), INVALID),
    (dict(groups=0), INVALID), (dict(states=0), INVALID), (dict(states=129), SIZE), (dict(A=0), INVALID),
    (dict(A=A + 2), ALIGN), (dict(D=A + 1), ALIGN), (dict(B=(0, 0, 0)), INVALID),
    (dict(z=(A + 1, 128, 16)), ALIGN), (dict(u=(A, 1 << 60, 16)), SIZE), (dict(length=1 << 31), SIZE)],
    ids=str)
def test_scan_refuses(lib, change, status):
    assert lib.fft_scan_forward(scan(**change), OUT, None, A, 1 << 40, None) == status


def test_scan_calls_refuse(lib):
    long = scan(nseq=1, length=4096)
    size = ctypes.c_size_t()
    assert lib.fft_scan_workspace(long, 0, size) == fx.FFT_OK and size.value > 0
    assert lib.fft_scan_forward(long, OUT, None, A, size.value - 1, None) == INVALID  # too small
    assert lib.fft_scan_forward(long, OUT, None, None, size.value, None) == INVALID
    assert lib.fft_scan_forward(long, OUT, None, A + 4, size.value, None) == ALIGN
    assert lib.fft_scan_workspace(long, 2, size) == INVALID
    assert lib.fft_scan_workspace(long, 0, None) == INVALID
    seqs = sq._SEQ.unpack(OUT)
    grads = sq._GRADS.pack(*seqs, 0, *seqs, *seqs, *seqs, *seqs, 0, 0, 0, 0, 0, 0, 0)
    assert lib.fft_scan_workspace(long, 1, size) == fx.FFT_OK
    assert lib.fft_scan_backward(long, grads, A, size.value - 1, None) == INVALID
    assert lib.fft_scan_backward(scan(z=(A, 128, 16)), grads, A, 1 << 40, None) == INVALID  # no dz
    assert lib.fft_scan_step(scan(), OUT, A, 4, None, None, None) == INVALID
    assert lib.fft_scan_step(scan(length=1), OUT, A + 2, 4, None, None, None) == ALIGN


def test_scan_workspace_goes_by_the_cut(lib):
    """Many channels need no workspace; few channels and a long row need a state per chunk."""
    size = ctypes.c_size_t()
    assert lib.fft_scan_workspace(scan(nseq=64, channels=4096, length=512), 0, size) == fx.FFT_OK
    assert size.value == 0
    assert lib.fft_scan_workspace(scan(nseq=1, channels=128, length=8192), 0, size) == fx.FFT_OK
    assert 0 < size.value <= 128 * 128 * (16 + 1) * 4 + 128 * 4 + 64
    assert lib.fft_scan_workspace(scan(length=0), 0, size) == fx.FFT_OK and size.value == 0


@pytest.mark.parametrize("change,status", [
    (dict(dtype=sq.E4M3), INVALID), (dict(res=sq.F16), INVALID), (dict(out=sq.F32), INVALID),
    (dict(columns=0), INVALID), (dict(columns=16385), SIZE), (dict(rows=-1), INVALID),
    (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(weight=0), INVALID),
    (dict(group=32), INVALID), (dict(out=sq.E4M3, group=48), INVALID), (dict(weight=A + 2), ALIGN)],
    ids=str)
def test_norm_refuses(lib, change, status):
    d = norm(**change)
    cols = max(1, change.get("columns", 64))
    assert lib.fft_norm_forward(d, A, cols, None, 0, A, cols, A, None, 0, None) == status


def test_norm_calls_refuse(lib):
    d = norm()
    assert lib.fft_norm_forward(d, None, 64, None, 0, A, 64, None, None, 0, None) == INVALID
    assert lib.fft_norm_forward(d, A, 63, None, 0, A, 64, None, None, 0, None) == INVALID
    assert lib.fft_norm_forward(d, A + 1, 64, None, 0, A, 64, None, None, 0, None) == ALIGN
    assert lib.fft_norm_forward(norm(out=sq.E4M3), A, 64, None, 0, A, 64, None, None, 0, None) == INVALID
    assert lib.fft_norm_backward(d, A, 64, A, 64, None, 0, None, 0, None, 0, None, None, 0,
                                 None) == INVALID  # nothing to compute
    assert lib.fft_norm_backward(d, A, 64, A, 64, None, 0, A, 64, None, 0, A, None, 0, None) == INVALID
    # no rows: nothing to do, and nothing read
    assert lib.fft_norm_forward(norm(rows=0), A, 64, None, 0, A, 64, None, None, 0, None) == fx.FFT_OK


def test_lib_names_are_exported():
    for name in sq.SYMBOLS:
        assert name in fx.ABI_SYMBOLS


def test_norm_of_no_rows_needs_no_address(lib):
    """Tensors without elements have the address 0."""
    d = norm(rows=0)
    assert lib.fft_norm_forward(d, None, 64, None, 0, None, 64, None, None, 0, None) == fx.FFT_OK
    q = norm(rows=0, out=sq.E4M3, group=32)
    assert lib.fft_norm_forward(q, None, 64, None, 0, None, 64, None, None, 64, None) == fx.FFT_OK
    assert lib.fft_norm_backward(d, None, 64, None, 64, None, 0, None, 64, None, 64, None, None, 0,
                                 None) == fx.FFT_OK
    assert lib.fft_norm_forward(norm(rows=0, columns=0), None, 1, None, 0, None, 1, None, None, 0,
                                None) == INVALID


def test_convolution_over_its_input_is_refused(lib):
    assert lib.fft_conv_forward(conv(), OUT, None, None) == INVALID
    assert lib.fft_conv_forward(conv(x=(A, 256, 32)), sq._SEQ.pack(A + 30, 256, 32), None, None) == INVALID
    apart = sq._SEQ.pack(A + 4096, 128, 16)
    assert lib.fft_conv_forward(conv(initial=A + 8192), apart, A + 8192 + 64, None) == INVALID
    assert lib.fft_conv_backward(conv(), apart, None, apart, None, None, None, None, 0, None) == INVALID


def test_scan_over_its_inputs_is_refused(lib):
    def at(offset):
        return A + (offset << 12), 128, 16

    apart = dict(u=at(1), delta=at(2), B=at(3), C=at(4))
    for name in apart:  # from the 8th column on
        data, *strides = apart[name]
        assert lib.fft_scan_forward(scan(**apart), sq._SEQ.pack(data + 16, *strides), None, None, 0,
                                    None) == INVALID, name
    for name in ("delta", "B", "C"):
        assert lib.fft_scan_forward(scan(**apart), sq._SEQ.pack(*apart[name]), None, None, 0,
                                    None) == INVALID, name
    state = A + (9 << 12)
    assert lib.fft_scan_forward(scan(**apart, initial=state), sq._SEQ.pack(*at(5)), state, None, 0,
                                None) == INVALID


def test_steps_over_their_inputs_are_refused(lib):
    one = conv(length=1, x=(A, 128, 16))
    assert lib.fft_conv_step(one, sq._SEQ.pack(A + 16, 128, 16), A + 4096, 4, None, None, None) == INVALID
    one = scan(length=1, u=(A, 128, 16), delta=(A + 4096, 128, 16), B=(A + 8192, 128, 16),
               C=(A + 12288, 128, 16))
    for at in (A + 16, A + 4096 + 16, A + 8192, A + 12288):
        assert lib.fft_scan_step(one, sq._SEQ.pack(at, 128, 16), A + 16384, 4, None, None, None) == INVALID


def test_norm_over_its_inputs_is_refused(lib):
    d = norm()
    for at in (A + 2, A + 16, A - 126):
        assert lib.fft_norm_forward(d, A, 64, None, 0, at, 64, None, None, 0, None) == INVALID
        assert lib.fft_norm_forward(norm(res=sq.BF16), A + 8192, 64, A, 64, A + 16384, 64, None, at, 64,
                                    None) == INVALID
    q = norm(out=sq.E4M3)
    assert lib.fft_norm_forward(q, A, 64, None, 0, A, 64, A + 8192, None, 0, None) == INVALID
