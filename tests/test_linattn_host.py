"""Host-side checks of linear attention and group norm (no GPU needed): descriptor layouts against the
header, refusals before anything is enqueued, workspace sizes, outputs over inputs."""
import ctypes
import os
import subprocess

import pytest

import fft_signal_processing_gb300 as fx
from fft_signal_processing_gb300 import sequence as sq

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INVALID, SIZE, ALIGN = fx.FFT_ERR_INVALID_ARG, fx.FFT_ERR_UNSUPPORTED_SIZE, fx.FFT_ERR_MISALIGNED
A = 1 << 20  # an address that is never read: the calls under test are refused on the host
MB = 1 << 20


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
    printf("%zu %zu %zu %zu %zu", sizeof(fft_heads), sizeof(fft_linattn_desc), sizeof(fft_linattn_grads),
           sizeof(fft_gnorm_desc), sizeof(fft_gnorm_grads));
    O(fft_linattn_desc, scale); O(fft_linattn_desc, nseq); O(fft_linattn_desc, offsets); O(fft_linattn_desc, q);
    O(fft_linattn_desc, decay); O(fft_linattn_grads, dq); O(fft_linattn_grads, ddecay);
    O(fft_linattn_grads, dinitial_state); O(fft_gnorm_desc, eps); O(fft_gnorm_desc, nseq); O(fft_gnorm_desc, x);
    O(fft_gnorm_grads, dout); O(fft_gnorm_grads, dweight);
    return 0;
}''')
    exe = tmp_path / "sizes"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = [int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True).stdout.split()]
    sizes = [s.size for s in (sq._HEADS, sq._ATTN, sq._ATTN_GRADS, sq._GNORM, sq._GNORM_GRADS)]
    assert got == sizes + [4, 8, 56, 72, 168, 40, 136, 160, 12, 16, 72, 16, 88]


def attn(**k):
    v = dict(dtype=sq.BF16, scale=1.0, nseq=2, length=8, heads=4, groups=2, dk=16, dv=32, offsets=0, initial=0,
             q=(A, 256, 32, 16), k=(A + MB, 256, 32, 16), v=(A + 2 * MB, 1024, 128, 32), decay=(A + 3 * MB, 32, 4))
    v.update(k)
    return sq._ATTN.pack(*list(v.values())[:10], *v["q"], *v["k"], *v["v"], *v["decay"])


OUT = (A + 4 * MB, 1024, 128, 32)


def forward(lib, desc, out=OUT, final=None, workspace=A + 64 * MB, size=1 << 40):
    return lib.fft_linattn_forward(desc, sq._HEADS.pack(*out), final, workspace, size, None)


@pytest.mark.parametrize("change,status", [
    (dict(dtype=7), INVALID), (dict(dtype=sq.E4M3), INVALID), (dict(nseq=0), INVALID), (dict(length=-1), INVALID),
    (dict(heads=0), INVALID), (dict(groups=0), INVALID), (dict(groups=3), INVALID), (dict(dk=0), INVALID),
    (dict(dv=0), INVALID), (dict(dk=257), SIZE), (dict(dv=257), SIZE), (dict(heads=65536, groups=65536), SIZE),
    (dict(length=1 << 31), SIZE), (dict(offsets=A + 4), ALIGN), (dict(initial=A + 2), ALIGN),
    (dict(q=(0, 256, 32, 16)), INVALID), (dict(q=(A + 1, 256, 32, 16)), ALIGN), (dict(k=(A, -1, 32, 16)), INVALID),
    (dict(v=(A, 1024, 1 << 27, 32)), SIZE), (dict(v=(A, 1 << 60, 128, 32)), SIZE),
    (dict(v=(A, 1024, 128, 1 << 60)), SIZE), (dict(decay=(0, 32, 4)), INVALID), (dict(decay=(A + 1, 32, 4)), ALIGN)],
    ids=str)
def test_linattn_refuses(lib, change, status):
    assert forward(lib, attn(**change)) == status
    step = {**change, "length": change.get("length", 1)}
    assert lib.fft_linattn_step(attn(**step), sq._HEADS.pack(*OUT), A + 8 * MB, 4, None, None, None) == status
    size = ctypes.c_size_t()
    if not set(change) & {"q", "k", "v", "decay", "initial"}:
        assert lib.fft_linattn_workspace(attn(**change), 0, size) == status


def test_linattn_calls_refuse(lib):
    d = attn()
    assert lib.fft_linattn_forward(None, sq._HEADS.pack(*OUT), None, None, 0, None) == INVALID
    assert lib.fft_linattn_forward(d, None, None, None, 0, None) == INVALID
    assert forward(lib, d, final=A + 2) == ALIGN
    assert forward(lib, d, workspace=A + 8) == ALIGN
    for out in ((OUT[0], 1024, 64, 32), (OUT[0], 1024, 128, 16), (OUT[0], 512, 128, 32), (OUT[0], 0, 128, 32)):
        assert forward(lib, d, out=out) == INVALID  # rows that overlap
    size = ctypes.c_size_t()
    long = attn(nseq=1, length=65536)
    assert lib.fft_linattn_workspace(long, 0, size) == fx.FFT_OK and size.value > 0
    far = (A + (1 << 30), 1024, 128, 32)
    wide = dict(q=(A, 0, 32, 16), k=(A + 64 * MB, 0, 32, 16), v=(A + 128 * MB, 0, 128, 32),
                decay=(A + 256 * MB, 0, 4))
    long = attn(nseq=1, length=65536, **wide)
    assert forward(lib, long, out=far, workspace=A + (1 << 34), size=size.value - 1) == INVALID
    assert forward(lib, long, out=far, workspace=None, size=size.value) == INVALID
    assert lib.fft_linattn_workspace(long, 2, size) == INVALID
    assert lib.fft_linattn_workspace(long, 0, None) == INVALID
    assert lib.fft_linattn_workspace(attn(length=0), 1, size) == fx.FFT_OK and size.value == 0


def grads(**k):
    v = dict(dout=(A + 5 * MB, 1024, 128, 32), dfinal=0, dq=(A + 6 * MB, 256, 32, 16), dk=(A + 7 * MB, 256, 32, 16),
             dv=(A + 8 * MB, 1024, 128, 32), ddecay=(A + 9 * MB, 32, 4), dinitial=0)
    v.update(k)
    return sq._ATTN_GRADS.pack(*v["dout"], v["dfinal"], *v["dq"], *v["dk"], *v["dv"], *v["ddecay"], v["dinitial"])


def test_linattn_gradients_refuse(lib):
    def call(workspace=A + 64 * MB, size=1 << 40, **k):
        return lib.fft_linattn_backward(attn(), grads(**k), workspace, size, None)

    assert lib.fft_linattn_backward(attn(), None, A, 0, None) == INVALID
    assert call(size=16) == INVALID and call(workspace=None) == INVALID and call(workspace=A + 8) == ALIGN
    assert call(dfinal=A + 2) == ALIGN and call(dinitial=A + 1) == ALIGN
    for name in ("dout", "dq", "dk", "dv", "ddecay"):
        n = 3 if name == "ddecay" else 4
        assert call(**{name: (0, 1024, 128, 32)[:n]}) == INVALID, name
        assert call(**{name: (A + 16 * MB + 1, 1024, 128, 32)[:n]}) == ALIGN, name
    for name in ("dq", "dk", "dv"):  # over what is read
        for at in (A, A + MB, A + 2 * MB, A + 3 * MB, A + 5 * MB):
            dim = (256, 32, 16) if name != "dv" else (1024, 128, 32)
            assert call(**{name: (at, *dim)}) == INVALID, (name, at)
    assert call(dfinal=A + 32 * MB, dinitial=A + 32 * MB + 64) == INVALID


def test_linattn_over_its_inputs_is_refused(lib):
    for at in (A, A + 16, A + MB, A + 2 * MB, A + 2 * MB + 64, A + 3 * MB):
        assert forward(lib, attn(), out=(at, 1024, 128, 32)) == INVALID
        one = attn(length=1)
        assert lib.fft_linattn_step(one, sq._HEADS.pack(at, 1024, 128, 32), A + 32 * MB, 4, None, None, None) == INVALID
    # heads around tokens: ranges of addresses that meet count as overlapping
    assert forward(lib, attn(v=(A + 2 * MB, 4096, 32, 512)), out=(A + 2 * MB + 512, 4096, 32, 512)) == INVALID
    assert forward(lib, attn(initial=A + 32 * MB), final=A + 32 * MB + 4096) == INVALID


def test_linattn_step_refuses(lib):
    out = sq._HEADS.pack(*OUT)
    one = attn(length=1)
    assert lib.fft_linattn_step(attn(), out, A + 32 * MB, 4, None, None, None) == INVALID  # more than one token
    assert lib.fft_linattn_step(one, None, A + 32 * MB, 4, None, None, None) == INVALID
    assert lib.fft_linattn_step(one, out, A + 32 * MB, 1, None, None, None) == INVALID  # pool below the sequences
    assert lib.fft_linattn_step(one, out, None, 4, None, None, None) == INVALID
    assert lib.fft_linattn_step(one, out, A + 2, 4, None, None, None) == ALIGN
    assert lib.fft_linattn_step(one, out, A + 32 * MB, 4, A + 4, None, None) == ALIGN
    assert lib.fft_linattn_step(one, out, A + 32 * MB, -1, None, None, None) == INVALID


def gnorm(**k):
    v = dict(dtype=sq.BF16, param=sq.F32, silu=0, eps=1e-5, nseq=2, length=8, channels=64, groups=4, offsets=0,
             weight=A + 32 * MB, bias=A + 33 * MB, x=(A, 512, 64), z=(0, 0, 0))
    v.update(k)
    return sq._GNORM.pack(*list(v.values())[:11], *v["x"], *v["z"])


NORMED, MEAN, RSTD, WORK = sq._SEQ.pack(A + MB, 512, 64), A + 40 * MB, A + 41 * MB, A + 64 * MB


@pytest.mark.parametrize("change,status", [
    (dict(dtype=sq.E4M3), INVALID), (dict(param=sq.F16), INVALID), (dict(silu=2), INVALID), (dict(eps=-1.0), INVALID),
    (dict(eps=float("nan")), INVALID), (dict(nseq=0), INVALID), (dict(length=-1), INVALID),
    (dict(channels=0), INVALID), (dict(groups=0), INVALID), (dict(groups=3), INVALID),
    (dict(channels=65544, groups=1), SIZE), (dict(length=1 << 31), SIZE), (dict(offsets=A + 4), ALIGN),
    (dict(weight=A + 2), ALIGN), (dict(bias=A + 1), ALIGN), (dict(x=(0, 512, 64)), INVALID),
    (dict(x=(A + 1, 512, 64)), ALIGN), (dict(x=(A, -1, 64)), INVALID), (dict(x=(A, 512, 1 << 27)), SIZE),
    (dict(z=(A + 2 * MB + 1, 512, 64)), ALIGN)], ids=str)
def test_gnorm_refuses(lib, change, status):
    assert lib.fft_gnorm_forward(gnorm(**change), NORMED, MEAN, RSTD, WORK, 1 << 40, None) == status
    size = ctypes.c_size_t()
    if not set(change) & {"x", "z", "weight", "bias"}:
        assert lib.fft_gnorm_workspace(gnorm(**change), 0, size) == status


def test_gnorm_calls_refuse(lib):
    d = gnorm()
    assert lib.fft_gnorm_forward(d, None, MEAN, RSTD, WORK, 1 << 40, None) == INVALID
    assert lib.fft_gnorm_forward(d, NORMED, None, RSTD, WORK, 1 << 40, None) == INVALID
    assert lib.fft_gnorm_forward(d, NORMED, MEAN, RSTD + 2, WORK, 1 << 40, None) == ALIGN
    assert lib.fft_gnorm_forward(d, NORMED, MEAN, RSTD, None, 0, None) == INVALID
    assert lib.fft_gnorm_forward(d, NORMED, MEAN, RSTD, WORK + 8, 1 << 40, None) == ALIGN
    assert lib.fft_gnorm_forward(d, sq._SEQ.pack(A + MB, 512, 32), MEAN, RSTD, WORK, 1 << 40, None) == INVALID
    assert lib.fft_gnorm_forward(d, sq._SEQ.pack(A + 16, 512, 64), MEAN, RSTD, WORK, 1 << 40, None) == INVALID
    size = ctypes.c_size_t()
    assert lib.fft_gnorm_workspace(gnorm(length=1), 0, size) == fx.FFT_OK and size.value == 0  # token by token
    assert lib.fft_gnorm_workspace(gnorm(length=0), 1, size) == fx.FFT_OK and size.value == 0
    assert lib.fft_gnorm_workspace(d, 0, size) == fx.FFT_OK and size.value > 0

    def back(desc=d, mean=MEAN, dout=(A + 2 * MB, 512, 64), dx=(A + 3 * MB, 512, 64), dz=(0, 0, 0), dw=A + 50 * MB,
             db=A + 51 * MB, work=WORK, size=1 << 40):
        g = sq._GNORM_GRADS.pack(mean, RSTD, *dout, *dx, *dz, dw, db)
        return lib.fft_gnorm_backward(desc, g, work, size, None)

    assert lib.fft_gnorm_backward(d, None, WORK, 1 << 40, None) == INVALID
    assert back(mean=0) == INVALID and back(work=None) == INVALID and back(size=16) == INVALID
    assert back(dz=(A + 4 * MB, 512, 64)) == INVALID  # no gate
    assert back(desc=gnorm(z=(A + 5 * MB, 512, 64))) == INVALID  # no dz
    assert back(dw=A + 2) == ALIGN and back(db=A + 1) == ALIGN
    for at in (A, A + 16, A + 2 * MB):
        assert back(dx=(at, 512, 64)) == INVALID


def test_names_are_exported():
    for name in sq.SYMBOLS:
        assert name in fx.ABI_SYMBOLS
    for name in ("linear_attention", "linear_attention_backward", "linear_attention_step", "linear_attention_check",
                 "group_norm", "group_norm_backward"):
        assert callable(getattr(fx, name))
