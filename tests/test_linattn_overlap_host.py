"""Linear attention's outputs over states and states over its inputs are refused (no GPU needed)."""
import pytest

import fft_signal_processing_gb300 as fx
from fft_signal_processing_gb300 import sequence as sq

INVALID = fx.FFT_ERR_INVALID_ARG
A, MB = 1 << 20, 1 << 20
STATES = 2 * 4 * 16 * 32 * 4  # bytes: sequences, heads, dk, dv


@pytest.fixture(scope="module")
def lib():
    from fft_signal_processing_gb300 import _build

    _build.build()
    return fx.lib()


def attn(length=8, initial=0, nseq=2):
    return sq._ATTN.pack(sq.F32, 1.0, nseq, length, 4, 2, 16, 32, 0, initial, A, 256, 32, 16, A + MB, 256, 32, 16,
                         A + 2 * MB, 1024, 128, 32, A + 3 * MB, 32, 4)


OUT = A + 4 * MB
SPAN = (1024 + 7 * 128 + 128) * 4  # bytes of v, dout, out and dv


def heads(at):
    return sq._HEADS.pack(at, 1024, 128, 32)


@pytest.mark.parametrize("pool", [2, 5])
def test_step_over_its_states(lib, pool):
    def call(at, state=A + 32 * MB):
        return lib.fft_linattn_step(attn(1), heads(at), state, pool, None, None, None)

    state = A + 32 * MB
    one = (1024 + 128) * 4  # bytes of two sequences' outputs
    for at in (state, state + 4, state + pool * STATES // 2 - 4, state - one + 4):
        assert call(at) == INVALID, at - state


def test_forward_over_states(lib):
    state = A + 32 * MB
    for at in (state, state + STATES - 4, state - SPAN + 4):
        assert lib.fft_linattn_forward(attn(initial=state), heads(at), None, A + 64 * MB, 1 << 40, None) == INVALID
        assert lib.fft_linattn_forward(attn(), heads(at), state, A + 64 * MB, 1 << 40, None) == INVALID
    for at in (A, A + MB, A + 2 * MB, A + 3 * MB):  # the final state over inputs
        assert lib.fft_linattn_forward(attn(), heads(OUT), at, A + 64 * MB, 1 << 40, None) == INVALID, at


def grads(dfinal=0, dinitial=0, **k):
    v = dict(dout=(A + 5 * MB, 1024, 128, 32), dq=(A + 6 * MB, 256, 32, 16), dk=(A + 7 * MB, 256, 32, 16),
             dv=(A + 8 * MB, 1024, 128, 32), ddecay=(A + 9 * MB, 32, 4))
    v.update(k)
    return sq._ATTN_GRADS.pack(*v["dout"], dfinal, *v["dq"], *v["dk"], *v["dv"], *v["ddecay"], dinitial)


def test_gradients_over_states(lib):
    def call(initial=0, **k):
        return lib.fft_linattn_backward(attn(initial=initial), grads(**k), A + 64 * MB, 1 << 40, None)

    state = A + 32 * MB
    for name, row in (("dq", (256, 32, 16)), ("dk", (256, 32, 16)), ("dv", (1024, 128, 32)), ("ddecay", (32, 4))):
        for at in (state, state + STATES - 4):
            assert call(initial=state, **{name: (at, *row)}) == INVALID, name
            assert call(dfinal=state, **{name: (at, *row)}) == INVALID, name
            assert call(dinitial=state, **{name: (at, *row)}) == INVALID, name
    for at in (A, A + MB, A + 2 * MB, A + 3 * MB, A + 5 * MB):  # the state's gradient over inputs
        assert call(dinitial=at) == INVALID, at


def test_pools_beyond_all_memory(lib):
    """A pool's size is not multiplied past 64 bits."""
    for pool in (1 << 40, 1 << 55, (1 << 63) - 1):
        assert lib.fft_linattn_step(attn(1), heads(A + 33 * MB), A + 32 * MB, pool, None, None, None) == INVALID
