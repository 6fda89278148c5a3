"""Steps below zero (softplus off) let a state grow.  Over a chunk of time the growth may be more than
float32 holds while the state before it is 0 or small: what leaves the chunk is the definition's."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import seqref  # noqa: E402
from test_gpu_sequence import close, d64, randn  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__

    __graft_entry__.build()


def data(n, quiet):
    """One row of 320 tokens, which is cut at every 64th.  The states fall by exp(-80) over the first
    64 tokens, grow by exp(100) over the next and fall from there on.  Inputs enter before token 8 and
    from token 128 on, quiet: from token 200 on."""
    rng = np.random.default_rng(n)
    d, length = 24, 320
    u = randn(rng, 1, length, d)
    u[:, 0 if quiet else 8:200 if quiet else 128] = 0
    step = torch.full((1, length, d), 0.4, device="cuda")
    step[:, :64], step[:, 64:128] = 80.0 / 64, -100.0 / 64
    A = -(1.0 - 0.05 * torch.rand(d, n, device="cuda", generator=torch.Generator("cuda").manual_seed(1)))
    B, C = randn(rng, 1, length, 1, n), randn(rng, 1, length, 1, n)
    return dict(u=u, delta=step, A=A, B=B, C=C)


@pytest.mark.parametrize("n", [1, 10, 16, 32])
@pytest.mark.parametrize("quiet", [False, True])
def test_growth_over_a_chunk(n, quiet):
    import fft_signal_processing_gb300 as fx

    c = data(n, quiet)
    out, final = fx.selective_scan(**c, return_state=True)
    ref, rfinal, size = seqref.scan(*(d64(c[k]) for k in "u delta A B C".split()), None, None, None,
                                    False, None, None, magnitude=True)
    close(out, ref, size)
    assert torch.isfinite(final).all()


@pytest.mark.parametrize("n", [1, 10, 16, 32])
@pytest.mark.parametrize("late", [False, True])
def test_gradients_of_growth_over_a_chunk(n, late):
    """late: gradients enter from token 300 on, else before token 50.  Errors: 2^-22 per step, each
    1 + 100/64 of a unit for its exponent, carried over the 128 steps of decay and growth."""
    import fft_signal_processing_gb300 as fx

    c = data(n, False)
    dout = randn(np.random.default_rng(5), *c["u"].shape)
    dout[:, 0 if late else 50:300 if late else None] = 0
    got = fx.selective_scan_backward(dout, **c)
    v = {k: d64(c[k]).requires_grad_(True) for k in c}
    out, _ = seqref.scan(*(v[k] for k in "u delta A B C".split()), None, None, None, False, None, None)
    grads = torch.autograd.grad((out * d64(dout)).sum(), list(v.values()))
    for k, ref in zip(v, grads):
        err = (d64(getattr(got, "d" + k)) - ref).norm()
        assert err <= 328 * 2.0 ** -22 * ref.norm(), (k, float(err / ref.norm()))
