"""What roundings leave of long-lived states.  A decay is one rounding of a number near 1, half a unit
of 2^-24; a walk of a thousand of them, as many tokens as the slowest states here are kept, is 16
units, 2^-20.  That holds as long as the roundings lean to no side."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import seqref  # noqa: E402
from test_gpu_sequence import d64, randn  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__

    __graft_entry__.build()


@pytest.mark.parametrize("n", [8, 16])
def test_gradients_of_slow_states(n):
    """Steps of 0.001 to 0.1, decay rates from 1 up: 1500 tokens."""
    import fft_signal_processing_gb300 as fx

    rng = np.random.default_rng(n)
    d, length = 64, 1500
    lead = (1, length)
    step = torch.from_numpy(np.exp(rng.uniform(np.log(0.001), np.log(0.1), d))).float().cuda()
    c = dict(u=randn(rng, *lead, d), delta=randn(rng, *lead, d, scale=0.5),
             A=-torch.arange(1, n + 1, device="cuda") * torch.exp(randn(rng, d, n, scale=0.2)),
             B=randn(rng, *lead, 1, n), C=randn(rng, *lead, 1, n), D=randn(rng, d),
             delta_bias=step + torch.log(-torch.expm1(-step)))
    dout = randn(rng, *lead, d)
    got = fx.selective_scan_backward(dout, softplus=True, **c)
    v = {k: d64(c[k]).requires_grad_(True) for k in c}
    out, _ = seqref.scan(v["u"], v["delta"], v["A"], v["B"], v["C"], v["D"], None, v["delta_bias"],
                         True, None, None)
    grads = torch.autograd.grad((out * d64(dout)).sum(), list(v.values()))
    for k, ref in zip(v, grads):
        err = float((d64(getattr(got, "d" + k)) - ref).norm() / ref.norm())
        assert err <= 2.0 ** -20, (k, err)


@pytest.mark.parametrize("n", [16, 32])
@pytest.mark.parametrize("nseq,d", [(1, 24), (160, 128)])
def test_steps_of_zero_keep_the_state(n, nseq, d):
    import fft_signal_processing_gb300 as fx

    rng = np.random.default_rng(n)
    length = 70 if nseq > 1 else 300
    zero = torch.zeros(nseq, length, d, device="cuda")
    B = randn(rng, nseq, length, 1, n)
    state = randn(rng, nseq, d, n)
    A = -torch.rand(d, n, device="cuda") * 16
    _, final = fx.selective_scan(randn(rng, nseq, length, d), zero, A, B, B, initial_state=state,
                                 return_state=True)
    assert torch.equal(final, state)
    pool = state.clone()
    fx.selective_scan_step(pool, randn(rng, nseq, d), zero[:, 0], A, B[:, 0], B[:, 0])
    assert torch.equal(pool, state)


def test_sums_over_long_chunks():
    """Sequences enough to fill the GPU, so that time is hardly cut: 4096 tokens enter dA, dD and the
    bias's gradient.  A walk of 256 additions is 8 units of 2^-24, the terms' own roundings 4."""
    import fft_signal_processing_gb300 as fx

    g = torch.Generator("cuda").manual_seed(1)
    nseq, length, d, n, some = 304, 4096, 128, 4, 8

    def rand(*shape):
        return torch.randn(*shape, device="cuda", generator=g)

    u, delta, dout = (rand(nseq, length, d) for _ in range(3))
    B, C = rand(nseq, length, 1, n), rand(nseq, length, 1, n)
    A = -torch.rand(d, n, device="cuda", generator=g) * 2 - 0.5
    D, bias = rand(d), rand(d) * 0.1 - 1.0
    got = fx.selective_scan_backward(dout, u, delta, A, B, C, D=D, delta_bias=bias, softplus=True)
    v = [A[:some].double().requires_grad_(True), D[:some].double().requires_grad_(True),
         bias[:some].double().requires_grad_(True)]
    us, gs = u[..., :some].double(), dout[..., :some].double()
    steps = torch.nn.functional.softplus(delta[..., :some].double() + v[2])
    h, loss = u.new_zeros(nseq, some, n, dtype=torch.float64), 0.0
    for t in range(length):
        dt = steps[:, t, :, None]
        h = torch.exp(dt * v[0]) * h + dt * us[:, t, :, None] * B[:, t].double()
        loss = loss + (gs[:, t] * ((h * C[:, t].double()).sum(-1) + v[1] * us[:, t])).sum()
    ref = torch.autograd.grad(loss, v)
    for k, r in zip(("dA", "dD", "ddelta_bias"), ref):
        mine = getattr(got, k)[:some].double()
        err = float((mine - r).norm() / r.norm())
        assert err <= 12 * 2.0 ** -24, (k, err)
