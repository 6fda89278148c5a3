"""Linear attention token by token for long answers: a state that is kept for hundreds of tokens leans to
no side.

Tolerance.  With keys of zeros every token multiplies a state by exp(g): one rounding of the exponential
and one of the product, each at most half a unit of 2^-24 of values in [1/2, 1) and of either sign.  The
average over `samples` independent tokens and heads of such errors has a standard deviation of
2^-24 * sqrt(1/6) / sqrt(samples), under 0.002 units here; 0.05 units are above that and below the 0.1 to
0.5 by which the GPU's approximate exponential lies low."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from test_gpu_linattn import fx, randn  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__

    __graft_entry__.build()


@pytest.mark.parametrize("rate,tokens", [(1e-4, 400), (0.01, 400), (0.3, 200), (0.69, 100)])
def test_kept_states_lean_to_no_side(rate, tokens):
    rng = np.random.default_rng(41)
    nseq, heads, dk, dv = 64, 16, 2, 8
    state = randn(rng, nseq, heads, dk, dv)
    want = state.double()
    q, v = randn(rng, nseq, heads, dk), randn(rng, nseq, heads, dv)
    k = torch.zeros_like(q)
    for _ in range(tokens):
        g = -torch.from_numpy(rng.random((nseq, heads)) * rate).float().cuda()
        fx().linear_attention_step(state, q, k, v, g)
        want *= torch.exp(g.double())[..., None, None]
    lean = float(((state.double() / want - 1).mean() / tokens) * 2.0 ** 24)
    assert abs(lean) <= 0.05, lean


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_decays_of_every_kind(dtype):
    """One step from states of 1: exp(g) itself, what counts as 0, what clears a state, and what is no
    number.  A power of 2 times 1 + s with |s| <= 0.42: its rounding is at most 2^-24 of the result, that of
    s 2^-26, and the argument's and the terms' of s are 2^-26 again: two units of 2^-24 bound them."""
    g = torch.cat([-torch.logspace(-8, 2, 500), torch.tensor([0.0, 0.5, 300.0, -103.0, -104.0, -1e4, -float("inf"),
                                                              float("nan")])]).to(dtype).cuda()
    n = g.numel()
    state = torch.ones(n, 1, 1, 4, device="cuda")
    z = torch.zeros(n, 1, 1, dtype=dtype, device="cuda")
    fx().linear_attention_step(state, z, z, torch.zeros(n, 1, 4, dtype=dtype, device="cuda"), g[:, None])
    want = torch.exp(g.double().clamp(max=0.0))
    got = state[:, 0, 0, 0].double()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    ok = ~torch.isnan(want)
    # below 2^-126 the spacing of float32 numbers is 2^-149
    assert ((got - want).abs() <= 2.0 ** -23 * want + 2.0 ** -149)[ok].all()
    assert (state == state[..., :1])[ok].all() and not state[n - 3: n - 1].any()
