"""A value that is not finite in linear attention's gradients: the decay's gradients of other sequences
and other heads are the same bits, and every token whose pairs it is in is marked."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from test_gpu_linattn import data, fx, randn  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__

    __graft_entry__.build()


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("lens,at", [([300, 400], 350), ([300, 400], 699), ([300, 400], 300), ([1500, 1500], 1900)],
                         ids=str)
def test_decays_of_other_sequences_and_heads(lens, at, dtype, bad):
    c = data(lens, 2, 2, 32, 32, dtype, False, "plain", seed=61)
    dout = randn(np.random.default_rng(62), *c["v"].shape, dtype=c["v"].dtype)
    good = fx().linear_attention_backward(dout, **c)
    assert all(torch.isfinite(t).all() for t in good if t is not None)
    for name in ("q", "k", "v"):
        t = c[name].clone()
        t[at, 1, 9] = bad
        r = fx().linear_attention_backward(dout, **{**c, name: t})
        for got, want in zip(r[:4], good):
            assert torch.equal(got[:lens[0]], want[:lens[0]]), name  # the first sequence
            assert torch.equal(got[:, 0], want[:, 0]), name  # the other head
        # the pairs (j, i), j < t <= i, of decay t: those with i = at, or with j = at
        marked = slice(lens[0] + 1, at + 1) if name == "q" else slice(at + 1, sum(lens))
        assert not torch.isfinite(r.ddecay[marked, 1]).any(), name
