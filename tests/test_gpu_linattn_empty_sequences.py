"""Linear attention over packed rows with sequences without tokens at their ends and between others, at
lengths of thousands of tokens, where time is cut: outputs, final states and all gradients against the
definition in 64 bits.  Tolerances as in test_gpu_linattn.py."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from test_gpu_linattn import STATE, TERM, close, data, fx, gradients, near, randn, reference  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__

    __graft_entry__.build()


def ragged(seed, nseq, total):
    """Cuts at random places, three sequences without tokens, at both ends and in the middle."""
    cuts = np.sort(np.random.default_rng(seed).integers(0, total + 1, nseq - 1))
    lens = np.diff(np.concatenate([[0], cuts, [total]])).tolist()
    return [0, *lens[:nseq // 2], 0, *lens[nseq // 2:], 0]


@pytest.mark.parametrize("shape,nseq,total", [((6, 3, 40, 72, "f32", True, "wide"), 34, 10007),
                                              ((6, 3, 40, 72, "bf16", True, "wide"), 34, 10007),
                                              ((2, 2, 64, 96, "f16", False, "plain"), 10, 5001)], ids=str)
def test_outputs_and_states(shape, nseq, total):
    c = data(ragged(21, nseq, total), *shape, seed=22, rate=0.01)
    out, final = fx().linear_attention(**c, return_state=True)
    ref, rfinal, size, whole = reference(c, magnitude=True)
    close(out, ref, size, TERM[out.dtype], "out")
    close(final, rfinal, whole, STATE, "final")
    empty = (c["offsets"][1:] == c["offsets"][:-1])
    want = c["initial_state"][empty] if c["initial_state"] is not None else torch.zeros_like(final[empty])
    assert torch.equal(final[empty], want)


@pytest.mark.parametrize("shape", [(2, 2, 64, 96, "f16", True, "plain"), (2, 1, 32, 24, "f32", True, "plain"),
                                   (2, 2, 64, 64, "bf16", True, "plain")], ids=str)
def test_gradients(shape):
    c = data(ragged(23, 10, 2003), *shape, seed=24, rate=0.01)
    rng = np.random.default_rng(25)
    dout, dfinal = randn(rng, *c["v"].shape, dtype=c["v"].dtype), randn(rng, *c["initial_state"].shape)
    r = fx().linear_attention_backward(dout, **c, dfinal_state=dfinal)
    for name, got, want in zip(r._fields, r, gradients(c, dout, dfinal)):
        near(got, want, name)
    empty = (c["offsets"][1:] == c["offsets"][:-1])
    assert torch.equal(r.dinitial_state[empty], dfinal[empty])
