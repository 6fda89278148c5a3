"""Gradients of group norm for many short sequences and for many rows in wide groups, whose sums over
tokens are left by blocks that take several tiles each: against the definition in 64 bits, the same bits
in every call.  Tolerances as in test_gpu_group_norm.py, but for the sums of the parameters: a thread
adds at most 2^13 terms here, of either sign, each rounding 2^-24 of a sum that grows as their root:
PARTS = 2^-17 of the absolute sums is above that."""
import pytest

torch = pytest.importorskip("torch")

from test_gpu_group_norm import data, d64, fx, gradients, near, randn, reference  # noqa: E402

pytestmark = pytest.mark.gpu
PARTS = 2.0 ** -17


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__

    __graft_entry__.build()


@pytest.mark.parametrize("layout,shape", [
    ((5000, 2), (40, 5, "bf16", "gate", "half")), ((3001, 3), (30, 6, "f32", "silu", "odd")),
    (4001, (1030, 1, "f32", "gate", "plain")), (3000, (4096, 2, "bf16", "silu gate", "half")),
    (2500, (2056, 1, "f16", "none", "plain")), ([3] * 1500 + [0, 1, 400], (264, 1, "bf16", "gate", "plain")),
    ((40, 300), (528, 3, "bf16", "silu", "plain")), ((1, 40001), (24, 1, "f32", "silu", "plain"))], ids=str)
def test_gradients(layout, shape):
    c, rng, groups = data(layout, *shape, seed=51)
    dout = randn(rng, *c["x"].shape, dtype=c["x"].dtype)
    f = fx().group_norm(**c, groups=groups)

    def back():
        return fx().group_norm_backward(dout, c["x"], f.mean, f.rstd, c["weight"], c["bias"], z=c["z"],
                                        silu=c["silu"], offsets=c["offsets"])

    r = back()
    assert all(torch.equal(a, b) for a, b in zip(r, back()) if a is not None)
    for name, got, want in zip(r._fields, r, gradients(c, groups, dout)):
        if want is None:
            assert got is None
            continue
        more = 0.0
        if name in ("dweight", "dbias"):
            dy = 1.1 * d64(dout).abs()
            if c["z"] is not None:
                dy = dy * (d64(c["z"]) * torch.sigmoid(d64(c["z"]))).abs()
            if name == "dweight":
                blank = {**c, "weight": torch.ones(()), "bias": torch.zeros(()), "z": None, "silu": False}
                dy = dy * reference(blank, groups)[0].abs()
            more = PARTS * float(dy.reshape(-1, dy.shape[-1]).sum(0).norm())
        near(got, want, name, more)
