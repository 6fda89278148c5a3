"""Group norm over the tokens of sequences that begin with a value far from all others, as the first token
of a prompt has them: mean, deviation and outputs against 64 bits.

Tolerances.  A run of at most 128 values is summed in float32 about a value near its mean, 128 additions
deep at most, and two dozen runs are joined about their means, each step off by a few units: 2^-24 of
the deviations' absolute sum for each, in no one direction.  FEW = 64 * 2^-24 of a deviation for the
mean (and the mean's own rounding) and 2^-16 of the inverse deviation, whose squares' error counts half,
are above both.  Outputs as in test_gpu_group_norm.py."""
import pytest

torch = pytest.importorskip("torch")

from test_gpu_group_norm import FEW, UNIT, bound, d64, data, fx, reference  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__

    __graft_entry__.build()


def far(layout, d, groups, dtype, value, everywhere, seed):
    c, _, _ = data(layout, d, groups, dtype, "none", "plain", seed=seed)
    rows = c["x"].view(-1, d)
    each = d // groups
    if c["offsets"] is not None:
        firsts = [int(a) for a, b in zip(c["offsets"][:-1], c["offsets"][1:]) if b > a]
    else:
        firsts = range(0, rows.shape[0], layout[1])
    for i, t in enumerate(firsts):
        rows[t, 0::each] = value * (-1) ** i
        if everywhere:  # later tiles begin with such a value as well
            rows[t + 32::128, 0::each] = -value
    return c


@pytest.mark.parametrize("everywhere", [False, True])
@pytest.mark.parametrize("value", [300.0, 1e4, 6e4])
@pytest.mark.parametrize("layout", [(1, 4096), (3, 200), [700, 0, 2000]], ids=str)
@pytest.mark.parametrize("d,groups,dtype", [(512, 1, "f32"), (512, 1, "bf16"), (1024, 2, "f16"), (4096, 1, "bf16"),
                                            (330, 6, "f32"), (1030, 1, "f32")])
def test_first_value_far_from_the_rest(d, groups, dtype, layout, value, everywhere):
    c = far(layout, d, groups, dtype, value, everywhere, 31)
    r = fx().group_norm(**c, groups=groups)
    out, mean, rstd = reference(c, groups)
    assert ((d64(r.rstd) - rstd).abs() <= 2.0 ** -16 * rstd).all()
    assert ((d64(r.mean) - mean).abs() <= 2.0 ** -24 * mean.abs() + FEW / rstd).all()
    tol = UNIT[r.out.dtype] * out.abs() * 1.001 + FEW * bound(c, groups, out, mean, rstd) + (
        2.0 ** -24 if dtype == "f16" else 0.0)
    assert ((d64(r.out) - out).abs() <= tol).all()


def test_values_whose_squares_leave_float32():
    """Deviations beyond float32 have the inverse 0: outputs are the bias, not NaN."""
    c, _, groups = data((1, 300), 64, 4, "f32", "none", "plain", seed=32)
    c["x"] = c["x"] * 1e30
    r = fx().group_norm(**c, groups=groups)
    assert not r.rstd.any() and torch.isfinite(r.mean).all()
    assert torch.equal(r.out, c["bias"].expand_as(r.out))
