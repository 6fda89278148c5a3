"""Group norm of groups whose values are all alike, at any level up to the largest number of their type:
the mean is that value, the deviation 0 and outputs are the bias, bit for bit; and of groups that hold the
type's lowest value beside ordinary ones, as masked places do."""
import pytest

torch = pytest.importorskip("torch")

from test_gpu_group_norm import TYPES, data, fx, reference, d64  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__

    __graft_entry__.build()


@pytest.mark.parametrize("layout", [(1, 1000), (3, 37), [700, 0, 129, 1], (2, 5)], ids=str)
@pytest.mark.parametrize("d,groups", [(64, 4), (33, 3), (2304, 1), (1030, 2)])
@pytest.mark.parametrize("dtype", TYPES)
def test_alike(d, groups, dtype, layout):
    c, _, _ = data(layout, d, groups, dtype, "none", "plain", seed=81)
    top = torch.finfo(TYPES[dtype]).max
    for level in (0.0, 0.1, 1234.567, -59999.0, 1e8, -top, top):
        if abs(level) > top:
            continue
        c["x"].fill_(level)
        value = float(c["x"].view(-1)[0])
        r = fx().group_norm(**c, groups=groups)
        live = torch.ones_like(r.mean, dtype=torch.bool)
        if c["offsets"] is not None:
            live &= (c["offsets"][1:] > c["offsets"][:-1])[:, None]
        assert (r.mean[live] == value).all(), level
        assert torch.allclose(r.rstd, torch.full_like(r.rstd, 1e-5 ** -0.5), rtol=2.0 ** -22), level
        assert torch.equal(r.out, c["bias"].to(r.out.dtype).expand_as(r.out)), level


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("layout", [(2, 300), [300, 0, 90]], ids=str)
def test_lowest_values_beside_others(dtype, layout):
    """Their squares leave float32: the inverse deviation is 0, other groups are what they were."""
    c, _, groups = data(layout, 64, 4, dtype, "none", "plain", seed=82)
    clean = fx().group_norm(**c, groups=groups)
    rows = c["x"].view(-1, 64)
    rows[3:7, 16:32] = torch.finfo(TYPES[dtype]).min
    rows[200, 17] = torch.finfo(TYPES[dtype]).min
    r = fx().group_norm(**c, groups=groups)
    hit = torch.zeros_like(r.rstd, dtype=torch.bool)
    hit[0, 1] = True
    assert (r.rstd[hit] == 0).all() and torch.isfinite(r.mean).all() and torch.isfinite(r.out.float()).all()
    assert torch.equal(r.rstd[~hit], clean.rstd[~hit]) and torch.equal(r.mean[~hit], clean.mean[~hit])
