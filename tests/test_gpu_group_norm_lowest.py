"""Group norm of single rows that hold the lowest value of their type in some places, as masked ones do: mean
and outputs are finite, the inverse deviation is 0 (squares leave float32), other groups and rows are the
same bits."""
import pytest

torch = pytest.importorskip("torch")

from test_gpu_group_norm import TYPES, data, fx  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__

    __graft_entry__.build()


@pytest.mark.parametrize("places", [1, 2, 15, 16])
@pytest.mark.parametrize("d,each,strides", [(64, 16, "plain"), (48, 16, "odd"), (1024, 512, "plain"), (30, 30, "plain")])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_lowest_values(dtype, d, each, strides, places):
    c, _, groups = data(40, d, d // each, dtype, "none", strides, seed=83)
    clean = fx().group_norm(**c, groups=groups)
    low = torch.finfo(TYPES[dtype]).min
    c["x"][17, :places] = low
    r = fx().group_norm(**c, groups=groups)
    hit = torch.zeros_like(r.rstd, dtype=torch.bool)
    hit[17, 0] = True
    if places == each:  # all alike
        assert float(r.mean[17, 0]) == float(torch.tensor(low).to(TYPES[dtype]))
    else:
        assert float(r.rstd[17, 0]) == 0.0
        want = float(c["x"][17, :each].double().mean())
        assert abs(float(r.mean[17, 0]) - want) <= 2.0 ** -20 * abs(want)
    assert torch.isfinite(r.out.float()).all()
    assert torch.equal(r.mean[~hit], clean.mean[~hit]) and torch.equal(r.rstd[~hit], clean.rstd[~hit])
    wide = hit.repeat_interleave(each, 1)
    assert torch.equal(r.out[~wide], clean.out[~wide])
    if places < each:
        assert torch.equal(r.out[wide], c["bias"][:each].to(r.out.dtype))
