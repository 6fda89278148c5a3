"""Batches of nothing: no rows, no sequences.  Outputs are as empty, gradients of parameters 0."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

FP8 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__

    __graft_entry__.build()


@pytest.mark.parametrize("shape", [(0, 64), (2, 0, 64), (0, 3, 64)])
@pytest.mark.parametrize("more", [{}, dict(out_dtype=FP8), dict(out_dtype=FP8, group=32)])
def test_norm_of_no_rows(shape, more):
    import fft_signal_processing_gb300 as fx

    x = torch.empty(*shape, device="cuda", dtype=torch.bfloat16)
    w = torch.ones(64, device="cuda")
    r = fx.residual_norm(x, w, residual=x, **more)
    assert r.out.shape == shape and r.residual.shape == shape
    assert (r.scale is None) == (not more)
    if more:
        assert r.scale.shape == (*shape[:-1], 2 if "group" in more else 1)
    r = fx.residual_norm(x, w, residual=x, inplace_residual=True)
    assert r.residual is x
    g = fx.residual_norm_backward(x, x, w, dresidual=x)
    assert g.dx.shape == shape and torch.equal(g.dweight, torch.zeros_like(w))
    wide = fx.residual_norm_backward(x, x.float(), w)
    assert wide.dresidual.shape == shape and wide.dx.dtype == torch.bfloat16
