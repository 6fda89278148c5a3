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


@pytest.mark.parametrize("packed", [False, True])
def test_no_sequences(packed):
    import fft_signal_processing_gb300 as fx

    d, n = 24, 6
    x = torch.empty(*((0,) if packed else (0, 5)), d, device="cuda")
    offsets = torch.zeros(1, dtype=torch.int64, device="cuda") if packed else None
    w, bias = torch.ones(d, 4, device="cuda"), torch.ones(d, device="cuda")
    init = torch.empty(0, 3, d, device="cuda")
    out, final = fx.causal_conv(x, w, bias, initial_state=init, offsets=offsets, return_state=True)
    assert out.shape == x.shape and final.shape == init.shape
    g = fx.causal_conv_backward(x, x, w, bias, initial_state=init, offsets=offsets, dfinal_state=init)
    assert g.dx.shape == x.shape and g.dinitial_state.shape == init.shape
    assert torch.equal(g.dweight, w * 0) and torch.equal(g.dbias, bias * 0)

    A, B = -torch.ones(d, n, device="cuda"), torch.empty(*x.shape[:-1], 2, n, device="cuda")
    h = torch.empty(0, d, n, device="cuda")
    c = dict(u=x, delta=x, A=A, B=B, C=B, D=bias, z=x, delta_bias=bias, softplus=True,
             initial_state=h, offsets=offsets)
    out, final = fx.selective_scan(**c, return_state=True)
    assert out.shape == x.shape and final.shape == h.shape
    g = fx.selective_scan_backward(x, **c, dfinal_state=h)
    for k in ("du", "ddelta", "dz"):
        assert getattr(g, k).shape == x.shape
    assert g.dB.shape == B.shape and g.dC.shape == B.shape and g.dinitial_state.shape == h.shape
    assert torch.equal(g.dA, A * 0) and torch.equal(g.dD, bias * 0)
    assert torch.equal(g.ddelta_bias, bias * 0)
    with pytest.raises(fx.GbfftError):  # what is wrong all the same is refused
        fx.causal_conv(x, torch.ones(d, 9, device="cuda"), offsets=offsets)
    if packed:
        with pytest.raises(ValueError):
            fx.causal_conv(torch.ones(3, d, device="cuda"), w, offsets=offsets)


def test_steps_of_no_sequences():
    import fft_signal_processing_gb300 as fx

    d, n = 24, 6
    x, none = torch.empty(0, d, device="cuda"), torch.empty(0, dtype=torch.int64, device="cuda")
    pool = torch.ones(2, 3, d, device="cuda")
    for slots in (None, none):
        y = fx.causal_conv_step(pool, x, torch.ones(d, 4, device="cuda"), slots=slots)
        assert y.shape == x.shape and (pool == 1).all()
    pool = torch.ones(2, d, n, device="cuda")
    B, out = torch.empty(0, n, device="cuda"), torch.empty_like(x)
    y = fx.selective_scan_step(pool, x, x, -torch.ones(d, n, device="cuda"), B, B, slots=none,
                               slots_out=none, out=out)
    assert y is out and (pool == 1).all()
