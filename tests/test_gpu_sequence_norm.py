"""Residual norm at the ends of its range and over many rows for each block (64-bit forms and derived
tolerances of test_gpu_sequence.py)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import seqref  # noqa: E402
from test_gpu_sequence import FEW, TYPES, close, d64, fx, near, randn  # noqa: E402

pytestmark = pytest.mark.gpu

FP8 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__

    __graft_entry__.build()


def check_8bit(got, x, residual, w, group):
    """Scales, and values within half a step of e4m3 of the exact quotient, as in test_norm_8bit."""
    y, _ = seqref.norm(d64(x), d64(residual), d64(w), 1e-6)
    q, scale = seqref.e4m3(y, group)
    close(got.scale, scale, scale)
    s = scale.repeat_interleave(group, 1)[:, :x.shape[1]] if group else scale
    v = y / torch.where(s > 0, s, torch.ones_like(s))
    out = got.out.float().cpu().double()
    err = (out - v).abs()
    assert (err <= torch.maximum(v.abs() * 2.0 ** -4, torch.tensor(2.0 ** -10)) * (1 + 2.0 ** -10)
            + FEW * v.abs()).all()
    # the definition's value, but where that stands on a rounding's edge
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
    edge = ((v.abs() / step).frac() - 0.5).abs() * step <= FEW * v.abs()
    assert ((out == q) | edge).all()


@pytest.mark.parametrize("d", [256, 100, 5000])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("group", [0, 32, 128])
def test_8bit_of_tiny_rows(d, dtype, group):
    """Rows whose largest value's 448th part has no float32 inverse, next to rows that are not tiny,
    and (of grouped scales) tiny groups in a row that is not."""
    rng = np.random.default_rng(d)
    x = randn(rng, 6, d, dtype=TYPES[dtype])
    x[1], x[3] = x[1] * 1e-37, x[3] * 2e-36
    x[4, :128] *= 1e-37
    x[5, 128:] = 0
    w = torch.ones(d, device="cuda")
    got = fx().residual_norm(x, w, out_dtype=FP8, group=group)
    if group == 0:
        keep = [0, 1, 2, 3, 5]  # in row 4 the tiny values are 0 next to the largest
        check_8bit(got._replace(out=got.out[keep], scale=got.scale[keep]), x[keep], None, w, 0)
    else:
        check_8bit(got, x, None, w, group)
    assert (got.out[1].float().abs().max() == 448.0) and (got.out[3].float().abs().max() == 448.0)


# Rows for three and more rounds of the blocks, the last one ragged: later rows wait in shared
# memory while a row is at hand, and sums and maxima take turns in two places.
MANY = [(5000, 128), (5000, 131), (1000, 4096), (1001, 4095), (500, 8200), (500, 8201), (400, 16384)]


@pytest.mark.parametrize("rows,d", MANY)
@pytest.mark.parametrize("dtype,res", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32"), ("f16", None)])
def test_many_rows(rows, d, dtype, res):
    rng = np.random.default_rng(d)
    x = randn(rng, rows, d, dtype=TYPES[dtype])
    r = randn(rng, rows, d, dtype=TYPES[res], scale=3.0) if res else None
    w = randn(rng, d)
    got = fx().residual_norm(x, w, residual=r)
    ref, total = seqref.norm(d64(x), d64(r), d64(w), 1e-6)
    close(got.out, ref, ref.abs())
    if res:
        close(got.residual, total, total.abs())
        again = fx().residual_norm(x, w, residual=r, inplace_residual=True)
        assert torch.equal(again.out, got.out) and torch.equal(r, got.residual)


@pytest.mark.parametrize("rows,d", MANY)
@pytest.mark.parametrize("dtype,group", [("bf16", 0), ("bf16", 128), ("f32", 32), ("f16", 64)])
def test_many_rows_8bit(rows, d, dtype, group):
    rng = np.random.default_rng(d + 1)
    x, r = randn(rng, rows, d, dtype=TYPES[dtype]), randn(rng, rows, d, scale=2.0)
    r *= torch.exp2(torch.arange(rows, device="cuda") % 7 - 3.0)[:, None]  # rows unlike their neighbours
    w = randn(rng, d)
    got = fx().residual_norm(x, w, residual=r, out_dtype=FP8, group=group)
    check_8bit(got, x, r, w, group)


@pytest.mark.parametrize("rows,d", [(5000, 320), (5000, 131), (1000, 3000), (700, 4096), (400, 8200),
                                    (400, 9001), (400, 16384)])
@pytest.mark.parametrize("dtype,res,extra", [("bf16", "f32", True), ("bf16", "bf16", False),
                                             ("f32", "f32", True)])
def test_many_rows_backward(rows, d, dtype, res, extra):
    rng = np.random.default_rng(d + 2)
    r, dout = randn(rng, rows, d, dtype=TYPES[res], scale=2.0), randn(rng, rows, d, dtype=TYPES[dtype])
    w, dres = randn(rng, d), randn(rng, rows, d, dtype=TYPES[res]) if extra else None
    got = fx().residual_norm_backward(dout, r, w, dresidual=dres)
    rr, ww = d64(r).requires_grad_(True), d64(w).requires_grad_(True)
    y, _ = seqref.norm(rr, None, ww, 1e-6)
    loss = (y * d64(dout)).sum() + ((rr * d64(dres)).sum() if extra else 0.0)
    dr, dw = torch.autograd.grad(loss, (rr, ww))
    for mine, ref in ((got.dresidual, dr), (got.dx, dr)):
        near(mine, ref)
        for part in (0, 1, 2):  # every round by itself: the last rows are few
            near(mine[part * rows // 3:(part + 1) * rows // 3], ref[part * rows // 3:(part + 1) * rows // 3])
        near(mine[-5:], ref[-5:])
    near(got.dweight, dw, "dweight")
    again = fx().residual_norm_backward(dout, r, w, dresidual=dres)
    assert torch.equal(again.dweight, got.dweight) and torch.equal(again.dx, got.dx)
