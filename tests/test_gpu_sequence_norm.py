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
