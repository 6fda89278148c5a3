"""Sizes, types and alignments at which the sequence operators take the kernels of ordinary calls:
whole 16-byte rows of B and C, time cut into several chunks, several lanes per channel where there are
channels enough, runs of many tokens.  Compared with 64-bit forms as in test_gpu_sequence.py, where
sizes are large on some sequences or channels."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import seqref  # noqa: E402
from test_gpu_sequence import (TYPES, close, count, d64, fx, lead_of, near, packing,  # noqa: E402
                               randn)

pytestmark = pytest.mark.gpu

SCAN_INPUTS = ("u", "delta", "A", "B", "C", "D", "z", "delta_bias")


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__

    __graft_entry__.build()


def scan_data(layout, d, n, groups, dtype, gate=True, initial=True, seed=0):
    """All rows on 16-byte boundaries: u and z halves of one tensor, B and C columns of another."""
    rng = np.random.default_rng(seed)
    lead = lead_of(layout)
    xz = randn(rng, *lead, 2 * d, dtype=dtype)
    bc = randn(rng, *lead, 8 + 2 * groups * n, dtype=dtype)
    return dict(u=xz[..., :d], z=xz[..., d:] if gate else None,
                delta=randn(rng, *lead, d, dtype=dtype, scale=0.7),
                A=-torch.exp(randn(rng, d, n, scale=0.5)) * torch.arange(1, n + 1, device="cuda"),
                B=bc[..., 8:8 + groups * n].unflatten(-1, (groups, n)),
                C=bc[..., 8 + groups * n:].unflatten(-1, (groups, n)),
                D=randn(rng, d), delta_bias=randn(rng, d) - 2.0, softplus=True,
                initial_state=randn(rng, count(layout), d, n) if initial else None,
                offsets=packing(layout) if isinstance(layout, list) else None)


def part(c, seqs=slice(None), chans=slice(None)):
    """The call's inputs of some sequences (of a dense batch) and channels (of one group)."""
    r = dict(c)
    packed = c["offsets"] is not None
    for k in ("u", "delta", "z", "B", "C"):
        if c[k] is not None:
            r[k] = c[k] if packed else c[k][seqs]
            if k not in ("B", "C"):
                r[k] = r[k][..., chans]
    for k in ("A", "D", "delta_bias"):
        r[k] = c[k][chans]
    if c["initial_state"] is not None:
        r["initial_state"] = c["initial_state"][slice(None) if packed else seqs][:, chans]
    return r


def scan_ref(c):
    return seqref.scan(*(d64(c[k]) for k in SCAN_INPUTS), True, d64(c["initial_state"]),
                       c["offsets"].cpu() if c["offsets"] is not None else None, magnitude=True)


# d, n, groups, dtype, gate, initial
WHOLE = [(128, 16, 1, "bf16", True, True), (64, 16, 2, "f32", False, False),
         (96, 8, 1, "bf16", True, False), (32, 8, 2, "f16", True, True), (40, 4, 1, "f32", True, True),
         (64, 12, 1, "f32", True, True), (64, 32, 1, "bf16", True, True), (32, 32, 2, "f32", False, False),
         (32, 64, 1, "f16", True, False), (16, 128, 1, "bf16", True, True), (16, 128, 1, "f32", True, True)]


@pytest.mark.parametrize("layout", [(2, 7), (1, 300), (2, 150), [64, 1, 130, 0, 63, 70]], ids=str)
@pytest.mark.parametrize("case", WHOLE, ids=str)
def test_scan_whole_rows(layout, case):
    d, n, groups, dtype, gate, initial = case
    c = scan_data(layout, d, n, groups, TYPES[dtype], gate, initial)
    out, final = fx().selective_scan(**c, return_state=True)
    ref, rfinal, size = scan_ref(c)
    close(out, ref, size)
    near(final, rfinal)


@pytest.mark.parametrize("layout", [(2, 20), (1, 300), [64, 1, 130, 0, 63, 70]], ids=str)
@pytest.mark.parametrize("case", WHOLE, ids=str)
def test_scan_backward_whole_rows(layout, case):
    d, n, groups, dtype, gate, initial = case
    c = scan_data(layout, d, n, groups, TYPES[dtype], gate, initial, seed=1)
    rng = np.random.default_rng(2)
    dout = randn(rng, *c["u"].shape, dtype=TYPES[dtype])
    dfinal = randn(rng, count(layout), d, n) if initial else None
    got = fx().selective_scan_backward(dout, **c, dfinal_state=dfinal)
    names = [k for k in (*SCAN_INPUTS, "initial_state") if c[k] is not None]
    v = {k: d64(c[k]).requires_grad_(True) for k in names}
    out, final = seqref.scan(*(v.get(k) for k in SCAN_INPUTS), True, v.get("initial_state"),
                             c["offsets"].cpu() if c["offsets"] is not None else None)
    loss = (out * d64(dout)).sum()
    if dfinal is not None:
        loss = loss + (final * d64(dfinal)).sum()
    for k, ref in zip(names, torch.autograd.grad(loss, list(v.values()))):
        near(getattr(got, "d" + k), ref, k)
    again = fx().selective_scan_backward(dout, **c, dfinal_state=dfinal)
    for a, b in zip(got, again):
        assert a is None or torch.equal(a, b)


@pytest.mark.parametrize("d,n,dtype", [(128, 16, "bf16"), (128, 16, "f32"), (128, 8, "bf16"),
                                       (128, 8, "f16"), (120, 13, "f32"), (127, 16, "bf16"),
                                       (126, 5, "f32"), (121, 8, "f16")])
@pytest.mark.parametrize("length,gate", [(40, True), (33, False), (16, True), (3, False)])
def test_scan_lanes_for_many_channels(d, n, dtype, length, gate):
    """160 sequences: blocks enough with two lanes for each channel, and time is not cut."""
    c = scan_data((160, length), d, n, 1, TYPES[dtype], gate, True, seed=3)
    out, final = fx().selective_scan(**c, return_state=True)
    some = [0, 77, 159]
    ref, rfinal, size = scan_ref(part(c, seqs=some))
    close(out[some], ref, size)
    near(final[some], rfinal)


@pytest.mark.parametrize("n,dtype", [(16, "bf16"), (8, "f32")])
def test_scan_lanes_for_one_packed_row(n, dtype):
    layout = [5, 0, 16, 1, 30]
    c = scan_data(layout, 32 * 620, n, 1, TYPES[dtype], True, True, seed=4)
    out, final = fx().selective_scan(**c, return_state=True)
    some = [0, 1, 31, 32, 9999, 32 * 620 - 1]
    ref, rfinal, size = scan_ref(part(c, chans=some))
    close(out[..., some], ref, size)
    near(final[:, some], rfinal)


@pytest.mark.parametrize("d,n,dtype", [(1024, 16, "bf16"), (1024, 8, "f32")])
def test_scan_backward_of_a_batch(d, n, dtype):
    """20 sequences of 200 tokens, eight channel tiles: gradients that cross channels are partial
    sums of all tiles, and are compared for two sequences that alone have an output gradient."""
    c = scan_data((20, 200), d, n, 1, TYPES[dtype], True, False, seed=5)
    some = [3, 19]
    dout = torch.zeros_like(c["u"])
    dout[some] = randn(np.random.default_rng(6), 2, 200, d, dtype=TYPES[dtype])
    got = fx().selective_scan_backward(dout, **c)
    p = part(c, seqs=some)
    names = [k for k in SCAN_INPUTS if c[k] is not None]
    v = {k: d64(p[k]).requires_grad_(True) for k in names}
    out, _ = seqref.scan(*(v.get(k) for k in SCAN_INPUTS), True, None, None)
    grads = torch.autograd.grad((out * d64(dout[some])).sum(), list(v.values()))
    for k, ref in zip(names, grads):
        mine = getattr(got, "d" + k)
        near(mine if k in ("A", "D", "delta_bias") else mine[some], ref, k)


# ---- short convolution: runs of many tokens ---------------------------------------------------


def conv64(x, w, b, silu, initial, offsets):
    """seqref.conv in whole tensors."""
    outs, finals, width = [], [], w.shape[1]
    for q, span in enumerate(seqref.spans(x, offsets)):
        xs = seqref.cut(x, span)
        head = initial[q] if initial is not None else x.new_zeros(width - 1, x.shape[-1])
        full = torch.cat([head, xs])
        p = b + sum(w[:, k] * full[k:k + xs.shape[0]] for k in range(width))
        outs.append(p * torch.sigmoid(p) if silu else p)
        finals.append(full[full.shape[0] - (width - 1):])
    return (torch.cat(outs) if offsets is not None else torch.stack(outs)), torch.stack(finals)


LONG = [(1, 12000), (4, 3000), [3, 0, 1, 700, 64, 5000, 65, 6167]]


def long_conv(layout, d, w, dtype, seed=0):
    rng = np.random.default_rng(seed)
    c = dict(x=randn(rng, *lead_of(layout), d, dtype=dtype), weight=randn(rng, d, w, scale=w ** -0.5),
             bias=randn(rng, d, scale=0.3),
             initial_state=randn(rng, count(layout), w - 1, d, dtype=dtype),
             offsets=packing(layout) if isinstance(layout, list) else None)
    some = [0, 1, 2, 3, 4, 127, 128, 1000, d - 1]
    small = dict(x=d64(c["x"][..., some]), weight=d64(c["weight"][some]), bias=d64(c["bias"][some]),
                 initial_state=d64(c["initial_state"][..., some]))
    return c, some, small, c["offsets"].cpu() if c["offsets"] is not None else None


@pytest.mark.parametrize("layout", LONG, ids=str)
@pytest.mark.parametrize("d,w,dtype", [(2000, 4, "bf16"), (2000, 4, "f32"), (2001, 3, "f16"), (2000, 8, "bf16")])
def test_conv_long_runs(layout, d, w, dtype):
    c, some, s, offsets = long_conv(layout, d, w, TYPES[dtype])
    out, final = fx().causal_conv(**c, silu=True, return_state=True)
    ref, rfinal = conv64(s["x"], s["weight"], s["bias"], True, s["initial_state"], offsets)
    size, _ = conv64(*(s[k].abs() for k in ("x", "weight", "bias")), False, s["initial_state"].abs(), offsets)
    close(out[..., some], ref, size)
    assert torch.equal(d64(final[..., some]), rfinal)


@pytest.mark.parametrize("layout", LONG, ids=str)
@pytest.mark.parametrize("d,w,dtype", [(2000, 4, "bf16"), (2000, 4, "f32"), (2001, 3, "f32"), (2000, 8, "f16")])
def test_conv_backward_long_runs(layout, d, w, dtype):
    c, some, s, offsets = long_conv(layout, d, w, TYPES[dtype], seed=1)
    rng = np.random.default_rng(2)
    dout = randn(rng, *c["x"].shape, dtype=TYPES[dtype])
    dfinal = randn(rng, count(layout), w - 1, d, dtype=TYPES[dtype])
    got = fx().causal_conv_backward(dout, silu=True, dfinal_state=dfinal, **c)
    v = {k: t.requires_grad_(True) for k, t in s.items()}
    out, final = conv64(v["x"], v["weight"], v["bias"], True, v["initial_state"], offsets)
    loss = (out * d64(dout[..., some])).sum() + (final * d64(dfinal[..., some])).sum()
    dx, dw, db, di = torch.autograd.grad(loss, list(v.values()))
    near(got.dx[..., some], dx)
    near(got.dweight[some], dw)
    near(got.dbias[some], db)
    near(got.dinitial_state[..., some], di)


def test_conv_full_runs():
    """Rounds of blocks enough that runs are of the greatest length."""
    c, some, s, _ = long_conv((8, 4096), 2048, 4, torch.bfloat16, seed=3)
    out, final = fx().causal_conv(**c, silu=True, return_state=True)
    ref, rfinal = conv64(s["x"], s["weight"], s["bias"], True, s["initial_state"], None)
    size, _ = conv64(*(s[k].abs() for k in ("x", "weight", "bias")), False, s["initial_state"].abs(), None)
    close(out[..., some], ref, size)
    assert torch.equal(d64(final[..., some]), rfinal)
