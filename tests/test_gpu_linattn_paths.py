"""Linear attention along the paths that ordinary calls take: the tcgen05 kernel with time cut, shared
heads, several tiles of columns and sequences that end anywhere in its chunks; the same shapes off
16-byte boundaries; both directions next to the group norm that follows the heads.  Tolerances as in
test_gpu_linattn.py."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import attnref  # noqa: E402
from test_gpu_linattn import (STATE, TERM, close, d64, data, fx, gradients, near, packing, randn,  # noqa: E402
                              reference)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__

    __graft_entry__.build()


# sequences that end at, before and behind a chunk's last token, in the middle of a cut's segment
EDGES = [127, 1, 128, 129, 0, 255, 256, 257, 3, 500]


@pytest.mark.parametrize("layout", [EDGES, (1, 1000), (3, 129)], ids=str)
@pytest.mark.parametrize("shape", [(2, 2, 128, 128), (4, 1, 64, 128), (2, 2, 128, 64), (2, 1, 64, 64), (1, 1, 8, 8),
                                   (1, 1, 104, 120), (1, 1, 128, 256), (2, 2, 72, 200)], ids=str)
def test_tensor_core_chunks(layout, shape):
    c = data(layout, *shape, "bf16", True, "plain", seed=1)
    out, final = fx().linear_attention(**c, return_state=True)
    ref, rfinal, size, total = reference(c, magnitude=True)
    close(out, ref, size, TERM[torch.bfloat16], "out")
    close(final, rfinal, total, STATE, "final")
    rng = np.random.default_rng(2)
    dout, dfinal = randn(rng, *c["v"].shape, dtype=torch.bfloat16), randn(rng, *final.shape)
    r = fx().linear_attention_backward(dout, **c, dfinal_state=dfinal)
    for name, got, want in zip(r._fields, r, gradients(c, dout, dfinal)):
        near(got, want, name)
    fx().linear_attention_check()


@pytest.mark.parametrize("what", ["q", "k", "v", "dout"])
def test_rows_off_16_byte_boundaries(what):
    """One tensor off them: another kernel, the same result within what both are good to."""
    c = data((2, 300), 2, 2, 64, 64, "bf16", True, "plain", seed=3)
    dout = randn(np.random.default_rng(4), *c["v"].shape, dtype=torch.bfloat16)

    def moved(t):
        wide = torch.zeros(*t.shape[:-1], t.shape[-1] + 1, dtype=t.dtype, device="cuda")
        wide[..., 1:] = t
        return wide[..., 1:]

    if what == "dout":
        dout = moved(dout)
    else:
        c[what] = moved(c[what])
    out, final = fx().linear_attention(**c, return_state=True)
    ref, rfinal, size, total = reference(c, magnitude=True)
    close(out, ref, size, TERM[torch.bfloat16], "out")
    close(final, rfinal, total, STATE, "final")
    r = fx().linear_attention_backward(dout, **c)
    for name, got, want in zip(r._fields, r, gradients(c, dout)):
        near(got, want, name)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_states_of_long_sequences(dtype):
    """A state that is kept for thousands of tokens stays good to float32: three pieces of 2^-24 each and
    a rounding of 2^-24 for every chunk, which have no one sign; 2^-20 of the norm is above both."""
    c = data((1, 6000), 1, 1, 64, 64, dtype, False, "plain", seed=5, rate=1e-3)
    _, final = fx().linear_attention(**c, return_state=True)
    _, want = reference(c)
    assert (d64(final) - want).norm() <= 2.0 ** -20 * want.norm()
    dout = randn(np.random.default_rng(6), *c["v"].shape, dtype=c["v"].dtype)
    c["initial_state"] = torch.zeros_like(final)
    r = fx().linear_attention_backward(dout, **c)
    want = gradients(c, dout)
    assert (d64(r.dinitial_state) - want[4]).norm() <= 2.0 ** -20 * want[4].norm()
    for name, got, ref in zip(r._fields[:4], r, want):
        near(got, ref, name)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_not_finite_in_long_sequences(dtype):
    """An infinite value in one column of v: that column from its token on, in its sequence only."""
    c = data([300, 400], 2, 2, 64, 64, dtype, False, "plain", seed=7)
    clean = fx().linear_attention(**c)
    ref, _, size, _ = reference(c, magnitude=True)
    # Other values are those without it: both within the bound of the definition, so apart by twice that at
    # most (a warp that meets such a value sums in another order).
    apart = 2 * (TERM[clean.dtype] * size + 2.0 ** -24 * ref.abs())
    for at in (0, 31, 127, 128, 200, 299):
        v = c["v"].clone()
        v[at, 0, 5] = float("inf")
        out = fx().linear_attention(**{**c, "v": v})
        bad = torch.zeros_like(out, dtype=torch.bool)
        bad[at:300, 0, 5] = True
        assert not torch.isfinite(out[bad]).any(), at
        same = torch.equal(out[~bad], clean[~bad]) if dtype == "bf16" else bool(
            ((d64(out) - d64(clean)).abs() <= apart)[~bad.cpu()].all())
        assert same, at
    dout = randn(np.random.default_rng(8), *c["v"].shape, dtype=c["v"].dtype)
    good = fx().linear_attention_backward(dout, **c)
    q = c["q"].clone()
    q[350, 1, 9] = float("nan")
    r = fx().linear_attention_backward(dout, **{**c, "q": q})
    # dk and the state's gradient of this head take q[350] for the tokens up to it, in its second sequence
    assert torch.isnan(r.dk[300:351, 1, 9]).all()
    for got, want in ((r.dk[351:], good.dk[351:]), (r.dk[:300], good.dk[:300]), (r.dk[:, 0], good.dk[:, 0]),
                      (r.dq, good.dq)):
        if dtype == "bf16":
            assert torch.equal(got, want)
        else:  # both within 2^-16 of the formula by norm
            assert (d64(got) - d64(want)).norm() <= 2.0 ** -15 * d64(want).norm()


def test_two_streams_at_once():
    """Calls on two streams, with workspaces of their own, next to each other."""
    cs = [data((2, 900), 2, 2, 128, 128, "bf16", True, "plain", seed=s) for s in (9, 10)]
    douts = [randn(np.random.default_rng(s), *cs[0]["v"].shape, dtype=torch.bfloat16) for s in (11, 12)]
    want = [(fx().linear_attention(**c, return_state=True), fx().linear_attention_backward(d, **c))
            for c, d in zip(cs, douts)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cs]
    got = []
    for _ in range(3):
        got = [(fx().linear_attention(**c, return_state=True, stream=s),
                fx().linear_attention_backward(d, **c, stream=s)) for c, d, s in zip(cs, douts, streams)]
    torch.cuda.synchronize()
    for (o, r), (wo, wr) in zip(got, want):
        assert all(torch.equal(a, b) for a, b in zip((*o, *r), (*wo, *wr)))


@pytest.mark.parametrize("offsets", [[0, 90, 40, 200], [0, 50, 50, 500], [5, 60, 100, 150], [0, 0, 0, 0], [-7, 20, 90, 200]],
                         ids=str)
@pytest.mark.parametrize("dtype,dim", [("bf16", 64), ("f32", 24)])
def test_offsets_that_break_the_rule(offsets, dtype, dim):
    """Undefined outputs, but nothing outside them is written: outputs and states inside larger ones."""
    c = data([60, 70, 70], 2, 2, dim, dim, dtype, True, "plain", seed=13)
    c["offsets"] = torch.tensor(offsets, device="cuda")
    whole = torch.full((400, 2, dim), 7.0, dtype=c["v"].dtype, device="cuda")
    fx().linear_attention(**c, out=whole[100:300], return_state=True)
    dout = torch.ones_like(c["v"])
    r = fx().linear_attention_backward(dout, **c, dfinal_state=torch.ones_like(c["initial_state"]))
    torch.cuda.synchronize()
    assert (whole[:100] == 7.0).all() and (whole[300:] == 7.0).all()
    assert r.dq.shape == c["q"].shape
    x = c["v"].flatten(1)
    big = torch.full((400, x.shape[1]), 7.0, dtype=x.dtype, device="cuda")
    f = fx().group_norm(x, 2, offsets=c["offsets"], out=big[100:300])
    fx().group_norm_backward(x, x, f.mean, f.rstd, offsets=c["offsets"])
    torch.cuda.synchronize()
    assert (big[:100] == 7.0).all() and (big[300:] == 7.0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("packed", [False, True])
def test_layer_gradients(dtype, packed):
    """Attention, the norm of every head and the gate, run together, and the gradients of all of it."""
    heads, groups, dk, dv = 4, 2, 32, 64
    layout = [70, 0, 130] if packed else (2, 140)
    c = data(layout, heads, groups, dk, dv, dtype, True, "plain", seed=14)
    rng = np.random.default_rng(15)
    z = randn(rng, *c["v"].shape[:-2], heads * dv, dtype=c["v"].dtype)
    w, b = randn(rng, heads * dv) + 1.0, randn(rng, heads * dv)
    dy = randn(rng, *z.shape, dtype=z.dtype)
    rows = lambda t: t.reshape(-1, heads * dv)  # noqa: E731

    out = fx().linear_attention(**c)
    n = fx().group_norm(rows(out), heads, w, b, z=rows(z))
    dn = fx().group_norm_backward(rows(dy), rows(out), n.mean, n.rstd, w, b, z=rows(z))
    da = fx().linear_attention_backward(dn.dx.view(out.shape), **c)

    names = ("q", "k", "v", "decay", "initial_state")
    leaves = [d64(c[x]).requires_grad_(True) for x in names] + [d64(t).requires_grad_(True) for t in (w, b, z)]
    o = c["offsets"].cpu() if packed else None
    ref, _ = attnref.attention(*leaves[:4], dk ** -0.5, leaves[4], o)
    y, _, _ = attnref.group_norm(rows(ref)[:, None], heads, leaves[5], leaves[6], rows(leaves[7])[:, None], False,
                                 1e-5, None)
    want = torch.autograd.grad((y[:, 0] * d64(rows(dy))).sum(), leaves)
    # the attention's outputs and their gradients are rounded on the way: 2^-8 and 2^-11 of their terms, which
    # the norm's gradient subtracts from each other; a few of them by norm
    more = 0.0 if dtype == "f32" else 8 * {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}[dtype]
    near(n.out, y[:, 0].detach(), "y", more)
    for name, got, ref in zip((*names, "weight", "bias", "z"), (*da, dn.dweight, dn.dbias, dn.dz.view(z.shape)), want):
        near(got, ref, name, more)
