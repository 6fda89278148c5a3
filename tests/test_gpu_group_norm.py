"""GPU parity of the group norm (channels last, SiLU, gate; dense, packed, token by token) and its
gradients with the definition in 64 bits.

Tolerances.  An output of type T carries one rounding, UNIT[T] of its own value.  Before it stand
float32 operations, each off by a few units of 2^-24 of its terms: FEW = 64 * 2^-24 of |x| rstd |w| + |b|
times what the activation makes of it bounds the chain (means and deviations are good to the sums of
at most 128 tokens per thread, joined in 64 bits).  Gradients are compared by norms: 2^-16 for
float32 results, twice UNIT[T] for rounded ones.  Those of the parameters are sums over tokens whose
terms may cancel: adding float32 numbers in any order of partial sums, at most 16 additions deep in a
thread and 2^8 parts, is off by (16 + 8) 2^-24 of the sum of their absolute values; PARTS = 2^-19 is
above that, and |dy| is at most 1.1 |dout| |z sigmoid(z)|, 1.1 being the steepest SiLU.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import attnref  # noqa: E402

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
UNIT = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
FEW = 64 * 2.0 ** -24
SUMS = 2.0 ** -16
PARTS = 2.0 ** -19
# rows by themselves, (sequences, tokens), or packed lengths
LAYOUTS = [7, 700, (1, 1), (3, 5), (2, 300), (1, 4000), [5], [0, 1, 0, 2, 31, 64, 0], [300, 0, 2, 1400]]
# channels, groups, type, activation, strides
SHAPES = [(64, 4, "bf16", "gate", "half"), (256, 1, "bf16", "silu", "plain"), (96, 3, "bf16", "none", "plain"),
          (30, 6, "bf16", "gate", "odd"), (5, 5, "f16", "silu", "odd"), (1024, 2, "f16", "gate", "half"),
          (1030, 1, "f32", "silu", "plain"), (330, 6, "f32", "gate", "odd"), (2304, 1, "bf16", "silu gate", "half"),
          (4096, 32, "bf16", "gate", "half"), (1, 1, "f32", "none", "plain"), (520, 65, "f32", "silu", "plain")]


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__

    __graft_entry__.build()


def fx():
    import fft_signal_processing_gb300 as m

    return m


def randn(rng, *shape, dtype=torch.float32, scale=1.0):
    return (torch.from_numpy(rng.standard_normal(shape)) * scale).to(dtype).cuda()


def d64(t):
    return t.detach().cpu().double() if t is not None else None


def near(got, ref, what="", more=0.0):
    tol = SUMS if got.dtype == torch.float32 else 2 * UNIT[got.dtype] + SUMS
    g = d64(got)
    assert g.shape == ref.shape, what
    assert torch.isfinite(g).all(), what
    assert (g - ref).norm() <= tol * ref.norm() + more + 1e-30, (what, float((g - ref).norm() / ref.norm()))


def data(layout, d, groups, dtype, act, strides, seed=0, level=1.0, param=None):
    rng = np.random.default_rng(seed)
    lead = (layout,) if isinstance(layout, int) else ((sum(layout),) if isinstance(layout, list) else layout)
    dtype = TYPES[dtype]
    skip = {"plain": 0, "half": d, "odd": 1}[strides]

    def rows():
        base = randn(rng, *lead, d + skip) + level * randn(rng, d + skip)
        return base.to(dtype)[..., skip:]

    offsets = None
    if isinstance(layout, list):
        offsets = torch.from_numpy(np.concatenate([[0], np.cumsum(layout)]).astype(np.int64)).cuda()
    return dict(x=rows(), weight=(randn(rng, d) + 1.0).to(param or torch.float32),
                bias=(0.3 * randn(rng, d)).to(param or torch.float32), z=rows() if "gate" in act else None,
                silu="silu" in act, offsets=offsets), rng, groups


def reference(c, groups, eps=1e-5, leaves=None):
    v = {n: (leaves or {}).get(n, d64(c[n])) for n in ("x", "weight", "bias", "z")}
    flat = c["offsets"] is None and c["x"].dim() == 2
    if flat:
        v["x"], v["z"] = v["x"][:, None], v["z"][:, None] if v["z"] is not None else None
    out, mean, rstd = attnref.group_norm(v["x"], groups, v["weight"], v["bias"], v["z"], c["silu"], eps,
                                         c["offsets"].cpu() if c["offsets"] is not None else None)
    return out[:, 0] if flat else out, mean, rstd


def bound(c, groups, out, mean, rstd):
    """|x| rstd |w| + |b| of every value, times the gate, twice for the activation's own steepness."""
    x = d64(c["x"])
    each = x.shape[-1] // groups
    if c["offsets"] is not None:
        lens = (c["offsets"][1:] - c["offsets"][:-1]).cpu()
        spread = lambda t: t.repeat_interleave(lens, 0)  # noqa: E731
    else:
        spread = (lambda t: t[:, None]) if x.dim() == 3 else (lambda t: t)
    wide = lambda t: spread(t).repeat_interleave(each, -1)  # noqa: E731
    size = (x.abs() + wide(mean.abs())) * wide(rstd) * d64(c["weight"]).abs() + d64(c["bias"]).abs()
    if c["z"] is not None:
        z = d64(c["z"])
        size = size * (z * torch.sigmoid(z)).abs()
    return 2 * size


@pytest.mark.parametrize("layout", LAYOUTS, ids=str)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_forward(layout, shape):
    c, _, groups = data(layout, *shape)
    r = fx().group_norm(**c, groups=groups)
    out, mean, rstd = reference(c, groups)
    tol = UNIT[r.out.dtype] * out.abs() * 1.001 + FEW * bound(c, groups, out, mean, rstd) + (
        2.0 ** -24 if r.out.dtype == torch.float16 else 0.0)
    assert ((d64(r.out) - out).abs() <= tol).all()
    near(r.mean, mean, "mean")
    near(r.rstd, rstd, "rstd")


@pytest.mark.parametrize("layout", [700, (2, 300), [300, 0, 2, 1400]], ids=str)
def test_far_from_zero(layout):
    """Channels at a thousand deviations from zero."""
    c, _, groups = data(layout, 32, 4, "f32", "none", "plain", seed=1, level=0.0)
    c["x"] = c["x"] + 1000.0
    r = fx().group_norm(**c, groups=groups)
    out, mean, rstd = reference(c, groups)
    near(r.mean, mean)
    assert ((d64(r.rstd) - rstd).abs() <= 1e-5 * rstd).all()
    assert ((d64(r.out) - out).abs() <= FEW * bound(c, groups, out, mean, rstd)).all()


def gradients(c, groups, dout):
    leaves = {n: d64(c[n]).requires_grad_(True) for n in ("x", "weight", "bias", "z") if c[n] is not None}
    out, _, _ = reference(c, groups, leaves=leaves)
    g = dict(zip(leaves, torch.autograd.grad((out * d64(dout)).sum(), list(leaves.values()))))
    return [g["x"], g.get("z"), g["weight"], g["bias"]]


@pytest.mark.parametrize("layout", LAYOUTS, ids=str)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_gradients(layout, shape):
    c, rng, groups = data(layout, *shape, seed=2)
    if shape[0] // shape[1] == 1 and layout in (7, 700, (1, 1)):
        pytest.skip("one value for each mean: its gradient is 0 and what roundings leave")
    dout = randn(rng, *c["x"].shape, dtype=c["x"].dtype)
    f = fx().group_norm(**c, groups=groups)
    r = fx().group_norm_backward(dout, c["x"], f.mean, f.rstd, c["weight"], c["bias"], z=c["z"], silu=c["silu"],
                                 offsets=c["offsets"])
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


def test_gradients_against_differences():
    c, rng, groups = data([40, 70], 24, 3, "f32", "silu gate", "plain", seed=3)
    dout = randn(rng, *c["x"].shape)
    f = fx().group_norm(**c, groups=groups)
    r = fx().group_norm_backward(dout, c["x"], f.mean, f.rstd, c["weight"], c["bias"], z=c["z"], silu=True,
                                 offsets=c["offsets"])
    for name, got in zip(("x", "z", "weight", "bias"), r):
        way = d64(randn(rng, *c[name].shape))
        ends = []
        for sign in (1, -1):
            moved = {n: d64(c[n]) for n in ("x", "weight", "bias", "z")}
            moved[name] = moved[name] + sign * 1e-4 * way
            ends.append(float((reference(c, groups, leaves=moved)[0] * d64(dout)).sum()))
        have, size = float((d64(got) * way).sum()), float((d64(got) * way).abs().sum())
        assert abs(have - (ends[0] - ends[1]) / 2e-4) <= 1e-5 * size + 1e-7 * abs(ends[0]), name


@pytest.mark.parametrize("param", ["f32", "bf16"])
def test_parameters(param):
    """Weights of both types, and none."""
    c, rng, groups = data((2, 40), 64, 4, "bf16", "gate", "half", seed=4, param=TYPES[param])
    dout = randn(rng, *c["x"].shape, dtype=c["x"].dtype)
    for use in ((True, True), (True, False), (False, True), (False, False)):
        w = {n: c[n] if u else None for n, u in zip(("weight", "bias"), use)}
        f = fx().group_norm(c["x"], groups, **w, z=c["z"])
        one = {"weight": torch.ones(64), "bias": torch.zeros(64)}
        full = {**c, **{n: (w[n] if w[n] is not None else one[n]) for n in w}}
        out, _, _ = reference(full, groups)
        near(f.out, out)
        r = fx().group_norm_backward(dout, c["x"], f.mean, f.rstd, **w, z=c["z"])
        want = gradients(full, groups, dout)
        near(r.dx, want[0])
        near(r.dz, want[1])
        for got, ref, u in zip(r[2:], want[2:], use):
            assert (got is not None) == u
            if u:
                near(got, ref)


@pytest.mark.parametrize("layout", [700, (2, 300), [300, 0, 2, 1400]], ids=str)
def test_in_place_same_bits_graph_and_stream(layout):
    c, rng, groups = data(layout, 256, 8, "bf16", "silu gate", "plain", seed=5)
    dout = randn(rng, *c["x"].shape, dtype=c["x"].dtype)

    def both(stream=None):
        f = fx().group_norm(**c, groups=groups, stream=stream)
        r = fx().group_norm_backward(dout, c["x"], f.mean, f.rstd, c["weight"], c["bias"], z=c["z"], silu=True,
                                     offsets=c["offsets"], stream=stream)
        return [*f, *r]

    first = both()
    assert all(torch.equal(a, b) for a, b in zip(first, both()))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = both(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, other))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = both()
    for t in captured:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, captured))
    for name in ("x", "z"):
        copy = {**c, name: c[name].clone()}
        out = fx().group_norm(**copy, groups=groups, out=copy[name]).out
        assert out.data_ptr() == copy[name].data_ptr() and torch.equal(out, first[0])


@pytest.mark.parametrize("layout", [(2, 70), 90, [60, 41]], ids=str)
def test_outputs_inside_larger_tensors(layout):
    c, _, groups = data(layout, 40, 5, "bf16", "gate", "half", seed=6)
    want = fx().group_norm(**c, groups=groups).out
    whole = torch.full((*c["x"].shape[:-1], 50), 7.0, dtype=torch.bfloat16, device="cuda")
    fx().group_norm(**c, groups=groups, out=whole[..., 8:48])
    assert torch.equal(whole[..., 8:48], want)
    whole[..., 8:48] = 7.0
    assert (whole == 7.0).all()


def test_empty():
    for shape in ((0, 8), (0, 3, 8), (2, 0, 8)):
        x = torch.zeros(shape, device="cuda")
        f = fx().group_norm(x, 2, torch.ones(8, device="cuda"), torch.ones(8, device="cuda"))
        assert f.out.shape == shape and f.mean.shape == (shape[0], 2)
        assert not f.mean.any() and torch.allclose(f.rstd, torch.full_like(f.rstd, 1e-5 ** -0.5))
        r = fx().group_norm_backward(x, x, f.mean, f.rstd, torch.ones(8, device="cuda"),
                                     torch.ones(8, device="cuda"))
        assert r.dx.shape == shape and not r.dweight.any() and not r.dbias.any()


def test_not_finite_stays_in_its_group():
    for layout in (50, (2, 60), [30, 90]):
        c, _, groups = data(layout, 32, 4, "f32", "silu", "plain", seed=7)
        clean = fx().group_norm(**c, groups=groups).out
        x = c["x"].clone()
        x.view(-1, 32)[20, 9] = float("inf")
        out = fx().group_norm(**{**c, "x": x}, groups=groups).out
        ref, _, _ = reference({**c, "x": x}, groups)
        bad = torch.isnan(ref)
        assert torch.equal(torch.isnan(out).cpu(), bad) and bad.any() and not bad.all()
        assert torch.equal(out[~bad.cuda()], clean[~bad.cuda()])


def test_heads_of_an_attention():
    """The norm of every head behind linear attention, as a layer runs them: prompts, then tokens."""
    rng = np.random.default_rng(8)
    b, length, heads, dk, dv = 2, 90, 4, 32, 64
    q, k = randn(rng, b, length, heads, dk), randn(rng, b, length, heads, dk)
    v, z = randn(rng, b, length, heads, dv), randn(rng, b, length, heads * dv)
    decay = -torch.rand(b, length, heads, device="cuda")
    w = randn(rng, heads * dv)
    out, state = fx().linear_attention(q, k, v, decay, return_state=True)
    y = fx().group_norm(out.flatten(0, 1).flatten(1), heads, w, z=z.flatten(0, 1)).out.view(b, length, -1)
    ref, _ = attnref.attention(*(d64(t) for t in (q, k, v, decay)), dk ** -0.5, None, None)
    want, _, _ = attnref.group_norm(ref.flatten(2).flatten(0, 1)[:, None], heads, d64(w), None,
                                    d64(z).flatten(0, 1)[:, None], False, 1e-5, None)
    near(y, want.view(b, length, -1))
    half, pool = fx().linear_attention(q[:, :64], k[:, :64], v[:, :64], decay[:, :64], return_state=True)
    for t in range(64, length):
        o = fx().linear_attention_step(pool, q[:, t], k[:, t], v[:, t], decay[:, t])
        near(fx().group_norm(o.flatten(1), heads, w, z=z[:, t]).out, want.view(b, length, -1)[:, t])
    near(pool, d64(state))
