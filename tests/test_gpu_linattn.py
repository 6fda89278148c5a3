"""GPU parity of linear attention with decays (whole sequences, single tokens, gradients) with its
definition in 64 bits, at the sizes, layouts and values where it can go wrong.

Tolerances.  An output of type T carries one rounding, UNIT[T] of its own value.  Before it, weighted
scores and the state as an operand are rounded to pieces of 8 significant bits: to within 2^-8 of
each term in one piece (bfloat16 outputs), 2^-16 in two (float16, and the gradients of bfloat16; the
product of two second pieces that is left out is 2^-16 too, so up to 3 of them), 2^-24 in three
(float32, again with up to 5 products of that size left out).  Matrix units add exact products in
float32 and may cut what lies below 2^-23 of a sum instead of rounding it: ACC = 2^-17 bounds 64
such steps.  All are relative to the sums over absolute values that attnref.attention(magnitude=True)
carries through the recurrence.  States hold values in three pieces: 8 * 2^-24 + ACC.  Gradients are
compared by norms: 2^-16 for float32 results (the bound of one of their terms would be ACC; over a
norm such errors do not all have one sign), twice UNIT[T] for rounded ones.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import attnref  # noqa: E402

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
UNIT = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
ACC = 2.0 ** -17
TERM = {torch.bfloat16: 2.0 ** -8 + ACC, torch.float16: 3 * 2.0 ** -16 + ACC,
        torch.float32: 8 * 2.0 ** -24 + ACC}
STATE = 8 * 2.0 ** -24 + ACC
SUMS = 2.0 ** -16

LAYOUTS = [(1, 1), (2, 3), (3, 64), (2, 65), (1, 700), [5], [0, 1, 0, 2, 31, 64, 0], [64, 1, 130, 63, 65],
           [300, 0, 2, 400], [1] * 9]
# heads, groups, dk, dv, type, initial state, strides
SHAPES = [(2, 2, 16, 16, "bf16", True, "plain"), (4, 2, 64, 64, "bf16", False, "wide"),
          (2, 1, 128, 128, "bf16", True, "wide"), (1, 1, 256, 96, "bf16", True, "heads first"),
          (3, 3, 7, 5, "bf16", True, "odd"), (2, 2, 24, 200, "f16", True, "wide"),
          (2, 1, 40, 33, "f16", False, "odd"), (1, 1, 128, 72, "f16", True, "heads first"),
          (2, 2, 256, 130, "f16", True, "plain"), (2, 2, 40, 72, "f32", True, "wide"),
          (1, 1, 130, 9, "f32", True, "odd"), (2, 1, 64, 128, "f32", False, "plain"),
          (1, 1, 256, 256, "f32", True, "plain"), (1, 1, 1, 1, "f32", True, "plain")]


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


def close(got, ref, size, term, what=""):
    tol = UNIT[got.dtype] * ref.abs() * 1.001 + term * size + 2.0 ** -24 * (got.dtype == torch.float16)
    err = (d64(got) - ref).abs()
    same = torch.isnan(ref) == torch.isnan(d64(got))
    bad = ~(err <= tol) & ~torch.isnan(ref) | ~same
    assert not bad.any(), (what, int(bad.sum()), float(err[bad].max()), float(tol[bad].min()))


def near(got, ref, what="", more=0.0):
    tol = (SUMS if got.dtype == torch.float32 else 2 * UNIT[got.dtype] + SUMS) + more
    g = d64(got)
    assert g.shape == ref.shape, what
    assert torch.isfinite(g).all(), what
    assert (g - ref).norm() <= tol * ref.norm() + 1e-30, (what, float((g - ref).norm() / ref.norm()))


def packing(lens):
    o = np.concatenate([[0], np.cumsum(lens)])
    return torch.from_numpy(o.astype(np.int64)).cuda()


def data(layout, heads, groups, dk, dv, dtype, initial, strides, seed=0, rate=0.1):
    """Inputs by name.  wide: columns of one projection; odd: the same behind one more value; heads
    first: [sequences, heads, tokens, d] seen as [sequences, tokens, heads, d]."""
    rng = np.random.default_rng(seed)
    lead = (sum(layout),) if isinstance(layout, list) else layout
    nseq = len(layout) if isinstance(layout, list) else layout[0]
    dtype = TYPES[dtype]
    if strides in ("wide", "odd"):
        skip = 1 if strides == "odd" else 0
        w = randn(rng, *lead, skip + 2 * groups * dk + heads * dv, dtype=dtype)[..., skip:]
        q = w[..., :groups * dk].unflatten(-1, (groups, dk))
        k = w[..., groups * dk:2 * groups * dk].unflatten(-1, (groups, dk))
        v = w[..., 2 * groups * dk:].unflatten(-1, (heads, dv))
    else:
        def make(h, d):
            if strides == "plain":
                return randn(rng, *lead, h, d, dtype=dtype)
            return randn(rng, *lead[:-1], h, lead[-1], d, dtype=dtype).transpose(-2, -3)
        q, k, v = make(groups, dk), make(groups, dk), make(heads, dv)
    decay = -(rng.exponential(size=(*lead, heads)) * rate)
    return dict(q=q, k=k, v=v, decay=torch.from_numpy(decay).to(dtype).cuda(),
                initial_state=randn(rng, nseq, heads, dk, dv) if initial else None,
                offsets=packing(layout) if isinstance(layout, list) else None)


def reference(c, scale=None, magnitude=False):
    scale = c["q"].shape[-1] ** -0.5 if scale is None else scale
    return attnref.attention(*(d64(c[n]) for n in ("q", "k", "v", "decay")), scale,
                             d64(c["initial_state"]),
                             c["offsets"].cpu() if c["offsets"] is not None else None, magnitude)


@pytest.mark.parametrize("layout", LAYOUTS, ids=str)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_forward(layout, shape):
    c = data(layout, *shape)
    out, final = fx().linear_attention(**c, return_state=True)
    ref, rfinal, size, total = reference(c, magnitude=True)
    close(out, ref, size, TERM[out.dtype], "out")
    close(final, rfinal, total, STATE, "final")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rate", [0.0, 1e-4, 3.0, 1000.0])
def test_rates(dtype, rate):
    """Heads that keep everything, and ones that forget within a token."""
    c = data((2, 333), 2, 2, 32, 48, dtype, True, "plain", seed=1, rate=rate)
    out, final = fx().linear_attention(**c, return_state=True, scale=0.3)
    ref, rfinal, size, total = reference(c, 0.3, magnitude=True)
    close(out, ref, size, TERM[out.dtype], "out")
    close(final, rfinal, total, STATE, "final")


@pytest.mark.parametrize("dtype", TYPES)
def test_decays_of_every_kind(dtype):
    """Resets by -infinity and by large values between slow decays, and values above 0, which count as
    0."""
    c = data([200, 150], 2, 2, 16, 24, dtype, True, "plain", seed=2, rate=0.01)
    g = c["decay"]
    g[7], g[64], g[100], g[201], g[3], g[250] = -float("inf"), -1e4, -300.0, -float("inf"), 2.0, 0.5
    out, final = fx().linear_attention(**c, return_state=True)
    ref, rfinal, size, total = reference(c, magnitude=True)
    close(out, ref, size, TERM[out.dtype], "out")
    close(final, rfinal, total, STATE, "final")
    dout = randn(np.random.default_rng(3), *c["v"].shape, dtype=TYPES[dtype])
    r = fx().linear_attention_backward(dout, **c)
    for got, want in zip(r, gradients(c, dout)):
        near(got, want)
    assert not r.ddecay[[7, 64, 100, 201, 3, 250]].any()


def gradients(c, dout, dfinal=None, scale=None):
    names = ["q", "k", "v", "decay"] + (["initial_state"] if c["initial_state"] is not None else [])
    leaves = {n: d64(c[n]).requires_grad_(True) for n in names}
    v = {n: leaves.get(n) for n in ("q", "k", "v", "decay", "initial_state")}
    scale = c["q"].shape[-1] ** -0.5 if scale is None else scale
    out, final = attnref.attention(v["q"], v["k"], v["v"], v["decay"], scale, v["initial_state"],
                                   c["offsets"].cpu() if c["offsets"] is not None else None)
    loss = (out * d64(dout)).sum()
    if dfinal is not None:
        loss = loss + (final * d64(dfinal)).sum()
    got = torch.autograd.grad(loss, [leaves[n] for n in names], allow_unused=True)
    return [torch.zeros_like(leaves[n]) if g is None else g for n, g in zip(names, got)]


@pytest.mark.parametrize("layout", [(1, 1), (3, 64), (2, 65), (1, 700), [0, 1, 0, 2, 31, 64, 0],
                                    [300, 0, 2, 400]], ids=str)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("end", [False, True])
def test_gradients(layout, shape, end):
    c = data(layout, *shape, seed=4)
    rng = np.random.default_rng(5)
    dout = randn(rng, *c["v"].shape, dtype=c["v"].dtype)
    nseq = len(layout) if isinstance(layout, list) else layout[0]
    dfinal = randn(rng, nseq, shape[0], shape[2], shape[3]) if end else None
    r = fx().linear_attention_backward(dout, **c, dfinal_state=dfinal)
    for name, got, want in zip(r._fields, r, gradients(c, dout, dfinal)):
        near(got, want, name)
    assert (r.dinitial_state is None) == (c["initial_state"] is None)


@pytest.mark.parametrize("rate", [0.0, 1e-3, 1.0, 5.0])
def test_gradients_of_decays_in_long_sequences(rate):
    """The decay's gradient is a difference of sums that run along the sequence: its error is that of
    its terms, not of all tokens' sums."""
    c = data((1, 2500), 2, 2, 32, 32, "f32", False, "plain", seed=6, rate=rate)
    dout = randn(np.random.default_rng(7), *c["v"].shape)
    r = fx().linear_attention_backward(dout, **c)
    for name, got, want in zip(r._fields, r, gradients(c, dout)):
        near(got, want, name)


def test_gradients_against_differences():
    c = data([40, 90], 2, 1, 12, 20, "f32", True, "plain", seed=8)
    rng = np.random.default_rng(9)
    dout, dfinal = randn(rng, *c["v"].shape), randn(rng, 2, 2, 12, 20)
    r = fx().linear_attention_backward(dout, **c, dfinal_state=dfinal)
    for name, got in zip(("q", "k", "v", "decay", "initial_state"), r):
        way = randn(rng, *c[name].shape, scale=1.0 if name != "decay" else 0.01)
        if name == "decay":  # stay below 0
            way = way * c["decay"].abs().clamp(max=1.0)
        ends = []
        for sign in (1, -1):
            moved = {**{n: d64(c[n]) for n in ("q", "k", "v", "decay", "initial_state")}}
            moved[name] = moved[name] + sign * 1e-4 * d64(way)
            out, final = attnref.attention(*(moved[n] for n in ("q", "k", "v", "decay")), 12 ** -0.5,
                                           moved["initial_state"], c["offsets"].cpu())
            ends.append(float((out * d64(dout)).sum() + (final * d64(dfinal)).sum()))
        want = (ends[0] - ends[1]) / 2e-4
        have = float((d64(got) * d64(way)).sum())
        size = float((d64(got) * d64(way)).abs().sum())
        # differences are off by h^2 of a third derivative and 2^-52 / h of the loss
        assert abs(have - want) <= 1e-5 * size + 1e-7 * abs(ends[0]), (name, have, want)


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("nseq", [1, 5])
def test_step(shape, nseq):
    heads, groups, dk, dv, dtype, _, strides = shape
    c = data((nseq, 1), heads, groups, dk, dv, dtype, False, strides, seed=10)
    one = {n: c[n][:, 0] for n in ("q", "k", "v", "decay")}
    rng = np.random.default_rng(11)
    pool = randn(rng, 2 * nseq + 1, heads, dk, dv)
    at = torch.from_numpy(rng.permutation(2 * nseq + 1)).cuda()
    slots, slots_out = at[:nseq].contiguous(), at[nseq:2 * nseq].contiguous()
    state = pool.clone()
    out = fx().linear_attention_step(state, **one, slots=slots, slots_out=slots_out)
    ref, rfinal, size, total = reference({**c, "initial_state": pool[slots]}, magnitude=True)
    close(out, ref[:, 0], size[:, 0], 64 * 2.0 ** -24, "out")  # float32 sums, dk terms at most 256 / 16 deep
    close(state[slots_out], rfinal, total, 8 * 2.0 ** -24, "state")
    rest = torch.ones(2 * nseq + 1, dtype=torch.bool, device="cuda")
    rest[slots_out] = False
    assert torch.equal(state[rest], pool[rest])
    # in place, without slots
    state = pool.clone()
    again = fx().linear_attention_step(state, **one)
    ref, rfinal, size, total = reference({**c, "initial_state": pool[:nseq]}, magnitude=True)
    close(again, ref[:, 0], size[:, 0], 64 * 2.0 ** -24, "out")
    close(state[:nseq], rfinal, total, 8 * 2.0 ** -24, "state")
    assert torch.equal(state[nseq:], pool[nseq:])


def test_step_padding():
    c = data((4, 1), 2, 2, 16, 16, "bf16", False, "plain", seed=12)
    one = {n: c[n][:, 0] for n in ("q", "k", "v", "decay")}
    pool = randn(np.random.default_rng(13), 3, 2, 16, 16)
    state = pool.clone()
    slots = torch.tensor([1, -1, 7, 2], device="cuda")
    out = fx().linear_attention_step(state, **one, slots=slots)
    assert not out[1:3].any() and out[[0, 3]].abs().sum() > 0
    assert torch.equal(state[0], pool[0]) and not torch.equal(state[1:], pool[1:])


@pytest.mark.parametrize("dtype", TYPES)
def test_prompt_then_tokens(dtype):
    """A prompt, then token by token, against the whole."""
    c = data((2, 150), 2, 1, 64, 32, dtype, True, "wide", seed=14)
    cut = {n: (c[n][:, :130] if n not in ("initial_state", "offsets") else c[n]) for n in c}
    out, pool = fx().linear_attention(**cut, return_state=True)
    outs = [out]
    for t in range(130, 150):
        outs.append(fx().linear_attention_step(pool, *(c[n][:, t] for n in ("q", "k", "v", "decay")))[:, None])
    ref, rfinal, size, total = reference(c, magnitude=True)
    close(torch.cat(outs, 1), ref, size, TERM[TYPES[dtype]], "out")
    close(pool, rfinal, total, STATE, "state")


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("dtype", TYPES)
def test_not_finite_stays_behind(dtype, bad):
    """What is not finite reaches its own token and later ones of its sequence only."""
    c = data([100, 90, 70], 2, 2, 32, 32, dtype, False, "plain", seed=15)
    clean, _ = fx().linear_attention(**c, return_state=True)
    for name in ("q", "k", "v"):
        dirty = {n: t for n, t in c.items()}
        dirty[name] = c[name].clone()
        dirty[name][140, 1, 3] = bad
        out = fx().linear_attention(**dirty)
        touched = torch.zeros(260, 2, 32, dtype=torch.bool, device="cuda")
        if name == "q":
            touched[140, 1] = True
        elif name == "k":
            touched[140:190, 1] = True
        else:
            touched[140:190, 1, 3] = True
        same = torch.isclose(out.float(), clean.float(), rtol=2 * UNIT[out.dtype], atol=1e-3 * float(
            clean.float().abs().max()))
        assert same[~touched].all(), name
        assert not torch.isfinite(out[140, 1, 3]), name


def test_shared_decays_and_scale():
    """Decays that do not change, as views whose strides are 0."""
    c = data((2, 100), 3, 3, 16, 16, "f32", False, "plain", seed=16)
    g = torch.tensor([-0.01, -0.1, 0.0], device="cuda")
    c["decay"] = g.expand(2, 100, 3)
    out = fx().linear_attention(**c, scale=-2.0)
    ref, _, size, _ = reference(c, -2.0, magnitude=True)
    close(out, ref, size, TERM[out.dtype])
    dout = randn(np.random.default_rng(17), *c["v"].shape)
    r = fx().linear_attention_backward(dout, **c, scale=-2.0)
    for got, want in zip(r, gradients(c, dout, scale=-2.0)):
        near(got, want)


@pytest.mark.parametrize("dtype", TYPES)
def test_same_bits_graph_and_stream(dtype):
    """Repeated calls, a captured and replayed one and one on another stream give the same bits."""
    c = data([700, 300], 2, 1, 64, 64, dtype, True, "wide", seed=18)
    dout = randn(np.random.default_rng(19), *c["v"].shape, dtype=c["v"].dtype)

    def both(stream=None):
        out, final = fx().linear_attention(**c, return_state=True, stream=stream)
        r = fx().linear_attention_backward(dout, **c, dfinal_state=final, stream=stream)
        return [out, final, *r]

    first = both()
    for other in (both(),):
        assert all(torch.equal(a, b) for a, b in zip(first, other))
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


@pytest.mark.parametrize("width,first", [(30, 3), (40, 8)])
def test_outputs_inside_larger_tensors(width, first):
    """out may be any view, on 16-byte boundaries or off them; what lies around it stays."""
    c = data((2, 70), 2, 2, 16, 24, "bf16", False, "plain", seed=20)
    ref, _, size, _ = reference(c, magnitude=True)
    whole = torch.full((2, 71, 3, width), 7.0, dtype=torch.bfloat16, device="cuda")
    out = whole[:, :70, 1:, first:first + 24]
    fx().linear_attention(**c, out=out)
    close(out, ref, size, TERM[torch.bfloat16])
    if width % 8 == 0:  # the same kernel as for outputs of their own
        assert torch.equal(out, fx().linear_attention(**c))
    out.fill_(7.0)
    assert (whole == 7.0).all()


def test_empty():
    f = fx().linear_attention
    c = data((2, 3), 2, 2, 8, 8, "f32", True, "plain")
    none = {n: (t[:, :0] if n != "initial_state" else t) for n, t in c.items() if n != "offsets"}
    out, final = f(**none, return_state=True)
    assert out.shape == (2, 0, 2, 8) and torch.equal(final, c["initial_state"])
    r = fx().linear_attention_backward(out, **none, dfinal_state=final)
    assert r.dq.shape == (2, 0, 2, 8) and torch.equal(r.dinitial_state, final)
    c = data([0, 0], 2, 2, 8, 8, "f32", True, "plain")
    out, final = f(**c, return_state=True)
    assert out.shape == (0, 2, 8) and torch.equal(final, c["initial_state"])
    c = {n: t[:0] for n, t in data((2, 3), 2, 2, 8, 8, "f32", True, "plain").items() if n != "offsets"}
    out, final = f(**c, return_state=True)
    assert out.shape == (0, 3, 2, 8) and final.shape == (0, 2, 8, 8)
