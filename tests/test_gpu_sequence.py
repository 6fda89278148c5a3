"""GPU parity of the sequence operators (short causal convolution, selective scan, residual norm)
with their definitions in 64 bits, at the sizes and values where they can go wrong.

Tolerances.  An output of type T carries one rounding, UNIT[T] = 2^-p of its own value for p
significant bits (8 of bfloat16, 11 of float16, 24 of float32).  Before it stand float32 operations: each result is within FEW units of 2^-24 of
the size of its terms (sums of absolute values, carried through the recurrence by
seqref.scan(magnitude=True) for the scan): the exponential and reciprocal approximations are good
to 2^-22, and a handful of roundings of 2^-24 join, so FEW = 32 bounds a chain of them.  Gradients
that add many tokens are compared by norms: a relative error of 2^-16 for float32 results (2^-22
per step, carried over at most 64 steps of decay) and twice UNIT[T] for rounded ones.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import seqref  # noqa: E402

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
UNIT = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
FEW = 32 * 2.0 ** -24
SUMS = 2.0 ** -16


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


def close(got, ref, size, what=""):
    """|got - ref| <= UNIT |ref| + FEW size, everywhere; not a number where ref is not."""
    tol = UNIT[got.dtype] * ref.abs() * 1.001 + FEW * size + 2.0 ** -24 * (
        got.dtype == torch.float16)  # f16 subnormals have steps of 2^-24
    err = (d64(got) - ref).abs()
    same = torch.isnan(ref) == torch.isnan(d64(got))
    bad = ~(err <= tol) & ~torch.isnan(ref) | ~same
    assert not bad.any(), (what, int(bad.sum()), float(err[bad].max()), float(tol[bad].min()))


def near(got, ref, what=""):
    tol = SUMS if got.dtype == torch.float32 else 2 * UNIT[got.dtype] + SUMS
    g = d64(got)
    assert g.shape == ref.shape, what
    assert (g - ref).norm() <= tol * ref.norm() + 1e-30, (what, float((g - ref).norm() / ref.norm()))


def packing(lens):
    o = np.concatenate([[0], np.cumsum(lens)])
    return torch.from_numpy(o.astype(np.int64)).cuda()


# lengths: (sequences, tokens) dense, or a list of packed lengths (with empty ones, at both ends)
LAYOUTS = [(1, 1), (2, 3), (3, 17), (1, 300), [5], [0, 1, 0, 2, 31, 16, 0], [64, 1, 130, 63, 65],
           [1] * 9]


def lead_of(layout):
    return (sum(layout),) if isinstance(layout, list) else layout


def count(layout):
    return len(layout) if isinstance(layout, list) else layout[0]


# ---- short causal convolution ---------------------------------------------------------------


def conv_data(layout, d, w, dtype, initial, strided, seed=0, param=None):
    rng = np.random.default_rng(seed)
    lead = lead_of(layout)
    wide = randn(rng, *lead, 2 * d + 1 if strided == "odd" else 2 * d, dtype=dtype)
    x = wide[..., 1:1 + d] if strided == "odd" else (wide[..., d:] if strided else
                                                     wide[..., :d].contiguous())
    param = param or dtype
    return dict(x=x, weight=randn(rng, d, w, dtype=param, scale=w ** -0.5),
                bias=randn(rng, d, dtype=param, scale=0.3),
                initial_state=randn(rng, count(layout), w - 1, d, dtype=dtype) if initial else None,
                offsets=packing(layout) if isinstance(layout, list) else None)


def conv_ref(c, silu):
    return seqref.conv(d64(c["x"]), d64(c["weight"]), d64(c["bias"]), silu, d64(c["initial_state"]),
                       c["offsets"].cpu() if c["offsets"] is not None else None)


@pytest.mark.parametrize("layout", LAYOUTS, ids=str)
@pytest.mark.parametrize("d,w,dtype,initial,strided", [
    (8, 4, "bf16", True, False), (40, 4, "bf16", False, "half"), (7, 3, "f16", True, "odd"),
    (33, 2, "f32", True, False), (64, 1, "f32", False, False), (136, 8, "bf16", True, "half"),
    (12, 5, "f32", True, "odd")])
@pytest.mark.parametrize("silu", [False, True])
def test_conv(layout, d, w, dtype, initial, strided, silu):
    c = conv_data(layout, d, w, TYPES[dtype], initial, strided)
    out, final = fx().causal_conv(**c, silu=silu, return_state=True)
    ref, rfinal = conv_ref(c, silu)
    size, _ = seqref.conv(d64(c["x"]).abs(), d64(c["weight"]).abs(), d64(c["bias"]).abs(), False,
                          d64(c["initial_state"]).abs() if initial else None,
                          c["offsets"].cpu() if c["offsets"] is not None else None)
    close(out, ref, size)
    assert torch.equal(d64(final), rfinal)  # inputs, moved


@pytest.mark.parametrize("layout", LAYOUTS, ids=str)
@pytest.mark.parametrize("d,w,dtype,initial,strided", [
    (8, 4, "bf16", True, False), (40, 4, "f32", False, "half"), (7, 3, "f32", True, "odd"),
    (33, 2, "f16", True, False), (16, 1, "f32", False, False), (24, 8, "f32", True, False),
    (1030, 4, "f32", False, False)])
@pytest.mark.parametrize("silu", [False, True])
def test_conv_backward(layout, d, w, dtype, initial, strided, silu):
    c = conv_data(layout, d, w, TYPES[dtype], initial, strided, seed=1)
    rng = np.random.default_rng(2)
    dout = randn(rng, *c["x"].shape, dtype=TYPES[dtype])
    dfinal = randn(rng, count(layout), w - 1, d, dtype=TYPES[dtype]) if initial and w > 1 else None
    got = fx().causal_conv_backward(dout, silu=silu, dfinal_state=dfinal, **c)
    leaves = {k: d64(c[k]).requires_grad_(True) for k in ("x", "weight", "bias")}
    if initial:
        leaves["initial_state"] = d64(c["initial_state"]).requires_grad_(True)
    out, final = seqref.conv(
        leaves["x"], leaves["weight"], leaves["bias"], silu, leaves.get("initial_state"),
        c["offsets"].cpu() if c["offsets"] is not None else None)
    loss = (out * d64(dout)).sum()
    if dfinal is not None:
        loss = loss + (final * d64(dfinal)).sum()
    ref = dict(zip(leaves, torch.autograd.grad(loss, list(leaves.values()))))
    near(got.dx, ref["x"], "dx")
    near(got.dweight, ref["weight"], "dweight")
    near(got.dbias, ref["bias"], "dbias")
    if initial:
        near(got.dinitial_state, ref["initial_state"], "dinitial")
    again = fx().causal_conv_backward(dout, silu=silu, dfinal_state=dfinal, **c)
    assert torch.equal(got.dweight, again.dweight) and torch.equal(got.dx, again.dx)


def test_conv_float32_parameters_and_no_bias():
    c = conv_data((2, 9), 24, 4, torch.bfloat16, True, False, param=torch.float32)
    c["bias"] = None
    out = fx().causal_conv(**c)
    ref, _ = seqref.conv(d64(c["x"]), d64(c["weight"]), None, False, d64(c["initial_state"]), None)
    close(out, ref, ref.abs() + 4.0)


@pytest.mark.parametrize("d,w,dtype", [(16, 4, "bf16"), (5, 3, "f32"), (24, 1, "f16"), (8, 8, "f32")])
def test_conv_step_follows_the_sequence(d, w, dtype):
    """Tokens taken one by one from a pool give the same outputs and states as the sequence."""
    c = conv_data((3, 11), d, w, TYPES[dtype], True, False, seed=3)
    ref, rfinal = conv_ref(c, True)
    pool = torch.full((7, w - 1, d), 9.0, dtype=TYPES[dtype], device="cuda")
    slots = torch.tensor([4, 0, 6], device="cuda")
    pool[slots] = c["initial_state"]
    for t in range(11):
        out = fx().causal_conv_step(pool, c["x"][:, t], c["weight"], c["bias"], silu=True, slots=slots)
        close(out, ref[:, t], ref[:, t].abs() + 8.0)
    assert torch.equal(d64(pool[slots]), rfinal)
    rest = [i for i in range(7) if i not in (4, 0, 6)]
    assert (pool[rest] == 9.0).all()


def test_steps_branch_and_pad():
    """slots_out writes elsewhere and keeps the source; slots outside the pool are padding."""
    rng = np.random.default_rng(4)
    d, n = 20, 6
    pool = randn(rng, 5, d, n)
    before = pool.clone()
    a = dict(A=-torch.rand(d, n, device="cuda") - 0.5)
    u, delta, B, C = (randn(rng, 3, k) for k in (d, d, n, n))
    slots = torch.tensor([2, -1, 5], device="cuda")
    to = torch.tensor([0, 1, 3], device="cuda")
    y = fx().selective_scan_step(pool, u, delta, a["A"], B, C, softplus=True, slots=slots, slots_out=to)
    assert (y[1:] == 0).all() and (y[0] != 0).any()
    assert torch.equal(pool[1:], before[1:]) and not torch.equal(pool[0], before[0])
    state = randn(rng, 5, 3, d)
    keep = state.clone()
    y = fx().causal_conv_step(state, u, randn(rng, d, 4), slots=slots, slots_out=to)
    assert (y[1:] == 0).all()
    assert torch.equal(state[1:], keep[1:])
    assert torch.equal(state[0, :2], keep[2, 1:]) and torch.equal(state[0, 2], u[0])


# ---- selective scan -------------------------------------------------------------------------


def scan_data(layout, d, n, groups, dtype, gate=True, initial=True, strided=True, seed=0,
              softplus=True, extras=True):
    rng = np.random.default_rng(seed)
    lead = lead_of(layout)
    xz = randn(rng, *lead, 2 * d, dtype=dtype)
    bc = randn(rng, *lead, 3 + 2 * groups * n, dtype=dtype)
    u, z = xz[..., :d], xz[..., d:]
    if not strided:
        u, z = u.contiguous(), z.contiguous()
    B = bc[..., 3:3 + groups * n].unflatten(-1, (groups, n))
    C = bc[..., 3 + groups * n:].unflatten(-1, (groups, n))
    delta = randn(rng, *lead, d, dtype=dtype, scale=0.7)
    if not softplus:
        delta = delta.abs() * 0.2
    A = -torch.exp(randn(rng, d, n, scale=0.5)) * torch.arange(1, n + 1, device="cuda")
    return dict(u=u, delta=delta, A=A, B=B, C=C, D=randn(rng, d) if extras else None,
                z=z if gate else None, delta_bias=((randn(rng, d) - 2.0) if softplus else randn(rng, d).abs() * 0.1)
                if extras else None,
                softplus=softplus,
                initial_state=randn(rng, count(layout), d, n) if initial else None,
                offsets=packing(layout) if isinstance(layout, list) else None)


def scan_ref(c, **more):
    return seqref.scan(*(d64(c[k]) for k in ("u", "delta", "A", "B", "C", "D", "z", "delta_bias")),
                       c["softplus"], d64(c["initial_state"]),
                       c["offsets"].cpu() if c["offsets"] is not None else None, **more)


SCANS = [  # d, n, groups, dtype, gate, initial, strided
    (32, 16, 1, "bf16", True, True, True), (37, 16, 1, "f32", True, False, False),
    (6, 1, 2, "f32", False, True, True), (130, 4, 1, "f16", True, True, True),
    (21, 5, 3, "f32", True, True, False), (10, 8, 2, "bf16", False, False, True),
    (9, 24, 1, "f32", True, True, True), (5, 64, 1, "f32", False, True, False),
    (4, 100, 2, "f32", True, True, True), (3, 128, 1, "bf16", True, False, False),
    (15, 10, 1, "f32", True, True, True), (16, 12, 2, "bf16", False, True, False),
    (24, 13, 1, "f16", True, False, True), (128, 32, 1, "bf16", True, True, False)]


@pytest.mark.parametrize("layout", LAYOUTS, ids=str)
@pytest.mark.parametrize("case", SCANS, ids=str)
def test_scan(layout, case):
    d, n, groups, dtype, gate, initial, strided = case
    c = scan_data(layout, d, n, groups, TYPES[dtype], gate, initial, strided)
    out, final = fx().selective_scan(**c, return_state=True)
    ref, rfinal, size = scan_ref(c, magnitude=True)
    close(out, ref, size, "out")
    near(final, rfinal, "final")
    again = fx().selective_scan(**c)
    assert torch.equal(out, again)


@pytest.mark.parametrize("softplus,extras", [(False, True), (True, False), (False, False)])
def test_scan_options(softplus, extras):
    c = scan_data((2, 40), 16, 16, 1, torch.float32, softplus=softplus, extras=extras)
    out = fx().selective_scan(**c)
    ref, _, size = scan_ref(c, magnitude=True)
    close(out, ref, size)


def test_scan_many_chunks():
    """A long row of few channels: time is cut, also inside sequences, with cuts on their ends."""
    for layout in ((1, 2500), [700, 0, 64, 1, 1200, 535]):
        c = scan_data(layout, 24, 16, 1, torch.float32, seed=5)
        out, final = fx().selective_scan(**c, return_state=True)
        ref, rfinal, size = scan_ref(c, magnitude=True)
        close(out, ref, size)
        near(final, rfinal)


def test_scan_continues_from_its_state():
    c = scan_data((2, 90), 40, 16, 1, torch.float32, seed=6)
    whole, end = fx().selective_scan(**c, return_state=True)
    cutat = lambda a, b: {k: (v[:, a:b] if k in ("u", "delta", "B", "C", "z") else v)
                          for k, v in c.items()}
    first, mid = fx().selective_scan(**cutat(0, 37), return_state=True)
    second, end2 = fx().selective_scan(**{**cutat(37, 90), "initial_state": mid}, return_state=True)
    ref, rend, size = scan_ref(c, magnitude=True)
    close(torch.cat([first, second], 1), ref, size)
    near(end2, rend)
    near(end, rend)


def test_scan_no_tokens():
    c = scan_data((2, 1), 12, 4, 1, torch.float32)
    none = {k: (v[:, :0] if k in ("u", "delta", "B", "C", "z") else v) for k, v in c.items()}
    out, final = fx().selective_scan(**none, return_state=True)
    assert out.shape == (2, 0, 12) and torch.equal(final, c["initial_state"])
    g = fx().selective_scan_backward(out, **none, dfinal_state=final)
    assert torch.equal(g.dinitial_state, final) and (g.dA == 0).all() and (g.dD == 0).all()
    x = torch.empty(2, 0, 8, device="cuda")
    init = torch.ones(2, 3, 8, device="cuda")
    y, end = fx().causal_conv(x, torch.ones(8, 4, device="cuda"), initial_state=init, return_state=True)
    assert y.shape == x.shape and torch.equal(end, init)
    g = fx().causal_conv_backward(y, x, torch.ones(8, 4, device="cuda"), initial_state=init,
                                  dfinal_state=init)
    assert torch.equal(g.dinitial_state, init) and (g.dweight == 0).all()


@pytest.mark.parametrize("n", [6, 10, 12, 16, 20])
def test_scan_infinite_and_missing_values(n):
    """A NaN or infinity reaches its own channel from its token on, and a new sequence is clean;
    a state beyond n stays out of it."""
    c = scan_data([30, 20], 8, n, 1, torch.float32, gate=False, seed=7)
    c["u"] = c["u"].clone()
    c["u"][10, 3] = float("nan")
    c["u"][12, 5] = float("inf")
    out, final = fx().selective_scan(**c, return_state=True)
    ref, rfinal, size = scan_ref(c, magnitude=True)
    o = d64(out)
    assert torch.equal(torch.isfinite(o), torch.isfinite(ref))
    assert torch.isfinite(o[30:]).all() and torch.isfinite(o[:10]).all()
    fine = torch.isfinite(ref)
    assert ((o - ref).abs()[fine] <= (FEW * size + 2.0 ** -23 * ref.abs())[fine]).all()


def test_scan_large_steps_forget():
    """Steps so large that the decay underflows: the state is the last input alone."""
    c = scan_data((1, 20), 8, 8, 1, torch.float32, gate=False, seed=8, softplus=False)
    c["delta"] = c["delta"] * 0 + 5000.0
    out = fx().selective_scan(**c)
    ref, _, size = scan_ref(c, magnitude=True)
    close(out, ref, ref.abs() + size)


@pytest.mark.parametrize("layout", [(2, 3), (3, 17), (1, 300), [0, 1, 0, 2, 31, 16, 0],
                                    [64, 1, 130, 63, 65]], ids=str)
@pytest.mark.parametrize("case", SCANS, ids=str)
def test_scan_backward(layout, case):
    d, n, groups, dtype, gate, initial, strided = case
    c = scan_data(layout, d, n, groups, TYPES[dtype], gate, initial, strided, seed=9)
    rng = np.random.default_rng(10)
    dout = randn(rng, *c["u"].shape, dtype=TYPES[dtype])
    dfinal = randn(rng, count(layout), d, n) if initial else None
    got = fx().selective_scan_backward(dout, **c, dfinal_state=dfinal)
    names = [k for k in ("u", "delta", "A", "B", "C", "D", "z", "delta_bias", "initial_state")
             if c[k] is not None]
    v = {k: d64(c[k]).requires_grad_(True) for k in names}
    out, final = seqref.scan(*(v.get(k) for k in ("u", "delta", "A", "B", "C", "D", "z", "delta_bias")),
                             True, v.get("initial_state"),
                             c["offsets"].cpu() if c["offsets"] is not None else None)
    loss = (out * d64(dout)).sum()
    if dfinal is not None:
        loss = loss + (final * d64(dfinal)).sum()
    ref = dict(zip(names, torch.autograd.grad(loss, list(v.values()))))
    for k in names:
        near(getattr(got, "d" + k), ref[k], k)
    again = fx().selective_scan_backward(dout, **c, dfinal_state=dfinal)
    for a, b in zip(got, again):
        assert a is None or torch.equal(a, b)


def test_scan_backward_agrees_with_differences():
    """The gradient of a weighted output against central differences of the 64-bit definition."""
    c = scan_data([7, 0, 12], 6, 5, 2, torch.float32, seed=11)
    rng = np.random.default_rng(12)
    dout = randn(rng, *c["u"].shape)
    got = fx().selective_scan_backward(dout, **c)
    names = ("u", "delta", "A", "B", "C", "D", "z", "delta_bias", "initial_state")
    base = {k: d64(c[k]) for k in names}

    def value(v):
        out, _ = seqref.scan(*(v[k] for k in names[:-1]), True, v["initial_state"], c["offsets"].cpu())
        return float((out * d64(dout)).sum())

    for k in names:
        way = torch.from_numpy(rng.standard_normal(base[k].shape))
        step = 1e-5
        diff = (value({**base, k: base[k] + step * way}) - value({**base, k: base[k] - step * way})) / (2 * step)
        mine = float((d64(getattr(got, "d" + k)) * way).sum())
        # the difference is good to step^2; the gradient to SUMS of its norm times the way's
        tol = SUMS * float(d64(getattr(got, "d" + k)).norm() * way.norm()) + 1e-6 * (1 + abs(diff))
        assert abs(mine - diff) <= tol, (k, mine, diff)


@pytest.mark.parametrize("case", SCANS, ids=str)
def test_scan_step_follows_the_sequence(case):
    d, n, groups, dtype, gate, initial, strided = case
    c = scan_data((3, 7), d, n, groups, TYPES[dtype], gate, True, strided, seed=13)
    ref, rfinal, size = scan_ref(c, magnitude=True)
    pool = torch.full((6, d, n), 9.0, device="cuda")
    slots = torch.tensor([5, 1, 2], device="cuda")
    pool[slots] = c["initial_state"]
    for t in range(7):
        y = fx().selective_scan_step(
            pool, c["u"][:, t], c["delta"][:, t], c["A"], c["B"][:, t], c["C"][:, t], D=c["D"],
            z=c["z"][:, t] if gate else None, delta_bias=c["delta_bias"], softplus=True, slots=slots)
        close(y, ref[:, t], size[:, t])
    near(pool[slots], rfinal)
    assert (pool[[0, 3, 4]] == 9.0).all()


def test_scan_in_place_and_on_another_stream():
    c = scan_data((2, 100), 64, 16, 1, torch.bfloat16, seed=14)
    want = fx().selective_scan(**c)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = fx().selective_scan(**c, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got, want)
    out = fx().selective_scan(**c, out=c["u"])
    assert out is c["u"] and torch.equal(out, want)


def test_scan_in_a_graph():
    c = scan_data((1, 400), 32, 16, 1, torch.bfloat16, seed=15)
    want = fx().selective_scan(**c)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = fx().selective_scan(**c)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, want)


def test_offsets_beyond_32_bits():
    """Rows 2^22 elements apart: the later of 600 tokens lie more than 2^31 elements in."""
    length, d, far = 600, 8, 1 << 22
    wide = torch.empty(length * far, dtype=torch.bfloat16, device="cuda")
    view = wide.as_strided((1, length, d), (length * far, far, 1))
    c = scan_data((1, length), d, 16, 1, torch.bfloat16, strided=False, seed=16)
    view.copy_(c["u"])
    want, state = fx().selective_scan(**c, return_state=True)
    out = wide.as_strided((1, length, d), (length * far, far, 1), far // 2)
    got, end = fx().selective_scan(**{**c, "u": view}, out=out, return_state=True)
    assert torch.equal(got, want) and torch.equal(end, state)
    dout = torch.randn_like(want)
    for a, b in zip(fx().selective_scan_backward(dout, **{**c, "u": view}),
                    fx().selective_scan_backward(dout, **c)):
        assert torch.equal(a, b)
    w = torch.randn(d, 4, device="cuda")
    assert torch.equal(fx().causal_conv(view, w, silu=True), fx().causal_conv(c["u"], w, silu=True))
    for a, b in zip(fx().causal_conv_backward(dout, view, w), fx().causal_conv_backward(dout, c["u"], w)):
        assert a is None or torch.equal(a, b)
    got = fx().residual_norm(view[0], torch.ones(d, device="cuda"), residual=c["z"][0])
    want = fx().residual_norm(c["u"][0], torch.ones(d, device="cuda"), residual=c["z"][0])
    assert torch.equal(got.out, want.out) and torch.equal(got.residual, want.residual)


# ---- residual norm --------------------------------------------------------------------------

ROWS = [(1, 8), (3, 1), (5, 7), (2, 100), (40, 128), (3, 1000), (2, 4096), (3, 8200), (1, 16384),
        (2, 9001)]


@pytest.mark.parametrize("rows,d", ROWS)
@pytest.mark.parametrize("dtype,res", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32"),
                                       ("f16", None), ("f16", "f16")])
def test_norm(rows, d, dtype, res):
    rng = np.random.default_rng(d)
    x = randn(rng, rows, d, dtype=TYPES[dtype])
    r = randn(rng, rows, d, dtype=TYPES[res], scale=3.0) if res else None
    w = randn(rng, d, dtype=TYPES[dtype])
    got = fx().residual_norm(x, w, residual=r, eps=1e-5)
    ref, total = seqref.norm(d64(x), d64(r), d64(w), 1e-5)
    close(got.out, ref, ref.abs())
    if r is None:
        assert got.residual is None
    else:
        close(got.residual, total, total.abs())
        keep = r.clone()
        again = fx().residual_norm(x, w, residual=keep, eps=1e-5, inplace_residual=True)
        assert again.residual is keep and torch.equal(keep, got.residual)
        assert torch.equal(again.out, got.out)


@pytest.mark.parametrize("rows,d", ROWS)
@pytest.mark.parametrize("dtype,group", [("f32", 0), ("bf16", 0), ("bf16", 32), ("bf16", 128),
                                         ("f32", 64), ("f32", 128), ("f16", 64)])
def test_norm_8bit(rows, d, dtype, group):
    rng = np.random.default_rng(d + 1)
    x = randn(rng, rows, d, dtype=TYPES[dtype])
    x[0] = 0  # a row of zeros: scale 0, values 0
    w = randn(rng, d)
    got = fx().residual_norm(x, w, out_dtype=torch.float8_e4m3fn, group=group)
    y, _ = seqref.norm(d64(x), None, d64(w), 1e-6)
    q, scale = seqref.e4m3(y, group)
    assert got.scale.shape == scale.shape
    close(got.scale, scale, scale)
    assert (got.scale[0] == 0).all() and (got.out[0].float() == 0).all()
    # within half a step of e4m3 (2^-4 of the value, 2^-10 below 2^-6) of the exact quotient,
    # and float32's share of it
    s = scale.repeat_interleave(group, 1)[:, :d] if group else scale
    v = y / torch.where(s > 0, s, torch.ones_like(s))
    err = (got.out.float().cpu().double() - v).abs()
    assert (err <= torch.maximum(v.abs() * 2.0 ** -4, torch.tensor(2.0 ** -10)) * (1 + 2.0 ** -10)
            + FEW * v.abs()).all()
    # and the same value as the definition's but where that stands on a rounding's edge
    assert (got.out.float().cpu().double() != q).double().mean() <= 1e-3


def test_norm_8bit_missing_values():
    x = torch.ones(3, 256, device="cuda", dtype=torch.bfloat16)
    x[1, 40] = float("nan")
    got = fx().residual_norm(x, torch.ones(256, device="cuda"), out_dtype=torch.float8_e4m3fn, group=64)
    assert torch.isnan(got.scale[1]).all()  # the row's mean square is not a number
    assert torch.isfinite(got.scale[[0, 2]]).all() and (got.out[[0, 2]].float() == 448.0).all()


@pytest.mark.parametrize("rows,d", ROWS + [(700, 320)])
@pytest.mark.parametrize("dtype,res,extra", [("f32", "f32", True), ("bf16", "f32", True),
                                             ("bf16", "bf16", False), ("f16", "f16", True)])
def test_norm_backward(rows, d, dtype, res, extra):
    rng = np.random.default_rng(d + 2)
    r = randn(rng, rows, d, dtype=TYPES[res], scale=2.0)
    dout = randn(rng, rows, d, dtype=TYPES[dtype])
    w = randn(rng, d, dtype=TYPES[dtype])
    dres = randn(rng, rows, d, dtype=TYPES[res]) if extra else None
    got = fx().residual_norm_backward(dout, r, w, dresidual=dres, eps=1e-5)
    rr, ww = d64(r).requires_grad_(True), d64(w).requires_grad_(True)
    y, _ = seqref.norm(rr, None, ww, 1e-5)
    loss = (y * d64(dout)).sum() + ((rr * d64(dres)).sum() if extra else 0.0)
    dr, dw = torch.autograd.grad(loss, (rr, ww))
    if d > 1:  # one column: y is the sign of r times w, its gradient a difference of equals
        near(got.dresidual, dr, "dr")
        near(got.dx, dr, "dx")
    near(got.dweight, dw, "dweight")
    assert (got.dx is got.dresidual) == (dtype == res)


def test_norm_strided_rows():
    rng = np.random.default_rng(3)
    wide = randn(rng, 4, 3, 200, dtype=torch.bfloat16)
    x, w = wide[..., 8:136], randn(rng, 128)
    got = fx().residual_norm(x, w)
    ref, _ = seqref.norm(d64(x), None, d64(w), 1e-6)
    close(got.out, ref, ref.abs())
    off = wide[..., 3:131]  # rows that start off a 16-byte boundary
    ref, _ = seqref.norm(d64(off), None, d64(w), 1e-6)
    close(fx().residual_norm(off, w).out, ref, ref.abs())


# ---- refusals -------------------------------------------------------------------------------


def test_binding_refuses():
    x = torch.zeros(2, 5, 8, device="cuda")
    w = torch.zeros(8, 4, device="cuda")
    f = fx()
    for bad, err in [(dict(x=x.cpu(), weight=w), TypeError), (dict(x=x.double(), weight=w), TypeError),
                     (dict(x=x[0], weight=w), ValueError), (dict(x=x.transpose(1, 2), weight=w), ValueError),
                     (dict(x=x, weight=w[:7]), ValueError), (dict(x=x, weight=w.bfloat16()), TypeError),
                     (dict(x=x, weight=w, offsets=torch.tensor([0, 5], device="cuda")), ValueError),
                     (dict(x=x, weight=w, initial_state=torch.zeros(2, 4, 8, device="cuda")), ValueError)]:
        with pytest.raises(err):
            f.causal_conv(**bad)
    with pytest.raises(f.GbfftError):
        f.causal_conv(x, torch.zeros(8, 9, device="cuda"))
    A, B = torch.zeros(8, 4, device="cuda"), torch.zeros(2, 5, 1, 4, device="cuda")
    f.selective_scan(x, x, A, B, B)
    for bad in (dict(A=A[:, :3]), dict(B=B[:, :4]), dict(C=B[..., :3]), dict(z=x[:1]),
                dict(D=torch.zeros(7, device="cuda")), dict(offsets=torch.tensor([0, 5], device="cuda"))):
        with pytest.raises((ValueError, TypeError)):
            f.selective_scan(**{**dict(u=x, delta=x, A=A, B=B, C=B), **bad})
    with pytest.raises(f.GbfftError):  # three groups do not divide eight channels
        B3 = torch.zeros(2, 5, 3, 4, device="cuda")
        f.selective_scan(x, x, A, B3, B3)
    with pytest.raises(f.GbfftError):
        f.residual_norm(x, w[:, 0].contiguous(), out_dtype=torch.float8_e4m3fn, group=48)
    with pytest.raises(TypeError):
        f.residual_norm(x, w[:, 0].contiguous(), out_dtype=torch.int8)
    with pytest.raises(f.GbfftError):
        f.selective_scan_step(torch.zeros(1, 8, 4, device="cuda"), x[:, 0], x[:, 0], A, B[:, 0], B[:, 0])
