"""Sequence-layer operators: the cases that are measured, their plain forms and their definitions.

The operators are the parts of a layer that filters a sequence with coefficients that change from
token to token, where no transfer function exists and the FFT plans do not apply:

  conv    short causal convolution along the tokens of every channel, with bias and SiLU
  scan    selective state-space scan h[t] = exp(d[t] A) h[t-1] + d[t] B[t] u[t], y[t] = C[t] h[t]
  norm    root-mean-square norm of x + residual, in the inputs' type or in 8 bits with scales

Each has its form for whole sequences (prompts), its backward pass (training), and conv and scan
their form for single tokens, which moves states within a pool.  `run` computes the plain
form (elementary torch operations in 32 bits, rounded once at the end) where `own` is false, and
calls the package where it is true.
"""
import math

import torch

own = False

_DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
_SIZE = {"f32": 4, "bf16": 2, "f16": 2}


def _pkg():
    import fft_signal_processing_gb300 as fx

    return fx


# ---- cases ----------------------------------------------------------------------------------


def listed():
    return [
        # one sequence being answered: the latency of one token in one layer
        dict(name="scan_step_one", op="scan_step", nseq=1, d=2048, n=16, groups=1, dtype="bf16"),
        # many sequences being answered, their states scattered over a pool
        dict(name="scan_step_many", op="scan_step", nseq=256, d=4096, n=16, groups=1,
             dtype="bf16"),
        # one long prompt: few channels, so time itself has to be split
        dict(name="scan_prompt_long", op="scan", nseq=1, length=16384, d=2048, n=16, groups=1,
             dtype="bf16", packed=False, gate=True, initial=False),
        # a batch of prompts that continue from earlier states
        dict(name="scan_prompt_batch", op="scan", nseq=8, length=2048, d=4096, n=16, groups=1,
             dtype="bf16", packed=False, gate=True, initial=True),
        # ragged prompts packed one after another, odd channel and state counts, two groups, 32 bits
        dict(name="scan_packed_odd", op="scan", nseq=37, length=10007, d=1002, n=10, groups=2,
             dtype="f32", packed=True, gate=False, initial=True),
        # a training step's reverse pass through the scan
        dict(name="scan_train", op="scan_backward", nseq=4, length=2048, d=2048, n=16, groups=1,
             dtype="bf16", packed=False, gate=True, initial=False),
        # one token of one sequence through the short convolution
        dict(name="conv_step_one", op="conv_step", nseq=1, d=4096, width=4, dtype="bf16"),
        # a batch of prompts through the short convolution; x is half of a wider projection
        dict(name="conv_prompt", op="conv", nseq=4, length=4096, d=4096, width=4, dtype="bf16",
             packed=False, initial=False),
        # training on packed documents of odd lengths
        dict(name="conv_train_packed", op="conv_backward", nseq=61, length=16001, d=2000, width=4,
             dtype="bf16", packed=True, initial=False),
        # a few tokens of answers: the norm before an 8-bit projection, one scale per 128 columns
        dict(name="norm_few_8bit", op="norm", rows=16, d=4096, dtype="bf16", res="bf16",
             out="e4m3", group=128),
        # a long prompt: the same with one scale per token
        dict(name="norm_prompt_8bit", op="norm", rows=16384, d=4096, dtype="bf16", res="bf16",
             out="e4m3", group=0),
        # training: gradients of the norm, the residual stream held in 32 bits
        dict(name="norm_train", op="norm_backward", rows=8192, d=2560, dtype="bf16", res="f32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["scan_step", "scan", "scan", "scan_backward", "conv_step", "conv",
                     "conv_backward", "norm", "norm", "norm_backward"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op in ("norm", "norm_backward"):
        d = _log(rng, 64, 8192)
        if rng.random() < 0.7:
            d = (d + 63) // 64 * 64
        if d == 3 * 1024:
            d += 64
        case = dict(op=op, d=d, dtype=dtype, res=rng.choice([dtype, "f32"]))
        each = 2 * _SIZE[dtype] + 3 * _SIZE[case["res"]]  # bytes per element, at most
        case["rows"] = _log(rng, 1, max(2, min(16384, 500000000 // (each * d))))
        if op == "norm":
            case["out"] = rng.choice(["same", "e4m3", "e4m3"])
            case["group"] = 0 if case["out"] == "same" else rng.choice([0, 32, 64, 128])
        return case
    if op in ("scan_step", "conv_step"):
        d = _log(rng, 64, 8192)
        if rng.random() < 0.7:
            d = (d + 31) // 32 * 32
        if d == 3 * 1024:
            d += 32
        case = dict(op=op, nseq=_log(rng, 1, max(2, min(512, (1 << 20) // d))), d=d, dtype=dtype)
        if op == "scan_step":
            case["n"] = rng.choice([4, 8, 10, 16, 16, 16])
            case["groups"] = 2 if d % 2 == 0 and rng.random() < 0.3 else 1
        else:
            case["width"] = rng.choice([2, 3, 4, 4])
        return case
    d = _log(rng, 64, 4096)
    if rng.random() < 0.7:
        d = (d + 31) // 32 * 32
    if d == 3 * 1024:
        d += 32
    backward = op.endswith("_backward")
    packed = rng.random() < 0.4
    if op.startswith("scan"):
        n = rng.choice([4, 8, 10, 16, 16, 16])
        cap = (1 << 24) // d if backward or dtype == "f32" else (1 << 25) // d
        tokens = _log(rng, 16, max(17, min(16384, cap)))
    else:
        tokens = _log(rng, 16, max(17, min(32768, (1 << 25) // d)))
    nseq = _log(rng, 1, max(1, min(64, tokens // 2)))
    case = dict(op=op, nseq=nseq, length=tokens if packed else max(1, tokens // nseq), d=d,
                dtype=dtype, packed=packed, initial=rng.random() < 0.5)
    if op.startswith("scan"):
        case.update(n=n, groups=2 if d % 2 == 0 and rng.random() < 0.3 else 1,
                    gate=rng.random() < 0.7)
    else:
        case["width"] = rng.choice([2, 3, 4, 4])
    return case


def _tokens(case):
    return case["length"] if case["packed"] else case["nseq"] * case["length"]


def work(case):
    op, d = case["op"], case["d"]
    e = _SIZE[case["dtype"]]
    if op == "norm":
        el, r = case["rows"] * d, _SIZE[case["res"]]
        o = e if case["out"] == "same" else 1
        groups = 0 if case["out"] == "same" else (1 if not case["group"] else
                                                  -(-d // case["group"]))
        return {"bytes": el * (e + 2 * r + o) + case["rows"] * groups * 4 + 4 * d, "flops": el * 6}
    if op == "norm_backward":
        el, r = case["rows"] * d, _SIZE[case["res"]]
        extra = e if r != e else 0  # the gradient of x apart from the residual's where types differ
        return {"bytes": el * (e + 2 * r + r + extra) + 8 * d, "flops": el * 12}
    if op == "conv_step":
        el, w = case["nseq"] * d, case["width"]
        return {"bytes": el * e * (2 + 2 * (w - 1)) + d * (w + 1) * e, "flops": el * (2 * w + 4)}
    if op == "scan_step":
        el, n = case["nseq"] * d, case["n"]
        return {"bytes": el * (8 * n + 4 * e) + 2 * case["nseq"] * case["groups"] * n * e
                + d * (4 * n + 8), "flops": el * (7 * n + 12)}
    el = _tokens(case) * d
    if op in ("conv", "conv_backward"):
        w = case["width"]
        states = case["nseq"] * (w - 1) * d * e
        if op == "conv":
            return {"bytes": 2 * el * e + d * (w + 1) * e + states * (1 + case["initial"]),
                    "flops": el * (2 * w + 4)}
        return {"bytes": 3 * el * e + d * (w + 1) * (e + 4) + 2 * states * case["initial"],
                "flops": el * (6 * w + 10)}
    n, bc = case["n"], 2 * _tokens(case) * case["groups"] * case["n"] * e
    states = case["nseq"] * d * n * 4
    streams = 3 + (1 if case["gate"] else 0)
    if op == "scan":
        return {"bytes": el * e * streams + bc + d * (4 * n + 8) + states * (1 + case["initial"]),
                "flops": el * (7 * n + 12)}
    # reads u, delta, dout (z); writes du, ddelta (dz)
    streams = 5 + (2 if case["gate"] else 0)
    return {"bytes": el * e * streams + 2 * bc + 2 * d * (4 * n + 8)
            + 2 * states * case["initial"], "flops": el * (24 * n + 30)}


# ---- inputs ---------------------------------------------------------------------------------


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _normal(g, *shape, dtype=torch.float32, scale=1.0):
    x = torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)
    return (x * scale).to(dtype)


def _offsets(g, nseq, total):
    """Cuts at random places: lengths from 0 up; the first and last sequence are not empty."""
    cuts = torch.randint(0, total + 1, (nseq - 1,), generator=g, device="cuda")
    cuts = torch.sort(cuts)[0]
    ends = torch.tensor([0], device="cuda"), torch.tensor([total], device="cuda")
    return torch.cat([ends[0], cuts, ends[1]]).to(torch.int64)


def _slots(g, nseq):
    """The pool's size, and the places that the states are read from and written to: other ones,
    as where a sequence keeps the state that it branched from (and so that a pass can be run
    again on the same pool)."""
    pool = 2 * nseq + nseq // 2 + 1
    at = torch.randperm(pool, generator=g, device="cuda").to(torch.int64)
    return pool, at[:nseq].contiguous(), at[nseq:2 * nseq].contiguous()


def prepare(case, seed):
    g, op, d = _gen(seed), case["op"], case["d"]
    dt = _DTYPES[case["dtype"]]
    st = {"case": case}
    if op.startswith("norm"):
        rows, rt = case["rows"], _DTYPES[case["res"]]
        st["weight"] = (1.0 + 0.2 * _normal(g, d)).contiguous()
        if op == "norm":
            st["x"] = _normal(g, rows, d, dtype=dt)
            st["residual"] = _normal(g, rows, d, dtype=rt, scale=3.0)
        else:
            st["sum"] = _normal(g, rows, d, dtype=rt, scale=3.0)
            st["dout"] = _normal(g, rows, d, dtype=dt, scale=0.5)
            st["dresidual"] = _normal(g, rows, d, dtype=rt, scale=0.5)
        return st
    nseq = case["nseq"]
    step = op.endswith("_step")
    packed = not step and case["packed"]
    lead = (nseq,) if step else ((case["length"],) if packed else (nseq, case["length"]))
    st["offsets"] = _offsets(g, nseq, case["length"]) if packed else None
    # x (or u) and the gate z are the two halves of one projection
    xz = _normal(g, *lead, 2 * d, dtype=dt)
    if op.startswith("conv"):
        w = case["width"]
        st["x"] = xz[..., :d]
        st["weight"] = _normal(g, d, w, dtype=dt, scale=w ** -0.5)
        st["bias"] = _normal(g, d, dtype=dt, scale=0.1)
        if step:
            pool, st["slots"], st["slots_out"] = _slots(g, nseq)
            st["state"] = _normal(g, pool, w - 1, d, dtype=dt)
        else:
            st["initial"] = _normal(g, nseq, w - 1, d, dtype=dt) if case["initial"] else None
            if op == "conv_backward":
                st["dout"] = _normal(g, *lead, d, dtype=dt, scale=0.5)
        return st
    n, groups = case["n"], case["groups"]
    st["u"], st["z"] = xz[..., :d], xz[..., d:]
    st["delta"] = _normal(g, *lead, d, dtype=dt, scale=0.5)
    # B and C are columns of one projection, behind the 128 columns that make delta
    bc = _normal(g, *lead, 128 + 2 * groups * n, dtype=dt)
    st["B"] = bc[..., 128:128 + groups * n].unflatten(-1, (groups, n))
    st["C"] = bc[..., 128 + groups * n:].unflatten(-1, (groups, n))
    k = torch.arange(1, n + 1, device="cuda", dtype=torch.float32)
    st["A"] = -(k * torch.exp(0.2 * _normal(g, d, n))).contiguous()
    st["D"] = (1.0 + 0.1 * _normal(g, d)).contiguous()
    # steps between 0.001 and 0.1, as such layers start from
    s = torch.exp(torch.rand(d, generator=g, device="cuda") * math.log(100.0) - math.log(1000.0))
    st["delta_bias"] = (s + torch.log(-torch.expm1(-s))).contiguous()
    if step:
        pool, st["slots"], st["slots_out"] = _slots(g, nseq)
        st["state"] = _normal(g, pool, d, n)
        return st
    if not case["gate"]:
        st["z"] = None
    st["initial"] = _normal(g, nseq, d, n) if case["initial"] else None
    if op == "scan_backward":
        st["dout"] = _normal(g, *lead, d, dtype=dt, scale=0.5)
    return st


# ---- one pass -------------------------------------------------------------------------------


def run(state):
    op = state["case"]["op"]
    return (_OWN if own else _PLAIN)[op](state)


def _own_norm(s):
    c = s["case"]
    more = {} if c["out"] == "same" else {"out_dtype": torch.float8_e4m3fn, "group": c["group"]}
    r = _pkg().residual_norm(s["x"], s["weight"], residual=s["residual"], **more)
    return {"out": r.out, "scale": r.scale, "residual": r.residual}


def _own_norm_backward(s):
    r = _pkg().residual_norm_backward(s["dout"], s["sum"], s["weight"], dresidual=s["dresidual"])
    return {"dx": r.dx, "dresidual": r.dresidual, "dweight": r.dweight}


def _own_conv(s):
    out, final = _pkg().causal_conv(s["x"], s["weight"], s["bias"], silu=True,
                                    initial_state=s["initial"], offsets=s["offsets"],
                                    return_state=True)
    return {"out": out, "final": final}


def _own_conv_backward(s):
    r = _pkg().causal_conv_backward(s["dout"], s["x"], s["weight"], s["bias"], silu=True,
                                    initial_state=s["initial"], offsets=s["offsets"])
    return {"dx": r.dx, "dweight": r.dweight, "dbias": r.dbias, "dinitial": r.dinitial_state}


def _own_conv_step(s):
    out = _pkg().causal_conv_step(s["state"], s["x"], s["weight"], s["bias"], silu=True,
                                  slots=s["slots"], slots_out=s["slots_out"])
    return {"out": out, "state": s["state"]}


def _own_scan(s):
    out, final = _pkg().selective_scan(
        s["u"], s["delta"], s["A"], s["B"], s["C"], D=s["D"], z=s["z"],
        delta_bias=s["delta_bias"], softplus=True, initial_state=s["initial"],
        offsets=s["offsets"], return_state=True)
    return {"out": out, "final": final}


def _own_scan_backward(s):
    r = _pkg().selective_scan_backward(
        s["dout"], s["u"], s["delta"], s["A"], s["B"], s["C"], D=s["D"], z=s["z"],
        delta_bias=s["delta_bias"], softplus=True, initial_state=s["initial"],
        offsets=s["offsets"])
    return {"du": r.du, "ddelta": r.ddelta, "dA": r.dA, "dB": r.dB, "dC": r.dC, "dD": r.dD,
            "dz": r.dz, "ddelta_bias": r.ddelta_bias, "dinitial": r.dinitial_state}


def _own_scan_step(s):
    out = _pkg().selective_scan_step(s["state"], s["u"], s["delta"], s["A"], s["B"], s["C"],
                                     D=s["D"], z=s["z"], delta_bias=s["delta_bias"],
                                     softplus=True, slots=s["slots"], slots_out=s["slots_out"])
    return {"out": out, "state": s["state"]}


# ---- plain forms ----------------------------------------------------------------------------


def _sigmoid(x):
    return 1.0 / (1.0 + torch.exp(-x))


def _softplus(x):
    return torch.clamp(x, min=0.0) + torch.log1p(torch.exp(-torch.abs(x)))


def _plain_norm(s):
    c = s["case"]
    r = s["x"].float() + s["residual"].float()
    y = r * torch.rsqrt((r * r).mean(dim=1, keepdim=True) + 1e-6) * s["weight"]
    res = r.to(s["residual"].dtype)
    if c["out"] == "same":
        return {"out": y.to(s["x"].dtype), "scale": None, "residual": res}
    rows, d = y.shape
    group = c["group"] or d
    yg = y
    if d % group:  # the last group is shorter
        yg = torch.cat([y, y.new_zeros(rows, -d % group)], dim=1)
    yg = yg.view(rows, -1, group)
    amax = yg.abs().amax(dim=2, keepdim=True)
    q = yg * torch.where(amax > 0, 448.0 / amax, torch.zeros_like(amax))
    q = q.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(rows, -1)
    return {"out": q[:, :d].contiguous(), "scale": (amax / 448.0).view(rows, -1),
            "residual": res}


def _plain_norm_backward(s):
    r, g = s["sum"].float(), s["dout"].float()
    rstd = torch.rsqrt((r * r).mean(dim=1, keepdim=True) + 1e-6)
    wg = g * s["weight"]
    dr = rstd * wg - r * rstd ** 3 * (wg * r).mean(dim=1, keepdim=True) + s["dresidual"].float()
    return {"dx": dr.to(s["dout"].dtype), "dresidual": dr.to(s["sum"].dtype),
            "dweight": (g * r * rstd).sum(dim=0)}


def _packed(s):
    """Of a packed batch: every token's sequence and place in it."""
    o, x = s["offsets"], s["x"] if "x" in s else s["u"]
    lens = o[1:] - o[:-1]
    seq = torch.repeat_interleave(torch.arange(len(lens), device=x.device), lens,
                                  output_size=x.shape[0])
    return seq, torch.arange(x.shape[0], device=x.device) - o[seq]


def _taps(s):
    """The w earlier inputs of every token, oldest first, in 32 bits: w tensors of x's shape."""
    x, w, init = s["x"].float(), s["weight"].shape[1], s["initial"]
    if s["offsets"] is None:
        head = init.float() if init is not None else x.new_zeros(x.shape[0], w - 1, x.shape[2])
        xe = torch.cat([head, x], dim=1)
        return [xe[:, k:k + x.shape[1]] for k in range(w)]
    seq, at = _packed(s)
    taps = []
    for back in range(w - 1, -1, -1):
        tap = torch.roll(x, back, dims=0)
        before = (at < back)[:, None]
        head = init.float()[seq, (w - 1 + at - back).clamp(0, max(w - 2, 0))] if (
            init is not None and w > 1) else torch.zeros_like(x)
        taps.append(torch.where(before, head, tap))
    return taps


def _preact(s, taps):
    p = s["bias"].float() + s["weight"][:, 0].float() * taps[0]
    for k in range(1, len(taps)):
        p = p + s["weight"][:, k].float() * taps[k]
    return p


def _plain_conv(s):
    x, w, init = s["x"], s["weight"].shape[1], s["initial"]
    p = _preact(s, _taps(s))
    out = (p * _sigmoid(p)).to(x.dtype)
    if s["offsets"] is None:
        head = init if init is not None else x.new_zeros(x.shape[0], w - 1, x.shape[2])
        final = torch.cat([head, x[:, max(0, x.shape[1] - (w - 1)):]], dim=1)[:, -(w - 1):]
        return {"out": out, "final": final.contiguous()}
    o = s["offsets"]
    lens = o[1:] - o[:-1]
    if init is None:
        init = x.new_zeros(len(lens), w - 1, x.shape[1])
    back = torch.arange(w - 1, 0, -1, device=x.device)  # rows of a state: w-1 .. 1 tokens back
    own_rows = x[(o[1:, None] - back).clamp(min=0)]
    at = (w - 1 + lens[:, None] - back).clamp(0, w - 2)
    kept = torch.gather(init, 1, at[:, :, None].expand(-1, -1, x.shape[1]))
    return {"out": out, "final": torch.where((back <= lens[:, None])[:, :, None], own_rows, kept)}


def _plain_conv_backward(s):
    x, weight, init = s["x"], s["weight"].float(), s["initial"]
    d, w = weight.shape
    taps = _taps(s)
    p = _preact(s, taps)
    sg = _sigmoid(p)
    dp = s["dout"].float() * (sg * (1.0 + p * (1.0 - sg)))
    over = tuple(range(dp.dim() - 1))
    dw = torch.stack([(dp * tap).sum(dim=over) for tap in taps], dim=1)
    if s["offsets"] is None:
        dxe = dp.new_zeros(dp.shape[0], dp.shape[1] + w - 1, d)
        for k in range(w):
            dxe[:, k:k + dp.shape[1]] += weight[:, k] * dp
        dx, dinit = dxe[:, w - 1:], dxe[:, :w - 1]
    else:
        seq, at = _packed(s)
        left = (s["offsets"][1:] - s["offsets"][:-1])[seq] - 1 - at  # tokens that follow
        dx = torch.zeros_like(dp)
        dinit = dp.new_zeros(s["case"]["nseq"], w - 1, d)
        for k in range(w):
            back = w - 1 - k
            term = weight[:, k] * dp
            dx += torch.where((left >= back)[:, None], torch.roll(term, -back, dims=0), 0.0)
            if back:
                early = at < back
                dinit.index_put_((seq[early], w - 1 + at[early] - back), term[early],
                                 accumulate=True)
    return {"dx": dx.to(x.dtype), "dweight": dw, "dbias": dp.sum(dim=over),
            "dinitial": dinit.to(x.dtype) if init is not None else None}


def _plain_conv_step(s):
    xe = torch.cat([s["state"][s["slots"]], s["x"][:, None]], dim=1)
    p = (xe.float() * s["weight"].t().float()).sum(dim=1) + s["bias"].float()
    s["state"][s["slots_out"]] = xe[:, 1:]
    return {"out": (p * _sigmoid(p)).to(s["x"].dtype), "state": s["state"]}


def _steps(s):
    return _softplus(s["delta"].float() + s["delta_bias"]), s["u"].float()


def _per_channel(x, d):
    """[..., groups, n] -> [..., d, n] in 32 bits: every channel reads its group's row."""
    groups, n = x.shape[-2:]
    x = x.float().unsqueeze(-2).expand(*x.shape[:-2], groups, d // groups, n)
    return x.reshape(*x.shape[:-3], d, n)


def _recurrence(a, b):
    """h[t] = a[t] h[t-1] + b[t] along dim 1 for all t, in log2(length) doublings."""
    k = 1
    while k < a.shape[1]:
        b = torch.cat([b[:, :k], torch.addcmul(b[:, k:], a[:, k:], b[:, :-k])], dim=1)
        if 2 * k < a.shape[1]:
            a = torch.cat([a[:, :k], a[:, k:] * a[:, :-k]], dim=1)
        k *= 2
    return b


def _starts(s):
    """(rows, tokens, sequences) of the first tokens in a [rows, tokens] batch."""
    if s["offsets"] is None:
        n = s["u"].shape[0]
        rows = torch.arange(n, device="cuda")
        return rows, torch.zeros_like(rows), rows
    o = s["offsets"]
    seq = torch.nonzero(o[1:] > o[:-1])[:, 0]
    return torch.zeros_like(seq), o[seq], seq


def _ends(s):
    if s["offsets"] is None:
        n = s["u"].shape[0]
        rows = torch.arange(n, device="cuda")
        return rows, torch.full_like(rows, s["u"].shape[1] - 1), rows
    o = s["offsets"]
    seq = torch.nonzero(o[1:] > o[:-1])[:, 0]
    return torch.zeros_like(seq), o[seq + 1] - 1, seq


def _batched(s, x):
    """Packed tokens as a batch of one row."""
    return x[None] if s["offsets"] is not None and x is not None else x


def _states(s, dl, uf, B):
    """decays, states and the states before every token, [rows, tokens, d, n]."""
    rows, first, seq = _starts(s)
    a = torch.exp(dl[..., None] * s["A"])
    b = (dl * uf)[..., None] * B
    cut = a.clone()
    cut[rows, first] = 0.0
    if s["initial"] is not None:
        b[rows, first] += a[rows, first] * s["initial"][seq]
    h = _recurrence(cut, b)
    before = torch.roll(h, 1, dims=1)
    before[rows, first] = s["initial"][seq] if s["initial"] is not None else 0.0
    return a, h, before


def _plain_scan(s):
    d = s["A"].shape[0]
    dl, uf = (_batched(s, x) for x in _steps(s))
    B, C = (_per_channel(_batched(s, s[k]), d) for k in ("B", "C"))
    _, h, _ = _states(s, dl, uf, B)
    y = (h * C).sum(dim=-1) + s["D"] * uf
    if s["z"] is not None:
        zf = _batched(s, s["z"]).float()
        y = y * (zf * _sigmoid(zf))
    final = s["initial"].clone() if s["initial"] is not None else h.new_zeros(
        s["case"]["nseq"], *s["A"].shape)
    rows, last, seq = _ends(s)
    final[seq] = h[rows, last]
    return {"out": y.to(s["u"].dtype).view(s["u"].shape), "final": final}


def _plain_scan_backward(s):
    A, D, dt, groups = s["A"], s["D"], s["u"].dtype, s["B"].shape[-2]
    d = A.shape[0]
    raw = _batched(s, s["delta"]).float() + s["delta_bias"]
    dl, uf = (_batched(s, x) for x in _steps(s))
    B, C = (_per_channel(_batched(s, s[k]), d) for k in ("B", "C"))
    a, h, before = _states(s, dl, uf, B)
    g = _batched(s, s["dout"]).float()
    dy, dz = g, None
    if s["z"] is not None:
        zf = _batched(s, s["z"]).float()
        sg = _sigmoid(zf)
        y = (h * C).sum(dim=-1) + D * uf
        dz = (g * y * sg * (1.0 + zf * (1.0 - sg))).to(dt).view(s["u"].shape)
        dy = g * zf * sg
    dC = (dy[..., None] * h).unflatten(2, (groups, d // groups)).sum(dim=3)
    # q[t] = dy[t] C[t] + a[t+1] q[t+1]: the same recurrence with the tokens in reverse
    rows, first, seq = _starts(s)
    cut = a.clone()
    cut[rows, first] = 0.0
    q = _recurrence(torch.roll(cut, -1, dims=1).flip(1), (dy[..., None] * C).flip(1)).flip(1)
    qb, qah = (q * B).sum(dim=-1), q * a * before
    ddelta = (uf * qb + (qah * A).sum(dim=-1)) * _sigmoid(raw)
    dB = (q * (dl * uf)[..., None]).unflatten(2, (groups, d // groups)).sum(dim=3)
    dinit = None
    if s["initial"] is not None:
        dinit = torch.zeros_like(s["initial"])
        dinit[seq] = a[rows, first] * q[rows, first]
    return {"du": (dl * qb + dy * D).to(dt).view(s["u"].shape),
            "ddelta": ddelta.to(dt).view(s["u"].shape),
            "dA": (qah * dl[..., None]).sum(dim=(0, 1)), "dB": dB.to(dt).view(s["B"].shape),
            "dC": dC.to(dt).view(s["C"].shape), "dD": (dy * uf).sum(dim=(0, 1)), "dz": dz,
            "ddelta_bias": ddelta.sum(dim=(0, 1)), "dinitial": dinit}


def _plain_scan_step(s):
    d = s["A"].shape[0]
    dl, uf = _steps(s)
    h = (torch.exp(dl[..., None] * s["A"]) * s["state"][s["slots"]]
         + (dl * uf)[..., None] * _per_channel(s["B"], d))
    s["state"][s["slots_out"]] = h
    zf = s["z"].float()
    y = ((h * _per_channel(s["C"], d)).sum(dim=-1) + s["D"] * uf) * (zf * _sigmoid(zf))
    return {"out": y.to(s["u"].dtype), "state": s["state"]}


_PLAIN = {"norm": _plain_norm, "norm_backward": _plain_norm_backward, "conv": _plain_conv,
          "conv_backward": _plain_conv_backward, "conv_step": _plain_conv_step,
          "scan": _plain_scan, "scan_backward": _plain_scan_backward,
          "scan_step": _plain_scan_step}
_OWN = {"norm": _own_norm, "norm_backward": _own_norm_backward, "conv": _own_conv,
        "conv_backward": _own_conv_backward, "conv_step": _own_conv_step, "scan": _own_scan,
        "scan_backward": _own_scan_backward, "scan_step": _own_scan_step}


# ---- the definitions in 64 bits -------------------------------------------------------------


def exact(case, seed):
    """The outputs of `run` from the definitions, token by token in 64 bits; gradients by
    differentiating the definition."""
    s = {k: (v.double() if isinstance(v, torch.Tensor) and v.is_floating_point() else v)
         for k, v in prepare(case, seed).items()}
    return _EXACT[case["op"]](s)


def _x_norm(s):
    c = s["case"]
    r = s["x"] + s["residual"]
    y = r / torch.sqrt(torch.mean(r ** 2, 1, True) + 1e-6) * s["weight"]
    if c["out"] == "same":
        return {"out": y, "scale": None, "residual": r}
    outs, scales = [], []
    for part in torch.split(y, c["group"] or c["d"], dim=1):
        scale = part.abs().max(dim=1, keepdim=True)[0] / 448.0
        q = part / torch.where(scale > 0, scale, torch.ones_like(scale))
        # e4m3: 3 bits behind the leading one, steps of 2^-9 below 2^-6
        step = torch.exp2(torch.floor(torch.log2(q.abs().clamp(min=2.0 ** -6))) - 3)
        outs.append(torch.round(q / step) * step)
        scales.append(scale)
    return {"out": torch.cat(outs, 1), "scale": torch.cat(scales, 1), "residual": r}


def _x_norm_backward(s):
    r = s["sum"].requires_grad_(True)
    w = s["weight"].requires_grad_(True)
    y = r / torch.sqrt(torch.mean(r ** 2, 1, True) + 1e-6) * w
    dr, dw = torch.autograd.grad((y * s["dout"] + r * s["dresidual"]).sum(), (r, w))
    return {"dx": dr, "dresidual": dr, "dweight": dw}


def _x_rows(s, i):
    """Sequence i alone, [length, d], as views."""
    if s["offsets"] is None:
        return lambda t: t[i]
    a, b = int(s["offsets"][i]), int(s["offsets"][i + 1])
    return lambda t: t[a:b]


def _x_conv_forward(s, x, weight, bias, initial):
    w = weight.shape[1]
    outs, finals = [], []
    for i in range(s["case"]["nseq"]):
        xi = _x_rows(s, i)(x)
        head = initial[i] if initial is not None else xi.new_zeros(w - 1, xi.shape[1])
        full = torch.cat([head, xi])
        taps = full.unfold(0, w, 1) if len(xi) else xi.new_zeros(0, xi.shape[1], w)
        p = torch.einsum("tcw,cw->tc", taps, weight) + bias
        outs.append(p * torch.sigmoid(p))
        finals.append(full[len(xi):])
    out = torch.cat(outs) if s["offsets"] is not None else torch.stack(outs)
    return out, torch.stack(finals)


def _x_conv(s):
    out, final = _x_conv_forward(s, s["x"], s["weight"], s["bias"], s["initial"])
    return {"out": out, "final": final}


def _x_conv_backward(s):
    leaves = [s["x"].clone(), s["weight"], s["bias"]]
    if s["initial"] is not None:
        leaves.append(s["initial"])
    leaves = [t.requires_grad_(True) for t in leaves]
    out, _ = _x_conv_forward(s, *leaves[:3], leaves[3] if len(leaves) > 3 else None)
    g = list(torch.autograd.grad((out * s["dout"]).sum(), leaves)) + [None]
    return {"dx": g[0], "dweight": g[1], "dbias": g[2], "dinitial": g[3]}


def _x_conv_step(s):
    pool, outs = s["state"].clone(), []
    for i, (src, dst) in enumerate(zip(s["slots"].tolist(), s["slots_out"].tolist())):
        full = torch.cat([s["state"][src], s["x"][i:i + 1]])
        p = torch.einsum("wc,cw->c", full, s["weight"]) + s["bias"]
        outs.append(p * torch.sigmoid(p))
        pool[dst] = full[1:]
    return {"out": torch.stack(outs), "state": pool}


def _x_scan_rows(u, delta, A, B, C, D, z, bias, h):
    """One batch of equally long sequences: u [nb, length, d], h [nb, d, n]; token by token."""
    dg = A.shape[0] // B.shape[-2]
    ys = []
    for t in range(u.shape[1]):
        dl = torch.logaddexp(delta[:, t] + bias, torch.zeros_like(delta[:, t]))
        Bt, Ct = (torch.repeat_interleave(m[:, t], dg, 1) for m in (B, C))
        h = h * torch.exp(torch.einsum("bc,cs->bcs", dl, A)) + Bt * (dl * u[:, t]).unsqueeze(2)
        ys.append(torch.einsum("bcs,bcs->bc", h, Ct) + D * u[:, t])
    y = torch.stack(ys, 1) if ys else u * 0
    return (y if z is None else y * z * torch.sigmoid(z)), h


def _x_scan_forward(s, v):
    """v: the inputs by name, so that the same code serves for gradients."""
    def start(i, j):
        return v["initial"][i:j] if v["initial"] is not None else v["A"].new_zeros(
            j - i, *v["A"].shape)

    if s["offsets"] is None:
        return _x_scan_rows(v["u"], v["delta"], v["A"], v["B"], v["C"], v["D"], v["z"],
                            v["delta_bias"], start(0, s["case"]["nseq"]))
    outs, finals = [], []
    for i in range(s["case"]["nseq"]):
        cut = _x_rows(s, i)
        seq = [cut(v[k]).unsqueeze(0) if v[k] is not None else None
               for k in ("u", "delta", "B", "C", "z")]
        out, h = _x_scan_rows(seq[0], seq[1], v["A"], seq[2], seq[3], v["D"], seq[4],
                              v["delta_bias"], start(i, i + 1))
        outs.append(out[0])
        finals.append(h)
    return torch.cat(outs), torch.cat(finals)


def _x_scan(s):
    out, final = _x_scan_forward(s, s)
    return {"out": out, "final": final}


def _x_scan_backward(s):
    c = s["case"]
    # the graph keeps about eight [d, n] states of 8 bytes per token
    if 64.0 * _tokens(c) * c["d"] * c["n"] > 8.0e10:
        return None
    names = [k for k in ("u", "delta", "A", "B", "C", "D", "z", "delta_bias", "initial")
             if s[k] is not None]
    v = dict(s)
    for k in names:
        v[k] = s[k].clone().requires_grad_(True)
    out, _ = _x_scan_forward(s, v)
    g = dict(zip(names, torch.autograd.grad((out * s["dout"]).sum(), [v[k] for k in names])))
    return {"du": g["u"], "ddelta": g["delta"], "dA": g["A"], "dB": g["B"], "dC": g["C"],
            "dD": g["D"], "dz": g.get("z"), "ddelta_bias": g["delta_bias"],
            "dinitial": g.get("initial")}


def _x_scan_step(s):
    pool = s["state"].clone()
    one = [s[k].unsqueeze(1) for k in ("u", "delta", "B", "C", "z")]
    out, h = _x_scan_rows(one[0], one[1], s["A"], one[2], one[3], s["D"], one[4],
                          s["delta_bias"], pool[s["slots"]])
    pool[s["slots_out"]] = h
    return {"out": out[:, 0], "state": pool}


_EXACT = {"norm": _x_norm, "norm_backward": _x_norm_backward, "conv": _x_conv,
          "conv_backward": _x_conv_backward, "conv_step": _x_conv_step, "scan": _x_scan,
          "scan_backward": _x_scan_backward, "scan_step": _x_scan_step}
