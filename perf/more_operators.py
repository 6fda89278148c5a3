"""More sequence-layer operators: the cases that are measured, their plain forms and definitions.

The operators are the parts of a layer whose memory is a matrix for each head instead of a few
states for each channel, next to the selective scan:

  attn   linear attention with a decay for each head and token:
         S[t] = exp(g[t]) S[t-1] + k[t] v[t]^T,  o[t] = scale S[t]^T q[t]
  gnorm  group norm, channels last, with SiLU or a gate: over each token's groups (what follows the
         attention's heads) or over all tokens of a sequence (frames of a spectrogram)

Each has its form for whole sequences (prompts) and its backward pass (training); attn has its form
for single tokens, which moves states within a pool.  `run` computes the plain form (elementary
torch operations in 32 bits, rounded once at the end; decays are summed in 64) where `own` is false,
and calls the package where it is true.
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
        dict(name="attn_step_one", op="attn_step", nseq=1, heads=32, groups=32, dk=64, dv=64,
             dtype="bf16"),
        # many sequences being answered, their states scattered over a pool
        dict(name="attn_step_many", op="attn_step", nseq=128, heads=16, groups=16, dk=128, dv=128,
             dtype="bf16"),
        # one long prompt: few heads, so time itself has to be split
        dict(name="attn_prompt_long", op="attn", nseq=1, length=16384, heads=16, groups=16, dk=128,
             dv=128, dtype="bf16", packed=False, initial=False),
        # a batch of prompts that continue from earlier states; heads share queries and keys
        dict(name="attn_prompt_batch", op="attn", nseq=8, length=2048, heads=32, groups=4, dk=128,
             dv=64, dtype="bf16", packed=False, initial=True),
        # ragged prompts packed one after another, odd head counts and sizes, 32 bits
        dict(name="attn_packed_odd", op="attn", nseq=37, length=10007, heads=6, groups=3, dk=40,
             dv=72, dtype="f32", packed=True, initial=True),
        # a training step's reverse pass
        dict(name="attn_train", op="attn_backward", nseq=4, length=2048, heads=16, groups=16,
             dk=128, dv=128, dtype="bf16", packed=False, initial=False),
        # the same on packed documents of odd lengths
        dict(name="attn_train_packed", op="attn_backward", nseq=13, length=4001, heads=8, groups=8,
             dk=64, dv=96, dtype="f16", packed=True, initial=True),
        # a few tokens of answers: the norm of every head, gated, behind the attention
        dict(name="gnorm_few", op="gnorm", nseq=16, length=1, d=4096, groups=32, dtype="bf16",
             packed=False, act="gate"),
        # a long prompt: the same for every token
        dict(name="gnorm_prompt", op="gnorm", nseq=16384, length=1, d=2048, groups=16,
             dtype="bf16", packed=False, act="gate"),
        # frames of spectrograms: statistics over a whole sequence
        dict(name="gnorm_frames", op="gnorm", nseq=8, length=4096, d=1024, groups=32, dtype="bf16",
             packed=False, act="silu"),
        # training: gradients of the gated norm of every head
        dict(name="gnorm_train", op="gnorm_backward", nseq=8192, length=1, d=2048, groups=16,
             dtype="bf16", packed=False, act="gate"),
        # training on packed recordings of odd lengths, in 32 bits
        dict(name="gnorm_train_packed", op="gnorm_backward", nseq=23, length=20011, d=330, groups=6,
             dtype="f32", packed=True, act="silu"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn_step", "attn", "attn", "attn", "attn_backward", "attn_backward", "gnorm",
                     "gnorm", "gnorm_backward"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f16", "f32"])
    if op.startswith("gnorm"):
        groups = rng.choice([1, 4, 6, 8, 16, 32])
        each = _log(rng, 8, 256)
        if rng.random() < 0.7:
            each = (each + 7) // 8 * 8
        d = groups * each
        most = 1 << 24 if dtype == "f32" or op == "gnorm_backward" else 1 << 25
        tokens = _log(rng, 4, max(5, min(16384, most // d)))
        act = rng.choice(["none", "silu", "gate", "gate"])
        if rng.random() < 0.5:  # every token by itself
            return dict(op=op, nseq=tokens, length=1, d=d, groups=groups, dtype=dtype,
                        packed=False, act=act)
        packed = rng.random() < 0.5
        nseq = _log(rng, 1, max(1, min(32, tokens // 4)))
        return dict(op=op, nseq=nseq, length=tokens if packed else tokens // nseq, d=d,
                    groups=groups, dtype=dtype, packed=packed, act=act)
    groups = rng.choice([1, 2, 3, 4, 8, 16])
    heads = groups * rng.choice([1, 1, 1, 2, 4])
    sizes = [16, 24, 32, 40, 64, 64, 72, 96, 128, 128, 192, 256]
    case = dict(op=op, heads=heads, groups=groups, dk=rng.choice(sizes), dv=rng.choice(sizes),
                dtype=dtype)
    state = heads * case["dk"] * case["dv"]
    if op == "attn_step":
        case["nseq"] = _log(rng, 1, max(2, min(256, (1 << 25) // state)))
        return case
    most = 1 << 24 if op == "attn_backward" or dtype == "f32" else 1 << 25
    row = heads * max(case["dk"], case["dv"])
    work_most = 1 << (31 if op == "attn_backward" else 32)
    tokens = _log(rng, 16, max(17, min(16384, most // row, work_most // state)))
    nseq = _log(rng, 1, max(1, min(32, tokens // 8)))
    packed = rng.random() < 0.4
    case.update(nseq=nseq, length=tokens if packed else tokens // nseq, packed=packed,
                initial=rng.random() < 0.5)
    return case


def _tokens(case):
    return case["length"] if case["packed"] else case["nseq"] * case["length"]


def work(case):
    op, e = case["op"], _SIZE[case["dtype"]]
    if op.startswith("gnorm"):
        el = _tokens(case) * case["d"]
        stats, gate = case["nseq"] * case["groups"] * 8, case["act"] == "gate"
        if op == "gnorm":
            return {"bytes": el * e * (2 + gate) + stats + 8 * case["d"], "flops": el * 12}
        return {"bytes": el * e * (3 + 2 * gate) + stats + 16 * case["d"], "flops": el * 25}
    heads, dk, dv = case["heads"], case["dk"], case["dv"]
    state = case["nseq"] * heads * dk * dv
    if op == "attn_step":
        row = 2 * case["groups"] * dk + 2 * heads * dv + heads
        return {"bytes": case["nseq"] * row * e + 8 * state, "flops": 5 * state}
    tokens = _tokens(case)
    qk, v = tokens * case["groups"] * dk * e, tokens * heads * dv * e
    g = tokens * heads * e
    if op == "attn":
        return {"bytes": 2 * qk + 2 * v + g + 4 * state * (1 + case["initial"]),
                "flops": 5 * tokens * heads * dk * dv}
    return {"bytes": 4 * qk + 3 * v + 2 * g + 8 * state * case["initial"],
            "flops": 16 * tokens * heads * dk * dv}


# ---- inputs ---------------------------------------------------------------------------------


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _normal(g, *shape, dtype=torch.float32, scale=1.0):
    x = torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)
    return (x * scale).to(dtype)


def _offsets(g, nseq, total):
    """Cuts at random places: lengths from 0 up."""
    cuts = torch.randint(0, total + 1, (nseq - 1,), generator=g, device="cuda")
    cuts = torch.sort(cuts)[0]
    ends = torch.tensor([0], device="cuda"), torch.tensor([total], device="cuda")
    return torch.cat([ends[0], cuts, ends[1]]).to(torch.int64)


def _prepare_gnorm(case, g, dt):
    d = case["d"]
    lead = (case["length"],) if case["packed"] else (case["nseq"], case["length"])
    st = {"case": case, "offsets": _offsets(g, case["nseq"], case["length"]) if case["packed"]
          else None}
    # channels lie at levels of their own, as bins of a spectrogram do
    st["x"] = (_normal(g, *lead, d) * 1.5 + _normal(g, d)).to(dt)
    st["weight"] = (1.0 + 0.2 * _normal(g, d)).contiguous()
    st["bias"] = 0.1 * _normal(g, d)
    st["z"] = None
    if case["act"] == "gate":  # the gate is the second half of a projection
        st["z"] = _normal(g, *lead, 2 * d, dtype=dt)[..., d:]
    if case["op"] == "gnorm_backward":
        st["dout"] = _normal(g, *lead, d, dtype=dt, scale=0.5)
        mean, rstd = _stats(st)  # what the forward pass has kept
        st["mean"], st["rstd"] = mean.float().contiguous(), rstd.float().contiguous()
    return st


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    dt = _DTYPES[case["dtype"]]
    if op.startswith("gnorm"):
        return _prepare_gnorm(case, g, dt)
    nseq, heads, groups, dk, dv = (case[k] for k in ("nseq", "heads", "groups", "dk", "dv"))
    step = op == "attn_step"
    packed = not step and case["packed"]
    lead = (nseq,) if step else ((case["length"],) if packed else (nseq, case["length"]))
    st = {"case": case, "offsets": _offsets(g, nseq, case["length"]) if packed else None}
    # queries, keys and values are columns of one projection
    wide = _normal(g, *lead, 2 * groups * dk + heads * dv, dtype=dt)
    st["q"] = wide[..., :groups * dk].unflatten(-1, (groups, dk))
    st["k"] = wide[..., groups * dk:2 * groups * dk].unflatten(-1, (groups, dk))
    st["v"] = wide[..., 2 * groups * dk:].unflatten(-1, (heads, dv))
    # heads remember from a few tokens to a thousand, and each token moves that
    rate = torch.exp(torch.rand(heads, generator=g, device="cuda") * math.log(500.0)) * 1e-3
    st["decay"] = (-rate * torch.exp(0.5 * _normal(g, *lead, heads))).to(dt)
    if step:
        pool = 2 * nseq + nseq // 2 + 1
        at = torch.randperm(pool, generator=g, device="cuda").to(torch.int64)
        st["slots"], st["slots_out"] = at[:nseq].contiguous(), at[nseq:2 * nseq].contiguous()
        st["state"] = _normal(g, pool, heads, dk, dv)
        return st
    st["initial"] = _normal(g, nseq, heads, dk, dv) if case["initial"] else None
    if op == "attn_backward":
        st["dout"] = _normal(g, *lead, heads, dv, dtype=dt, scale=0.5)
    return st


# ---- one pass -------------------------------------------------------------------------------


def run(state):
    op = state["case"]["op"]
    return (_OWN if own else _PLAIN)[op](state)


def _own_attn(s):
    out, final = _pkg().linear_attention(s["q"], s["k"], s["v"], s["decay"],
                                         initial_state=s["initial"], offsets=s["offsets"],
                                         return_state=True)
    return {"out": out, "final": final}


def _own_attn_backward(s):
    r = _pkg().linear_attention_backward(s["dout"], s["q"], s["k"], s["v"], s["decay"],
                                         initial_state=s["initial"], offsets=s["offsets"])
    return {"dq": r.dq, "dk": r.dk, "dv": r.dv, "ddecay": r.ddecay, "dinitial": r.dinitial_state}


def _own_attn_step(s):
    out = _pkg().linear_attention_step(s["state"], s["q"], s["k"], s["v"], s["decay"],
                                       slots=s["slots"], slots_out=s["slots_out"])
    return {"out": out, "state": s["state"]}


def _own_gnorm(s):
    c = s["case"]
    r = _pkg().group_norm(s["x"], c["groups"], s["weight"], s["bias"], z=s["z"],
                          silu=c["act"] == "silu", offsets=s["offsets"])
    return {"out": r.out, "mean": r.mean, "rstd": r.rstd}


def _own_gnorm_backward(s):
    r = _pkg().group_norm_backward(s["dout"], s["x"], s["mean"], s["rstd"], s["weight"], s["bias"],
                                   z=s["z"], silu=s["case"]["act"] == "silu", offsets=s["offsets"])
    return {"dx": r.dx, "dz": r.dz, "dweight": r.dweight, "dbias": r.dbias}


# ---- plain forms ----------------------------------------------------------------------------

_CHUNK = 64


def _sigmoid(x):
    return 1.0 / (1.0 + torch.exp(-x))


def _places(s, x):
    """Sequences laid out in whole chunks, one after another: where every token goes, how many
    chunks there are at most, every chunk's sequence, every sequence's chunks and tokens."""
    n = s["case"]["nseq"]
    if s["offsets"] is None:
        o = torch.arange(n + 1, device=x.device) * x.shape[1]
        tokens = n * x.shape[1]
    else:
        o, tokens = s["offsets"], x.shape[0]
    lens = o[1:] - o[:-1]
    seq = torch.repeat_interleave(torch.arange(n, device=x.device), lens, output_size=tokens)
    ends = torch.cumsum((lens + _CHUNK - 1) // _CHUNK, 0)
    begins = ends - (lens + _CHUNK - 1) // _CHUNK
    place = begins[seq] * _CHUNK + torch.arange(tokens, device=x.device) - o[seq]
    count = -(-tokens // _CHUNK) + n
    of = torch.searchsorted(ends, torch.arange(count, device=x.device), right=True)
    return place, count, of, begins, ends, lens


def _spread(x, place, count, heads=None):
    """[..., h, d] -> [chunks, heads, tokens, d] in 32 bits, zeros behind a sequence's end."""
    x = x.float().reshape(-1, *x.shape[-2:])
    if heads is not None and heads != x.shape[1]:
        x = x.repeat_interleave(heads // x.shape[1], dim=1)
    full = x.new_zeros(count * _CHUNK, *x.shape[1:])
    full[place] = x
    return full.view(count, _CHUNK, *x.shape[1:]).transpose(1, 2)


def _linear(x, y, z, g, of, begins, ends, initial):
    """o[i] = sum_{j<=i} exp(G[i] - G[j]) (x[i] y[j]) z[j] + exp(G[i]) x[i] initial, and the states
    behind every chunk: the sums over a chunk as products, those over chunks as one more."""
    G = torch.cumsum(g.double(), dim=2)  # [chunks, heads, tokens], within the chunk
    i = torch.arange(_CHUNK, device=x.device)
    D = torch.where(i[:, None] >= i, torch.exp(G[..., :, None] - G[..., None, :]), 0.0).float()
    out = ((x @ y.transpose(-1, -2)) * D) @ z
    left = torch.exp(G[..., -1:] - G).float()
    own_states = (y * left[..., None]).transpose(-1, -2) @ z  # [chunks, heads, dk, dv]
    total = torch.cumsum(G[..., -1], dim=0)  # behind every chunk
    c = torch.arange(len(of), device=x.device)
    same = (of[:, None] == of) & (c[:, None] >= c)
    M = torch.where(same, torch.exp((total[:, None] - total).permute(2, 0, 1)), 0.0).float()
    heads, shape = x.shape[1], own_states.shape
    after = (M @ own_states.transpose(0, 1).reshape(heads, len(of), -1)).view(
        heads, shape[0], *shape[2:]).transpose(0, 1)
    if initial is not None:
        some = of.clamp(max=len(begins) - 1)
        first = total[begins.clamp(max=len(of) - 1)] - G[begins.clamp(max=len(of) - 1), :, -1]
        since = torch.exp(total - first[some]).float()
        after = after + since[..., None, None] * initial[some]
    before = torch.roll(after, 1, dims=0)
    start = torch.zeros(len(of), dtype=torch.bool, device=x.device)
    some = ends > begins
    start[begins.clamp(max=len(of) - 1)] |= some
    blank = torch.zeros_like(after) if initial is None else initial[of.clamp(max=len(begins) - 1)]
    before = torch.where(start[:, None, None, None], blank, before)
    return out + (x * torch.exp(G).float()[..., None]) @ before, after


def _final(after, begins, ends, initial):
    got = after[(ends - 1).clamp(min=0)]
    rest = torch.zeros_like(got) if initial is None else initial
    return torch.where((ends > begins)[:, None, None, None], got, rest)


def _gather(out, place, like):
    """[chunks, heads, tokens, d] -> the tokens' rows, of the type and lead of `like`."""
    out = out.transpose(1, 2).reshape(-1, out.shape[1], out.shape[3])[place]
    return out.reshape(*like.shape[:-2], *out.shape[1:])


def _plain_attn(s):
    heads, scale = s["v"].shape[-2], s["q"].shape[-1] ** -0.5
    place, count, of, begins, ends, _ = _places(s, s["q"])
    q, k, v = (_spread(s[n], place, count, heads) for n in ("q", "k", "v"))
    g = _spread(s["decay"][..., None], place, count)[..., 0]
    out, after = _linear(q, k, v, g, of, begins, ends, s["initial"])
    return {"out": _gather(out * scale, place, s["v"]).to(s["v"].dtype),
            "final": _final(after, begins, ends, s["initial"])}


def _plain_attn_backward(s):
    heads, dk = s["v"].shape[-2], s["q"].shape[-1]
    groups, dt, scale = s["q"].shape[-2], s["q"].dtype, dk ** -0.5
    place, count, of, begins, ends, lens = _places(s, s["q"])
    q, k, v, do = (_spread(s[n], place, count, heads) for n in ("q", "k", "v", "dout"))
    decay = s["decay"].reshape(-1, heads)
    g = _spread(decay[..., None], place, count)[..., 0]
    init = s["initial"].transpose(-1, -2) if s["initial"] is not None else None
    dq, _ = _linear(do, v, k, g, of, begins, ends, init)

    # the same with time reversed: a token's state then decays by its follower's rate
    seq = of[place // _CHUNK]
    back = 2 * begins[seq] * _CHUNK + lens[seq] - 1 - place
    rq, rk, rv, rdo = (_spread(s[m], back, count, heads) for m in ("q", "k", "v", "dout"))
    rg = _spread(torch.roll(decay, -1, dims=0)[..., None], back, count)[..., 0]
    dv, _ = _linear(rk, rq, rdo, rg, of, begins, ends, None)
    dkey, after = _linear(rv, rdo, rq, rg, of, begins, ends, None)
    dinit = None
    if s["initial"] is not None:
        got = _final(after, begins, ends, None).transpose(-1, -2)
        first = torch.exp(g[begins.clamp(max=count - 1), :, 0].double()).float()
        dinit = got * first[..., None, None] * scale

    # pairs j < t <= i: what the rows from t on have taken less what they have given
    rows = lambda x, at: _gather(x, at, s["v"]).reshape(-1, heads, x.shape[-1])  # noqa: E731
    dq, dv, dkey = rows(dq, place), rows(dv, back), rows(dkey, back)
    wide = lambda m: s[m].reshape(-1, groups, dk).repeat_interleave(  # noqa: E731
        heads // groups, dim=1).double()
    net = (wide("q") * dq.double() - wide("k") * dkey.double()).sum(-1)
    total = torch.cumsum(net, dim=0)
    tail = torch.cumsum(lens, 0)[seq] - 1
    dg = total[tail] - total + net

    def shared(x):
        return x.view(-1, groups, heads // groups, dk).sum(dim=2).mul(scale).to(dt)

    return {"dq": shared(dq).view(s["q"].shape), "dk": shared(dkey).view(s["k"].shape),
            "dv": dv.mul(scale).to(dt).view(s["v"].shape),
            "ddecay": dg.mul(scale).to(dt).view(s["decay"].shape), "dinitial": dinit}


def _plain_attn_step(s):
    heads, groups, dk = s["v"].shape[-2], s["q"].shape[-2], s["q"].shape[-1]
    q, k = (s[n].float().repeat_interleave(heads // groups, dim=1) for n in ("q", "k"))
    h = (torch.exp(s["decay"].float())[..., None, None] * s["state"][s["slots"]]
         + k[..., None] * s["v"].float()[..., None, :])
    s["state"][s["slots_out"]] = h
    out = (h * q[..., None]).sum(dim=-2) * dk ** -0.5
    return {"out": out.to(s["v"].dtype), "state": s["state"]}


def _stats(s):
    """Mean and inverse deviation of every sequence's groups, [sequences, groups] in 64 bits."""
    groups, x = s["case"]["groups"], s["x"].float()
    if s["offsets"] is None:
        y = x.unflatten(-1, (groups, -1)).transpose(1, 2).flatten(2)
        mean = y.mean(dim=2, dtype=torch.float64)
        var = (y - mean.float()[..., None]).square().mean(dim=2, dtype=torch.float64)
        return mean, torch.rsqrt(var + 1e-5)
    seq, lens = _whose(s)
    y = x.unflatten(-1, (groups, -1))
    count = (lens * y.shape[2]).clamp(min=1)[:, None]

    def total(v):  # of every sequence
        return v.new_zeros(len(lens), groups, dtype=torch.float64).index_add_(
            0, seq, v.sum(dim=2, dtype=torch.float64))

    mean = total(y) / count
    var = total((y - mean.float()[seq][..., None]).square()) / count
    return mean, torch.rsqrt(var + 1e-5)


def _whose(s):
    o = s["offsets"]
    lens = o[1:] - o[:-1]
    return torch.repeat_interleave(torch.arange(len(lens), device=o.device), lens,
                                   output_size=s["x"].shape[0]), lens


def _to_tokens(s, v):
    """[sequences, groups] -> [..., groups, 1] beside the tokens."""
    if s["offsets"] is None:
        return v[:, None, :, None]
    return v[_whose(s)[0]][..., None]


def _plain_gnorm(s):
    groups = s["case"]["groups"]
    mean, rstd = (v.float() for v in _stats(s))
    x = s["x"].float().unflatten(-1, (groups, -1))
    y = ((x - _to_tokens(s, mean)) * _to_tokens(s, rstd)).flatten(-2) * s["weight"] + s["bias"]
    if s["case"]["act"] == "silu":
        y = y * _sigmoid(y)
    if s["z"] is not None:
        z = s["z"].float()
        y = y * (z * _sigmoid(z))
    return {"out": y.to(s["x"].dtype), "mean": mean, "rstd": rstd}


def _plain_gnorm_backward(s):
    groups, dt = s["case"]["groups"], s["x"].dtype
    x, g = s["x"].float().unflatten(-1, (groups, -1)), s["dout"].float()
    rstd = _to_tokens(s, s["rstd"])
    n = (x - _to_tokens(s, s["mean"])) * rstd
    y = n.flatten(-2) * s["weight"] + s["bias"]
    dz = None
    if s["z"] is not None:
        z = s["z"].float()
        sg = _sigmoid(z)
        p = y * _sigmoid(y) if s["case"]["act"] == "silu" else y
        dz = (g * p * (sg * (1.0 + z * (1.0 - sg)))).to(dt)
        g = g * (z * sg)
    if s["case"]["act"] == "silu":
        sg = _sigmoid(y)
        g = g * (sg * (1.0 + y * (1.0 - sg)))
    over = tuple(range(g.dim() - 1))
    dw = (g.double() * n.flatten(-2)).sum(dim=over).float()
    db = g.sum(dim=over, dtype=torch.float64).float()
    w = (g * s["weight"]).unflatten(-1, (groups, -1))
    if s["offsets"] is None:
        def average(v):
            return v.mean(dim=(1, 3), dtype=torch.float64).float()
    else:
        seq, lens = _whose(s)
        count = (lens * x.shape[2]).clamp(min=1)[:, None]

        def average(v):
            return (v.new_zeros(len(lens), groups, dtype=torch.float64).index_add_(
                0, seq, v.sum(dim=2, dtype=torch.float64)) / count).float()
    dx = (w - _to_tokens(s, average(w)) - n * _to_tokens(s, average(w * n))) * rstd
    return {"dx": dx.flatten(-2).to(dt), "dz": dz, "dweight": dw, "dbias": db}


_PLAIN = {"attn": _plain_attn, "attn_backward": _plain_attn_backward,
          "attn_step": _plain_attn_step, "gnorm": _plain_gnorm,
          "gnorm_backward": _plain_gnorm_backward}
_OWN = {"attn": _own_attn, "attn_backward": _own_attn_backward, "attn_step": _own_attn_step,
        "gnorm": _own_gnorm, "gnorm_backward": _own_gnorm_backward}


# ---- the definitions in 64 bits -------------------------------------------------------------


def exact(case, seed):
    """The outputs of `run` from the definitions, token by token in 64 bits; gradients by
    differentiating the definition."""
    s = {k: (v.double() if isinstance(v, torch.Tensor) and v.is_floating_point() else v)
         for k, v in prepare(case, seed).items()}
    return _EXACT[case["op"]](s)


def _x_tokens(q, k, v, decay, S):
    """One batch of equally long sequences: q, k [nb, length, groups, dk], v [nb, length, heads,
    dv], S [nb, heads, dk, dv]."""
    each, outs = v.shape[2] // q.shape[2], []
    for t in range(q.shape[1]):
        qt, kt = (m[:, t].repeat_interleave(each, 1) for m in (q, k))
        S = S * torch.exp(decay[:, t])[..., None, None] + torch.einsum("bhd,bhe->bhde", kt, v[:, t])
        outs.append(torch.einsum("bhd,bhde->bhe", qt, S) / math.sqrt(q.shape[-1]))
    return (torch.stack(outs, 1) if outs else v * 0), S


def _x_forward(c, offsets, q, k, v, decay, initial):
    def start(i, j):
        return initial[i:j] if initial is not None else v.new_zeros(j - i, c["heads"], c["dk"],
                                                                    c["dv"])

    if offsets is None:
        return _x_tokens(q, k, v, decay, start(0, c["nseq"]))
    outs, finals, o = [], [], offsets.tolist()
    for i in range(c["nseq"]):
        out, S = _x_tokens(*(m[o[i]:o[i + 1]].unsqueeze(0) for m in (q, k, v, decay)),
                           start(i, i + 1))
        outs.append(out[0])
        finals.append(S)
    return torch.cat(outs), torch.cat(finals)


def _x_attn(s):
    out, final = _x_forward(s["case"], s["offsets"], s["q"], s["k"], s["v"], s["decay"],
                            s["initial"])
    return {"out": out, "final": final}


def _x_attn_backward(s):
    c = s["case"]
    # the graph keeps about three [dk, dv] states of 8 bytes per token and head
    if 24.0 * _tokens(c) * c["heads"] * c["dk"] * c["dv"] > 8.0e10:
        return None
    leaves = [s[n].clone().requires_grad_(True) for n in ("q", "k", "v", "decay")]
    init = s["initial"].clone().requires_grad_(True) if s["initial"] is not None else None
    out, _ = _x_forward(c, s["offsets"], *leaves, init)
    g = torch.autograd.grad((out * s["dout"]).sum(), leaves + ([init] if init is not None else []))
    return dict(zip(("dq", "dk", "dv", "ddecay", "dinitial"), [*g, None]))


def _x_attn_step(s):
    pool = s["state"].clone()
    out, S = _x_tokens(*(s[n].unsqueeze(1) for n in ("q", "k", "v", "decay")), pool[s["slots"]])
    pool[s["slots_out"]] = S
    return {"out": out[:, 0], "state": pool}


def _x_norm_one(x, groups):
    """Sequences [nb, length, d]: normalised, mean, inverse deviation."""
    parts = [p.flatten(1) for p in torch.chunk(x, groups, dim=2)]
    mean = torch.stack([p.mean(1) for p in parts], 1)
    rstd = torch.stack([(((p - p.mean(1, True)) ** 2).mean(1) + 1e-5) ** -0.5 for p in parts], 1)
    each = x.shape[2] // groups
    wide_mean, wide_rstd = (t.repeat_interleave(each, 1)[:, None] for t in (mean, rstd))
    return (x - wide_mean) * wide_rstd, mean, rstd


def _x_gnorm_forward(s, x, weight, bias, z):
    c = s["case"]
    if s["offsets"] is None:
        n, mean, rstd = _x_norm_one(x, c["groups"])
    else:
        o, parts = s["offsets"].tolist(), []
        for a, b in zip(o[:-1], o[1:]):
            one = _x_norm_one(x[a:b].unsqueeze(0), c["groups"]) if b > a else (
                x[a:a], x.new_zeros(1, c["groups"]), x.new_full((1, c["groups"]), 1e-5 ** -0.5))
            parts.append((one[0].reshape(b - a, x.shape[1]), one[1], one[2]))
        n, mean, rstd = (torch.cat(p) for p in zip(*parts))
    y = n * weight + bias
    if c["act"] == "silu":
        y = torch.nn.functional.silu(y)
    if z is not None:
        y = y * torch.nn.functional.silu(z)
    return y, mean, rstd


def _x_gnorm(s):
    out, mean, rstd = _x_gnorm_forward(s, s["x"], s["weight"], s["bias"], s["z"])
    return {"out": out, "mean": mean, "rstd": rstd}


def _x_gnorm_backward(s):
    names = [n for n in ("x", "weight", "bias", "z") if s[n] is not None]
    v = {n: s[n].clone().requires_grad_(True) for n in names}
    out, _, _ = _x_gnorm_forward(s, v["x"], v["weight"], v["bias"], v.get("z"))
    g = dict(zip(names, torch.autograd.grad((out * s["dout"]).sum(), [v[n] for n in names])))
    return {"dx": g["x"], "dz": g.get("z"), "dweight": g["weight"], "dbias": g["bias"]}


_EXACT = {"attn": _x_attn, "attn_backward": _x_attn_backward, "attn_step": _x_attn_step,
          "gnorm": _x_gnorm, "gnorm_backward": _x_gnorm_backward}
