"""Plain 64-bit forms of linear attention and group norm for the tests: the definitions of
include/gbfft.h, token by token, on CPU tensors.  Shares no code with the package."""
import torch


def spans(x, offsets):
    if offsets is None:
        return [(i, slice(0, x.shape[1])) for i in range(x.shape[0])]
    return [(None, slice(int(a), int(b))) for a, b in zip(offsets[:-1], offsets[1:])]


def cut(x, span):
    i, sl = span
    return x[sl] if i is None else x[i, sl]


def attention(q, k, v, decay, scale, initial, offsets, magnitude=False):
    """out, final state; with magnitude also the same sums over absolute values for every output and
    state, which rounding errors scale with."""
    heads, dv, dk = v.shape[-2], v.shape[-1], q.shape[-1]
    each = heads // q.shape[-2]
    outs, finals, sizes, totals = [], [], [], []
    for n, sp in enumerate(spans(q, offsets)):
        qs, ks = (cut(t, sp).repeat_interleave(each, 1) for t in (q, k))
        vs, a = cut(v, sp), torch.exp(cut(decay, sp).clamp(max=0.0))
        S = initial[n] if initial is not None else v.new_zeros(heads, dk, dv)
        M, rows, size = S.abs(), [], []
        for t in range(qs.shape[0]):
            kv = ks[t][:, :, None] * vs[t][:, None, :]
            S = a[t][:, None, None] * S + kv
            rows.append(scale * (qs[t][:, :, None] * S).sum(1))
            if magnitude:
                M = a[t][:, None, None] * M + kv.abs()
                size.append(abs(scale) * (qs[t].abs()[:, :, None] * M).sum(1))
        outs.append(torch.stack(rows) if rows else vs * 0)
        finals.append(S)
        sizes.append(torch.stack(size) if size else vs * 0)
        totals.append(M)
    join = torch.cat if offsets is not None else torch.stack
    if not outs:
        return v * 0, v.new_zeros(0, heads, dk, dv)
    res = join(outs), torch.stack(finals)
    return (*res, join(sizes), torch.stack(totals)) if magnitude else res


def group_norm(x, groups, weight, bias, z, silu, eps, offsets):
    """out, mean, inverse deviation; x [sequences, tokens, channels] or packed [tokens, channels]."""
    outs, means, rstds = [], [], []
    for sp in spans(x, offsets):
        xs = cut(x, sp)
        p = xs.reshape(xs.shape[0], groups, xs.shape[1] // groups)
        if xs.shape[0]:
            mean = p.mean((0, 2))
            rstd = (((p - mean[:, None]) ** 2).mean((0, 2)) + eps) ** -0.5
        else:
            mean, rstd = x.new_zeros(groups), x.new_full((groups,), eps ** -0.5)
        y = ((p - mean[:, None]) * rstd[:, None]).reshape(xs.shape)
        if weight is not None:
            y = y * weight
        if bias is not None:
            y = y + bias
        if silu:
            y = y * torch.sigmoid(y)
        if z is not None:
            zs = cut(z, sp)
            y = y * zs * torch.sigmoid(zs)
        outs.append(y)
        means.append(mean)
        rstds.append(rstd)
    join = torch.cat if offsets is not None else torch.stack
    return join(outs), torch.stack(means), torch.stack(rstds)
