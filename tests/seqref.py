"""Plain 64-bit forms of the sequence operators for the tests: the definitions of include/gbfft.h,
token by token, on CPU tensors.  Shares no code with the package."""
import torch

F64 = torch.float64


def softplus(x):
    return torch.logaddexp(x, torch.zeros_like(x))


def spans(x, offsets):
    """Row slices of every sequence: (leading index, slice)."""
    if offsets is None:
        return [(i, slice(0, x.shape[1])) for i in range(x.shape[0])]
    return [(None, slice(int(a), int(b))) for a, b in zip(offsets[:-1], offsets[1:])]


def cut(x, span):
    i, sl = span
    return x[sl] if i is None else x[i, sl]


def conv(x, weight, bias, silu, initial, offsets):
    """out, final state."""
    w, outs, finals = weight.shape[1], [], []
    for q, sp in enumerate(spans(x, offsets)):
        xs = cut(x, sp)
        head = initial[q] if initial is not None else x.new_zeros(w - 1, x.shape[-1])
        full = torch.cat([head, xs])
        rows = []
        for t in range(xs.shape[0]):
            p = bias if bias is not None else x.new_zeros(x.shape[-1])
            for k in range(w):
                p = p + weight[:, k] * full[t + k]
            rows.append(p * torch.sigmoid(p) if silu else p)
        outs.append(torch.stack(rows) if rows else xs)
        finals.append(full[full.shape[0] - (w - 1):])
    out = torch.cat(outs) if offsets is not None else torch.stack(outs)
    return out, torch.stack(finals)


def scan(u, delta, A, B, C, D, z, bias, use_softplus, initial, offsets, magnitude=False):
    """out, final state; with magnitude also, for every output, the size that rounding errors
    scale with: the same recurrence on absolute values, every step's relative error carried on."""
    dg = A.shape[0] // B.shape[-2]
    outs, finals, sizes = [], [], []
    for q, sp in enumerate(spans(u, offsets)):
        us, ds, Bs, Cs = (cut(t, sp) for t in (u, delta, B, C))
        zs = cut(z, sp) if z is not None else None
        h = initial[q] if initial is not None else A.new_zeros(A.shape)
        H, E, rows, size = h.abs(), h.abs(), [], []
        for t in range(us.shape[0]):
            e = ds[t] + bias if bias is not None else ds[t]
            d = softplus(e) if use_softplus else e
            a = torch.exp(d[:, None] * A)
            b = (d * us[t])[:, None] * Bs[t].repeat_interleave(dg, 0)
            h = a * h + b
            c = Cs[t].repeat_interleave(dg, 0)
            y = (c * h).sum(1)
            if D is not None:
                y = y + D * us[t]
            if zs is not None:
                y = y * zs[t] * torch.sigmoid(zs[t])
            rows.append(y)
            if magnitude:
                # a and b are off by a few units each, relative to their own size
                E = a * E + a * H * (1 + (d[:, None] * A).abs()) + b.abs()
                H = a * H + b.abs()
                s = (c.abs() * (E + H)).sum(1)
                if D is not None:
                    s = s + (D * us[t]).abs()
                if zs is not None:
                    s = s * (zs[t] * torch.sigmoid(zs[t])).abs()
                size.append(s)
        outs.append(torch.stack(rows) if rows else us * 0)
        finals.append(h)
        sizes.append(torch.stack(size) if size else us * 0)
    join = torch.cat if offsets is not None else torch.stack
    res = join(outs), torch.stack(finals)
    return (*res, join(sizes)) if magnitude else res


def norm(x, residual, weight, eps):
    r = x + residual if residual is not None else x
    return r / torch.sqrt((r * r).mean(-1, keepdim=True) + eps) * weight, r


def e4m3(y, group):
    """Values and scales: 3 bits behind the leading one, steps of 2^-9 below 2^-6."""
    outs, scales = [], []
    for part in torch.split(y, group or y.shape[-1], dim=-1):
        s = part.abs().amax(-1, keepdim=True) / 448.0
        v = part / torch.where(s > 0, s, torch.ones_like(s))
        step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
        outs.append(torch.round(v / step) * step)
        scales.append(s)
    return torch.cat(outs, -1), torch.cat(scales, -1)
