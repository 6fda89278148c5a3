"""Sequence operators: short causal convolution, selective state-space scan, residual norm.

Filters along the tokens of a sequence whose coefficients change from token to token (so that no
transform plan describes them), and the norm between two such layers; see include/gbfft.h for the
definitions.  Like the rest of the binding this marshals torch tensors to device pointers and the
current CUDA stream: every step runs in the library's kernels.

    out, state = causal_conv(x, weight, bias, silu=True, return_state=True)    # x [b, l, d]
    y, h = selective_scan(u, delta, A, B, C, D=D, z=z, softplus=True, return_state=True)
    r = residual_norm(x, weight, residual=res)                      # r.out, r.residual
    q = residual_norm(x, weight, out_dtype=torch.float8_e4m3fn, group=128)     # q.out, q.scale

Sequences are [sequences, tokens, channels] or, with `offsets` (int64, on the device, sequences + 1
ascending values from 0 to the number of tokens), packed [tokens, channels].  The last axis is
contiguous, the others may have any stride: halves of a projection need no copy.  The *_backward
calls return the gradients; nothing is recorded for autograd.  The *_step calls take one token per
sequence and move its state from slots[i] to slots_out[i] of a pool (in place by default).
Outputs and workspaces are allocated by torch on the stream that the call runs on.
"""
import contextlib
import ctypes
from typing import NamedTuple, Optional

_i32, _i64, _vp = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p

F32, BF16, F16, E4M3 = 0, 1, 2, 3


class Seq(ctypes.Structure):  # fft_seq
    _fields_ = [("data", _vp), ("seq_stride", _i64), ("tok_stride", _i64)]


class ConvDesc(ctypes.Structure):  # fft_conv_desc
    _fields_ = [("dtype", _i32), ("param_dtype", _i32), ("width", _i32), ("silu", _i32),
                ("nseq", _i64), ("length", _i64), ("channels", _i64), ("offsets", _vp),
                ("weight", _vp), ("bias", _vp), ("initial_state", _vp), ("x", Seq)]


class ScanDesc(ctypes.Structure):  # fft_scan_desc
    _fields_ = [("dtype", _i32), ("softplus", _i32), ("nseq", _i64), ("length", _i64),
                ("channels", _i64), ("groups", _i64), ("states", _i64), ("offsets", _vp),
                ("A", _vp), ("D", _vp), ("delta_bias", _vp), ("initial_state", _vp), ("u", Seq),
                ("delta", Seq), ("B", Seq), ("C", Seq), ("z", Seq)]


class ScanGradsArg(ctypes.Structure):  # fft_scan_grads
    _fields_ = [("dout", Seq), ("dfinal_state", _vp), ("du", Seq), ("ddelta", Seq), ("dB", Seq),
                ("dC", Seq), ("dz", Seq), ("dA", _vp), ("dD", _vp), ("ddelta_bias", _vp),
                ("dinitial_state", _vp)]


class NormDesc(ctypes.Structure):  # fft_norm_desc
    _fields_ = [("dtype", _i32), ("res_dtype", _i32), ("param_dtype", _i32), ("out_dtype", _i32),
                ("rows", _i64), ("columns", _i64), ("group", _i64), ("eps", ctypes.c_float),
                ("weight", _vp)]


class ConvGrads(NamedTuple):
    dx: object
    dweight: object  # float32 [channels, width]
    dbias: Optional[object]  # float32 [channels]
    dinitial_state: Optional[object]


class ScanGrads(NamedTuple):
    du: object
    ddelta: object
    dA: object
    dB: object
    dC: object
    dD: Optional[object]
    dz: Optional[object]
    ddelta_bias: Optional[object]
    dinitial_state: Optional[object]


class NormOut(NamedTuple):
    out: object
    scale: Optional[object]  # float32 [rows, groups], 8-bit outputs
    residual: Optional[object]  # x + residual, None without a residual


class NormGrads(NamedTuple):
    dx: object
    dresidual: object  # the same tensor as dx where the types agree
    dweight: object


def declare(L):
    """Argument types of the sequence operators (called when the library is loaded)."""
    pc, ps, pn, pq = (ctypes.POINTER(t) for t in (ConvDesc, ScanDesc, NormDesc, Seq))
    sz = ctypes.c_size_t
    L.fft_conv_forward.argtypes = [pc, pq, _vp, _vp]
    L.fft_conv_workspace.argtypes = [pc, ctypes.POINTER(sz)]
    L.fft_conv_backward.argtypes = [pc, pq, _vp, pq, _vp, _vp, _vp, _vp, sz, _vp]
    L.fft_conv_step.argtypes = [pc, pq, _vp, _i64, _vp, _vp, _vp]
    L.fft_scan_workspace.argtypes = [ps, ctypes.c_int, ctypes.POINTER(sz)]
    L.fft_scan_forward.argtypes = [ps, pq, _vp, _vp, sz, _vp]
    L.fft_scan_backward.argtypes = [ps, ctypes.POINTER(ScanGradsArg), _vp, sz, _vp]
    L.fft_scan_step.argtypes = [ps, pq, _vp, _i64, _vp, _vp, _vp]
    L.fft_norm_forward.argtypes = [pn, _vp, _i64, _vp, _i64, _vp, _i64, _vp, _vp, _i64, _vp]
    L.fft_norm_workspace.argtypes = [pn, ctypes.POINTER(sz)]
    L.fft_norm_backward.argtypes = [pn, _vp, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _vp, _i64,
                                    _vp, _vp, sz, _vp]


SYMBOLS = ("fft_conv_forward", "fft_conv_workspace", "fft_conv_backward", "fft_conv_step",
           "fft_scan_workspace", "fft_scan_forward", "fft_scan_backward", "fft_scan_step",
           "fft_norm_forward", "fft_norm_workspace", "fft_norm_backward")


# ---- checks ---------------------------------------------------------------------------------

_CODES = {}


def _codes():
    if not _CODES:
        import torch

        _CODES.update({torch.float32: F32, torch.bfloat16: BF16, torch.float16: F16})
    return _CODES


def _lib():
    from . import lib

    return lib()


def _check(rc, what):
    if rc:
        from . import GbfftError

        raise GbfftError(rc, what)


def _dtype(t, what):
    code = _codes().get(getattr(t, "dtype", None))
    if code is None:
        raise TypeError(f"{what}: expected a float32, bfloat16 or float16 CUDA tensor")
    return code


def _need(t, like, shape, dtype, what):
    """t on like's device, of this dtype (None: like's) and shape, its last axis contiguous."""
    if not hasattr(t, "data_ptr") or not t.is_cuda or t.device != like.device:
        raise TypeError(f"{what}: expected a CUDA tensor on {like.device}")
    if t.dtype != (like.dtype if dtype is None else dtype):
        raise TypeError(f"{what}: expected {like.dtype if dtype is None else dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{what}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.stride(-1) != 1 and t.shape[-1] > 1:
        raise ValueError(f"{what}: the last axis must be contiguous")
    return t


def _flat(t, like, shape, dtype, what):
    """The address of a contiguous tensor, or None for None."""
    if t is None:
        return None
    _need(t, like, shape, dtype, what)
    if not t.is_contiguous():
        raise ValueError(f"{what}: tensor must be contiguous")
    return t.data_ptr()


def _on(t):
    """The tensor's device has to be the current one: the library launches there."""
    import torch

    if not t.is_cuda:
        raise TypeError("expected CUDA tensors")
    if t.device.index != torch.cuda.current_device():
        raise ValueError("expected tensors on the current CUDA device")


def _offsets(offsets, like):
    if offsets is None:
        return None
    import torch

    if offsets.dim() != 1 or offsets.numel() < 2:
        raise ValueError("offsets: expected one more value than sequences")
    return _flat(offsets, like, offsets.shape, torch.int64, "offsets")


def _seq(t, packed):
    return Seq(t.data_ptr(), 0, t.stride(0)) if packed else Seq(t.data_ptr(), t.stride(0), t.stride(1))


def _row(t):
    return Seq(t.data_ptr(), t.stride(0), 0)


def _groups(t, like, lead, what):
    """B or C: [..., groups, n] or [..., n], groups back to back."""
    if t.dim() == len(lead) + 1:
        t = t.unsqueeze(-2)
    _need(t, like, (*lead, *t.shape[-2:]), None, what)
    if t.shape[-2] > 1 and t.stride(-2) != t.shape[-1]:
        raise ValueError(f"{what}: the groups must lie back to back")
    return t


def _empty(like, shape=None, dtype=None):
    import torch

    return torch.empty(like.shape if shape is None else shape,
                       dtype=like.dtype if dtype is None else dtype, device=like.device)


def _out(out, like, shape=None):
    if out is None:
        return _empty(like, shape)
    return _need(out, like, like.shape if shape is None else shape, None, "out")


_SAME = contextlib.nullcontext()


def _stream(stream):
    """(context in which torch allocates for the stream, the stream's handle)."""
    import torch

    if stream is None:
        return _SAME, torch.cuda.current_stream().cuda_stream
    return torch.cuda.stream(stream), stream.cuda_stream


def _workspace(fn, args, like, what):
    import torch

    size = ctypes.c_size_t()
    _check(fn(*args, ctypes.byref(size)), what)
    if size.value == 0:
        return None, None, 0
    w = torch.empty(size.value, dtype=torch.uint8, device=like.device)
    return w, w.data_ptr(), size.value


def _lead(x, offsets, what):
    packed = offsets is not None
    if x.dim() != (2 if packed else 3):
        raise ValueError(f"{what}: expected [tokens, channels] with offsets, "
                         "[sequences, tokens, channels] without")
    nseq = offsets.numel() - 1 if packed else x.shape[0]
    return packed, nseq, (x.shape[0] if packed else x.shape[1])


# ---- short causal convolution ---------------------------------------------------------------


def _conv_desc(x, weight, bias, silu, initial_state, offsets, step=False):
    code = _dtype(x, "x")
    _on(x)
    d = x.shape[-1]
    off = _offsets(offsets, x)
    if step:
        packed, nseq, length = False, x.shape[0], 1
    else:
        packed, nseq, length = _lead(x, offsets, "x")
    _need(x, x, x.shape, None, "x")
    if weight.dim() != 2:
        raise ValueError("weight: expected [channels, width]")
    w = weight.shape[1]
    pcode = _dtype(weight, "weight")
    if pcode not in (F32, code):
        raise TypeError("weight: expected float32 or the type of x")
    return ConvDesc(code, pcode, w, int(bool(silu)), nseq, length, d, off,
                    _flat(weight, x, (d, w), weight.dtype, "weight"),
                    _flat(bias, x, (d,), weight.dtype, "bias"),
                    _flat(initial_state, x, (nseq, w - 1, d), None, "initial_state"),
                    _row(x) if step else _seq(x, packed))


def causal_conv(x, weight, bias=None, silu=False, initial_state=None, offsets=None,
                return_state=False, out=None, stream=None):
    """Short causal convolution of every channel (fft_conv_forward): weight [channels, width],
    bias [channels], both float32 or of x's type; initial_state [sequences, width-1, channels].
    Returns out, or (out, final_state)."""
    desc = _conv_desc(x, weight, bias, silu, initial_state, offsets)
    on, s = _stream(stream)
    with on:
        out = _out(out, x)
        state = _empty(x, (desc.nseq, desc.width - 1, desc.channels)) if return_state else None
        _check(_lib().fft_conv_forward(desc, _seq(out, offsets is not None),
                                       state.data_ptr() if return_state else None, s),
               "fft_conv_forward")
    return (out, state) if return_state else out


def causal_conv_backward(dout, x, weight, bias=None, silu=False, initial_state=None, offsets=None,
                         dfinal_state=None, stream=None):
    """Gradients of causal_conv from dout (and dfinal_state): ConvGrads."""
    import torch

    desc = _conv_desc(x, weight, bias, silu, initial_state, offsets)
    _need(dout, x, x.shape, None, "dout")
    packed, shape = offsets is not None, (desc.nseq, desc.width - 1, desc.channels)
    dfin = _flat(dfinal_state, x, shape, None, "dfinal_state")
    on, s = _stream(stream)
    with on:
        dx = _empty(x)
        dw = _empty(x, weight.shape, torch.float32)
        db = _empty(x, (desc.channels,), torch.float32) if bias is not None else None
        di = _empty(x, shape) if initial_state is not None else None
        w, wp, size = _workspace(_lib().fft_conv_workspace, (desc,), x, "fft_conv_workspace")
        _check(_lib().fft_conv_backward(desc, _seq(dout, packed), dfin, _seq(dx, packed),
                                        dw.data_ptr(), db.data_ptr() if db is not None else None,
                                        di.data_ptr() if di is not None else None, wp, size, s),
               "fft_conv_backward")
    return ConvGrads(dx, dw, db, di)


def _slot(t, like, nseq, what):
    if t is None:
        return None
    import torch

    return _flat(t, like, (nseq,), torch.int64, what)


def causal_conv_step(state, x, weight, bias=None, silu=False, slots=None, slots_out=None, out=None,
                     stream=None):
    """One token for each sequence (fft_conv_step): x [sequences, channels], state the pool
    [pool, width-1, channels], updated in place; slots, slots_out int64 [sequences]."""
    if x.dim() != 2:
        raise ValueError("x: expected [sequences, channels]")
    desc = _conv_desc(x, weight, bias, silu, None, None, step=True)
    pool = _flat(state, x, (state.shape[0], desc.width - 1, desc.channels), None, "state")
    on, s = _stream(stream)
    with on:
        out = _out(out, x)
        _check(_lib().fft_conv_step(desc, _row(out), pool, state.shape[0],
                                    _slot(slots, x, desc.nseq, "slots"),
                                    _slot(slots_out, x, desc.nseq, "slots_out"), s),
               "fft_conv_step")
    return out


# ---- selective scan -------------------------------------------------------------------------


def _scan_desc(u, delta, A, B, C, D, z, delta_bias, softplus, initial_state, offsets, step=False):
    import torch

    f32 = torch.float32
    code = _dtype(u, "u")
    _on(u)
    d = u.shape[-1]
    off = _offsets(offsets, u)
    if step:
        packed, nseq, length = False, u.shape[0], 1
    else:
        packed, nseq, length = _lead(u, offsets, "u")
    _need(u, u, u.shape, None, "u")
    _need(delta, u, u.shape, None, "delta")
    lead = u.shape[:-1]
    B, C = _groups(B, u, lead, "B"), _groups(C, u, lead, "C")
    groups, n = B.shape[-2:]
    if C.shape[-2:] != B.shape[-2:]:
        raise ValueError("C: expected the shape of B")
    view = _row if step else (lambda t: _seq(t, packed))
    return ScanDesc(code, int(bool(softplus)), nseq, length, d, groups, n, off,
                    _flat(A, u, (d, n), f32, "A"), _flat(D, u, (d,), f32, "D"),
                    _flat(delta_bias, u, (d,), f32, "delta_bias"),
                    _flat(initial_state, u, (nseq, d, n), f32, "initial_state"),
                    view(u), view(delta), view(B), view(C),
                    view(_need(z, u, u.shape, None, "z")) if z is not None else Seq())


def selective_scan(u, delta, A, B, C, D=None, z=None, delta_bias=None, softplus=False,
                   initial_state=None, offsets=None, return_state=False, out=None, stream=None):
    """Selective state-space scan (fft_scan_forward): u, delta, z [..., channels], A [channels, n],
    B, C [..., groups, n] or [..., n], D, delta_bias [channels]; states [sequences, channels, n].
    A, D, delta_bias and states are float32.  Returns out, or (out, final_state)."""
    import torch

    desc = _scan_desc(u, delta, A, B, C, D, z, delta_bias, softplus, initial_state, offsets)
    on, s = _stream(stream)
    with on:
        out = _out(out, u)
        state = (_empty(u, (desc.nseq, desc.channels, desc.states), torch.float32)
                 if return_state else None)
        w, wp, size = _workspace(_lib().fft_scan_workspace, (desc, 0), u, "fft_scan_workspace")
        _check(_lib().fft_scan_forward(desc, _seq(out, offsets is not None),
                                       state.data_ptr() if return_state else None, wp, size, s),
               "fft_scan_forward")
    return (out, state) if return_state else out


def selective_scan_backward(dout, u, delta, A, B, C, D=None, z=None, delta_bias=None,
                            softplus=False, initial_state=None, offsets=None, dfinal_state=None,
                            stream=None):
    """Gradients of selective_scan from dout (and dfinal_state): ScanGrads."""
    import torch

    f32 = torch.float32
    desc = _scan_desc(u, delta, A, B, C, D, z, delta_bias, softplus, initial_state, offsets)
    _need(dout, u, u.shape, None, "dout")
    packed, shape = offsets is not None, (desc.nseq, desc.channels, desc.states)
    dfin = _flat(dfinal_state, u, shape, f32, "dfinal_state")
    on, s = _stream(stream)
    with on:
        du, dd = _empty(u), _empty(u)
        dz = _empty(u) if z is not None else None
        dB, dC = _empty(u, B.shape), _empty(u, C.shape)
        dA = _empty(u, A.shape, f32)
        dD = _empty(u, D.shape, f32) if D is not None else None
        db = _empty(u, delta_bias.shape, f32) if delta_bias is not None else None
        di = _empty(u, shape, f32) if initial_state is not None else None
        at = [t.data_ptr() if t is not None else None for t in (dA, dD, db, di)]
        grads = ScanGradsArg(_seq(dout, packed), dfin, _seq(du, packed), _seq(dd, packed),
                             _seq(dB, packed), _seq(dC, packed),
                             _seq(dz, packed) if dz is not None else Seq(), *at)
        w, wp, size = _workspace(_lib().fft_scan_workspace, (desc, 1), u, "fft_scan_workspace")
        _check(_lib().fft_scan_backward(desc, grads, wp, size, s), "fft_scan_backward")
    return ScanGrads(du, dd, dA, dB, dC, dD, dz, db, di)


def selective_scan_step(state, u, delta, A, B, C, D=None, z=None, delta_bias=None, softplus=False,
                        slots=None, slots_out=None, out=None, stream=None):
    """One token for each sequence (fft_scan_step): u, delta, z [sequences, channels], B, C
    [sequences, groups, n] or [sequences, n], state the pool [pool, channels, n] float32, updated
    in place; slots, slots_out int64 [sequences]."""
    import torch

    if u.dim() != 2:
        raise ValueError("u: expected [sequences, channels]")
    desc = _scan_desc(u, delta, A, B, C, D, z, delta_bias, softplus, None, None, step=True)
    pool = _flat(state, u, (state.shape[0], desc.channels, desc.states), torch.float32, "state")
    on, s = _stream(stream)
    with on:
        out = _out(out, u)
        _check(_lib().fft_scan_step(desc, _row(out), pool, state.shape[0],
                                    _slot(slots, u, desc.nseq, "slots"),
                                    _slot(slots_out, u, desc.nseq, "slots_out"), s),
               "fft_scan_step")
    return out


# ---- residual norm --------------------------------------------------------------------------


def _rows(t):
    """[..., columns] as rows of one stride: (rows, stride)."""
    if t.dim() < 2:
        return (1, t.shape[-1])
    rows, stride = t.shape[-2], t.stride(-2)
    for k in range(t.dim() - 3, -1, -1):
        if t.shape[k] != 1 and rows != 1 and t.stride(k) != rows * stride:
            raise ValueError("expected rows at one stride")
        if rows == 1:
            stride = t.stride(k)
        rows *= t.shape[k]
    return rows, stride


def _norm_desc(x, res_dtype, weight, eps, out_code, group):
    code = _dtype(x, "x")
    _on(x)
    _need(x, x, x.shape, None, "x")
    d = x.shape[-1]
    rows, stride = _rows(x)
    pcode = _dtype(weight, "weight")
    if pcode not in (F32, code):
        raise TypeError("weight: expected float32 or the type of x")
    return NormDesc(code, _codes().get(res_dtype, -1), pcode, code if out_code is None else out_code,
                    rows, d, group, eps, _flat(weight, x, (d,), weight.dtype, "weight")), stride


def residual_norm(x, weight, residual=None, eps=1e-6, out_dtype=None, group=0, out=None,
                  inplace_residual=False, stream=None):
    """Root-mean-square norm of x + residual (fft_norm_forward), rows along the last axis: NormOut.
    residual is of x's type or float32, and so is the sum that is returned (written over it with
    inplace_residual).  out_dtype torch.float8_e4m3fn: out in 8 bits with scale
    [..., ceil(columns / group)], group 32, 64 or 128 columns, or 0 for one scale per row."""
    import torch

    e4m3 = out_dtype is not None and out_dtype != x.dtype
    if e4m3 and out_dtype != torch.float8_e4m3fn:
        raise TypeError("out_dtype: expected the type of x or torch.float8_e4m3fn")
    res_dtype = x.dtype if residual is None else residual.dtype
    desc, xs = _norm_desc(x, res_dtype, weight, eps, E4M3 if e4m3 else None, int(group))
    rp, rs, total, ts = None, 0, None, 0
    if residual is not None:
        _need(residual, x, x.shape, res_dtype, "residual")
        rp, rs = residual.data_ptr(), _rows(residual)[1]
    on, s = _stream(stream)
    with on:
        if out is None:
            out = _empty(x, None, out_dtype)
        else:
            _need(out, x, x.shape, out_dtype, "out")
        scale = None
        if e4m3:
            groups = -(-desc.columns // group) if group > 0 else 1
            scale = _empty(x, (*x.shape[:-1], groups), torch.float32)
        if residual is not None:
            total = residual if inplace_residual else _empty(x, None, res_dtype)
            ts = _rows(total)[1]
        _check(_lib().fft_norm_forward(desc, x.data_ptr(), xs, rp, rs, out.data_ptr(),
                                       _rows(out)[1], scale.data_ptr() if e4m3 else None,
                                       total.data_ptr() if total is not None else None, ts, s),
               "fft_norm_forward")
    return NormOut(out, scale, total)


def residual_norm_backward(dout, r, weight, dresidual=None, eps=1e-6, stream=None):
    """Gradients of residual_norm at its sum r (NormOut.residual, or x without a residual) from
    dout and from dresidual, the gradient that reaches the sum by itself: NormGrads."""
    import torch

    desc, gs = _norm_desc(dout, r.dtype, weight, eps, None, 0)
    _need(r, dout, dout.shape, r.dtype, "r")
    if dresidual is not None:
        _need(dresidual, dout, dout.shape, r.dtype, "dresidual")
    on, s = _stream(stream)
    with on:
        dr = _empty(dout, None, r.dtype)
        dx = dr if r.dtype == dout.dtype else _empty(dout)
        dw = _empty(dout, weight.shape, torch.float32)
        w, wp, size = _workspace(_lib().fft_norm_workspace, (desc,), dout, "fft_norm_workspace")
        _check(_lib().fft_norm_backward(
            desc, dout.data_ptr(), gs, r.data_ptr(), _rows(r)[1],
            dresidual.data_ptr() if dresidual is not None else None,
            _rows(dresidual)[1] if dresidual is not None else 0, dr.data_ptr(), _rows(dr)[1],
            None if dx is dr else dx.data_ptr(), _rows(dx)[1], dw.data_ptr(), wp, size, s),
            "fft_norm_backward")
    return NormGrads(dx, dr, dw)
