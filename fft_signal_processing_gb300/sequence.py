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
ascending values from 0 to the number of tokens), packed [tokens, channels]; sequences may be without
tokens and batches without sequences.  The last axis is
contiguous, the others may have any stride: halves of a projection need no copy.  The *_backward
calls return the gradients; nothing is recorded for autograd, and outputs of inputs that require
gradients do not require any.  The *_step calls take one token per
sequence and move its state from slots[i] to slots_out[i] of a pool (in place by default).
Outputs and workspaces are allocated by torch on the stream that the call runs on.
"""
import contextlib
import ctypes
import struct
from typing import NamedTuple, Optional

F32, BF16, F16, E4M3 = 0, 1, 2, 3

# The descriptors of include/gbfft.h, packed in one go: building a ctypes structure field by field
# takes longer than a single-token call's kernel.
_SEQ = struct.Struct("@P2q")  # fft_seq
_CONV = struct.Struct("@4i3q4PP2q")  # fft_conv_desc
_SCAN = struct.Struct("@2i5q5P" + "P2q" * 5)  # fft_scan_desc
_GRADS = struct.Struct("@P2qP" + "P2q" * 5 + "4P")  # fft_scan_grads
_NORM = struct.Struct("@4i3qfP")  # fft_norm_desc
_NONE = (0, 0, 0)  # an absent fft_seq


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
    desc, vp, i64, sz = ctypes.c_char_p, ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t
    L.fft_conv_forward.argtypes = [desc, desc, vp, vp]
    L.fft_conv_workspace.argtypes = [desc, ctypes.POINTER(sz)]
    L.fft_conv_backward.argtypes = [desc, desc, vp, desc, vp, vp, vp, vp, sz, vp]
    L.fft_conv_step.argtypes = [desc, desc, vp, i64, vp, vp, vp]
    L.fft_scan_workspace.argtypes = [desc, ctypes.c_int, ctypes.POINTER(sz)]
    L.fft_scan_forward.argtypes = [desc, desc, vp, vp, sz, vp]
    L.fft_scan_backward.argtypes = [desc, desc, vp, sz, vp]
    L.fft_scan_step.argtypes = [desc, desc, vp, i64, vp, vp, vp]
    L.fft_norm_forward.argtypes = [desc, vp, i64, vp, i64, vp, i64, vp, vp, i64, vp]
    L.fft_norm_workspace.argtypes = [desc, ctypes.POINTER(sz)]
    L.fft_norm_backward.argtypes = [desc, vp, i64, vp, i64, vp, i64, vp, i64, vp, i64, vp, vp, sz,
                                    vp]


SYMBOLS = ("fft_conv_forward", "fft_conv_workspace", "fft_conv_backward", "fft_conv_step",
           "fft_scan_workspace", "fft_scan_forward", "fft_scan_backward", "fft_scan_step",
           "fft_norm_forward", "fft_norm_workspace", "fft_norm_backward")


# ---- checks ---------------------------------------------------------------------------------

_L = torch = _CODES = _raw_stream = _device = None


def _setup():
    """Bind the library and torch on the first call."""
    global _L, torch, _CODES, _raw_stream, _device
    import torch as _torch

    from . import lib

    _CODES = {_torch.float32: F32, _torch.bfloat16: BF16, _torch.float16: F16}
    _raw_stream = getattr(_torch._C, "_cuda_getCurrentRawStream", None) or (
        lambda device: _torch.cuda.current_stream(device).cuda_stream)
    _device = getattr(_torch._C, "_cuda_getDevice", None) or _torch.cuda.current_device
    torch = _torch
    _L = lib()


def _check(rc, what):
    if rc:
        from . import GbfftError

        raise GbfftError(rc, what)


def _first(t, what):
    """(type code, device index) of the tensor that the others are compared with."""
    if _L is None:
        _setup()
    code, dev = _CODES.get(t.dtype), t.get_device()
    if code is None or dev < 0:
        raise TypeError(f"{what}: expected a float32, bfloat16 or float16 CUDA tensor")
    if dev != _device():  # the library launches there
        raise ValueError(f"{what}: expected a tensor on the current CUDA device")
    return code, dev


def _tell(t, dev, dtype, shape, what):
    """Say what is wrong with a tensor that failed a check."""
    if not hasattr(t, "data_ptr") or not t.is_cuda or t.get_device() != dev:
        raise TypeError(f"{what}: expected a CUDA tensor on device {dev}")
    if t.dtype != dtype:
        raise TypeError(f"{what}: expected {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{what}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    raise ValueError(f"{what}: the last axis must be contiguous, and parameters and states whole")


def _need(t, dev, dtype, shape, what):
    """t on the device, of this dtype and shape, its last axis contiguous."""
    if (t.dtype is not dtype or t.shape != shape or t.get_device() != dev
            or (t.stride(-1) != 1 and t.shape[-1] > 1)):
        _tell(t, dev, dtype, shape, what)
    return t


def _flat(t, dev, dtype, shape, what):
    """The address of a contiguous tensor, or 0 for None."""
    if t is None:
        return 0
    if (t.dtype is not dtype or t.shape != shape or t.get_device() != dev
            or not t.is_contiguous()):
        _tell(t, dev, dtype, shape, what)
    return t.data_ptr()


def _token(t, dev, dtype, shape, what):
    """The fields of an fft_seq of one token per sequence, [sequences, ...]: one question each, as
    a single-token call takes less time on the GPU than a dozen tensors asked twice."""
    st = t.stride()
    if (t.dtype is not dtype or t.shape != shape or t.get_device() != dev
            or (st[-1] != 1 and shape[-1] > 1)):
        _tell(t, dev, dtype, shape, what)
    if len(st) == 3 and shape[1] > 1 and st[1] != shape[2]:
        raise ValueError(f"{what}: the groups must lie back to back")
    return t.data_ptr(), st[0], 0


def _offsets(offsets, dev):
    if offsets is None:
        return 0
    if offsets.dim() != 1 or offsets.numel() < 1:
        raise ValueError("offsets: expected one more value than sequences")
    return _flat(offsets, dev, torch.int64, offsets.shape, "offsets")


def _seq(t, packed):
    """The fields of an fft_seq."""
    if t is None:
        return _NONE
    return (t.data_ptr(), 0, t.stride(0)) if packed else (t.data_ptr(), t.stride(0), t.stride(1))


def _row(t):
    return t.data_ptr(), t.stride(0), 0


def _ptr(t):
    return t.data_ptr() if t is not None else None


def _groups(t, dev, dtype, lead, what):
    """B or C: [..., groups, n] or [..., n], groups back to back."""
    if t.dim() == len(lead) + 1:
        t = t.unsqueeze(-2)
    shape = tuple(t.shape)
    if (t.dtype is not dtype or shape[:-2] != lead or t.get_device() != dev
            or (t.stride(-1) != 1 and shape[-1] > 1)):
        _tell(t, dev, dtype, (*lead, *shape[-2:]), what)
    if shape[-2] > 1 and t.stride(-2) != shape[-1]:
        raise ValueError(f"{what}: the groups must lie back to back")
    return t


def _out(out, like, dev):
    if out is None:
        return like.new_empty(like.shape)
    return _need(out, dev, like.dtype, like.shape, "out")


_SAME = contextlib.nullcontext()


def _stream(stream, dev):
    """(context in which torch allocates for the stream, the stream's handle)."""
    if stream is None:
        return _SAME, _raw_stream(dev)
    return torch.cuda.stream(stream), stream.cuda_stream


def _workspace(fn, args, like, what):
    """(tensor, address, bytes): the tensor is freed to torch's allocator when the caller is done
    with it, which hands it out again on this stream only."""
    size = ctypes.c_size_t()
    _check(fn(*args, size), what)
    if size.value == 0:
        return None, None, 0
    w = torch.empty(size.value, dtype=torch.uint8, device=like.device)
    return w, w.data_ptr(), size.value


def _lead(x, offsets, what):
    packed = offsets is not None
    if x.dim() != (2 if packed else 3):
        raise ValueError(f"{what}: expected [tokens, channels] with offsets, "
                         "[sequences, tokens, channels] without")
    shape = x.shape
    return packed, offsets.numel() - 1 if packed else shape[0], shape[0] if packed else shape[1]


def _batch(offsets, dev, nseq, length, packed):
    """What the library is told of (sequences, tokens, offsets).  No sequences are one without
    tokens, which writes nothing (states of no sequences have no address) but zeros to gradients of
    parameters."""
    at = _offsets(offsets, dev)
    if nseq:
        return nseq, length, at
    if packed and length:
        raise ValueError("offsets: tokens that belong to no sequence")
    return 1, 0, 0


# ---- short causal convolution ---------------------------------------------------------------


def _conv_desc(x, weight, bias, silu, initial_state, offsets):
    """(packed fft_conv_desc, device, sequences, channels, width)."""
    code, dev = _first(x, "x")
    dtype, shape = x.dtype, x.shape
    d = shape[-1]
    packed, nseq, length = _lead(x, offsets, "x")
    if x.stride(-1) != 1 and d > 1:
        _tell(x, dev, dtype, shape, "x")
    if weight.dim() != 2:
        raise ValueError("weight: expected [channels, width]")
    w, ptype = weight.shape[1], weight.dtype
    if ptype is not dtype and ptype is not torch.float32:
        raise TypeError("weight: expected float32 or the type of x")
    count, length, at = _batch(offsets, dev, nseq, length, packed)
    desc = _CONV.pack(code, F32 if ptype is torch.float32 else code, w, 1 if silu else 0, count,
                      length, d, at,
                      _flat(weight, dev, ptype, (d, w), "weight"),
                      _flat(bias, dev, ptype, (d,), "bias"),
                      _flat(initial_state, dev, dtype, (nseq, w - 1, d), "initial_state"),
                      *_seq(x, packed))
    return desc, dev, nseq, d, w


def causal_conv(x, weight, bias=None, silu=False, initial_state=None, offsets=None,
                return_state=False, out=None, stream=None):
    """Short causal convolution of every channel (fft_conv_forward): weight [channels, width],
    bias [channels], both float32 or of x's type; initial_state [sequences, width-1, channels].
    out may not overlap x.  Returns out, or (out, final_state).  Not recorded for autograd: gradients
    come from causal_conv_backward."""
    desc, dev, nseq, d, w = _conv_desc(x, weight, bias, silu, initial_state, offsets)
    on, s = _stream(stream, dev)
    with on:
        out = _out(out, x, dev)
        state = x.new_empty((nseq, w - 1, d)) if return_state else None
        _check(_L.fft_conv_forward(desc, _SEQ.pack(*_seq(out, offsets is not None)), _ptr(state),
                                   s), "fft_conv_forward")
    return (out, state) if return_state else out


def causal_conv_backward(dout, x, weight, bias=None, silu=False, initial_state=None, offsets=None,
                         dfinal_state=None, stream=None):
    """Gradients of causal_conv from dout (and dfinal_state): ConvGrads."""
    desc, dev, nseq, d, w = _conv_desc(x, weight, bias, silu, initial_state, offsets)
    _need(dout, dev, x.dtype, x.shape, "dout")
    packed, shape = offsets is not None, (nseq, w - 1, d)
    dfin = _flat(dfinal_state, dev, x.dtype, shape, "dfinal_state")
    on, s = _stream(stream, dev)
    with on:
        dx = x.new_empty(x.shape)
        dw = x.new_empty(weight.shape, dtype=torch.float32)
        db = x.new_empty((d,), dtype=torch.float32) if bias is not None else None
        di = x.new_empty(shape) if initial_state is not None else None
        ws, wp, size = _workspace(_L.fft_conv_workspace, (desc,), x, "fft_conv_workspace")
        _check(_L.fft_conv_backward(desc, _SEQ.pack(*_seq(dout, packed)), dfin,
                                    _SEQ.pack(*_seq(dx, packed)), dw.data_ptr(), _ptr(db),
                                    _ptr(di), wp, size, s), "fft_conv_backward")
    return ConvGrads(dx, dw, db, di)


def causal_conv_step(state, x, weight, bias=None, silu=False, slots=None, slots_out=None, out=None,
                     stream=None):
    """One token for each sequence (fft_conv_step): x [sequences, channels], state the pool
    [pool, width-1, channels], updated in place; slots, slots_out int64 [sequences].  A slot outside
    the pool marks a padding row (output 0, no state written); a slot that one sequence writes may
    not be read or written by another.  out may be x itself."""
    code, dev = _first(x, "x")
    dtype, shape = x.dtype, x.shape
    if len(shape) != 2 or weight.dim() != 2:
        raise ValueError("x: expected [sequences, channels], weight: [channels, width]")
    nseq, d = shape
    w, ptype = weight.shape[1], weight.dtype
    if ptype is not dtype and ptype is not torch.float32:
        raise TypeError("weight: expected float32 or the type of x")
    desc = _CONV.pack(code, F32 if ptype is torch.float32 else code, w, 1 if silu else 0, nseq, 1, d,
                      0, _flat(weight, dev, ptype, (d, w), "weight"),
                      _flat(bias, dev, ptype, (d,), "bias"), 0, *_token(x, dev, dtype, shape, "x"))
    size = state.shape[0]
    pool = _flat(state, dev, dtype, (size, w - 1, d), "state")
    src = _flat(slots, dev, torch.int64, (nseq,), "slots")
    dst = _flat(slots_out, dev, torch.int64, (nseq,), "slots_out")
    if nseq == 0:
        return _out(out, x, dev)
    if out is None and stream is None:  # the usual call
        out = x.new_empty(shape)
        _check(_L.fft_conv_step(desc, _SEQ.pack(out.data_ptr(), d, 0), pool, size, src, dst,
                                _raw_stream(dev)), "fft_conv_step")
        return out
    on, s = _stream(stream, dev)
    with on:
        out = _out(out, x, dev)
        _check(_L.fft_conv_step(desc, _SEQ.pack(*_row(out)), pool, size, src, dst, s),
               "fft_conv_step")
    return out


# ---- selective scan -------------------------------------------------------------------------


def _scan_desc(u, delta, A, B, C, D, z, delta_bias, softplus, initial_state, offsets):
    """(packed fft_scan_desc, device, sequences, channels, states)."""
    code, dev = _first(u, "u")
    f32, dtype, shape = torch.float32, u.dtype, tuple(u.shape)
    d, lead = shape[-1], shape[:-1]
    packed, nseq, length = _lead(u, offsets, "u")
    if u.stride(-1) != 1 and d > 1:
        _tell(u, dev, dtype, shape, "u")
    _need(delta, dev, dtype, shape, "delta")
    B, C = _groups(B, dev, dtype, lead, "B"), _groups(C, dev, dtype, lead, "C")
    groups, n = B.shape[-2:]
    if C.shape != B.shape:
        raise ValueError("C: expected the shape of B")
    if z is not None:
        _need(z, dev, dtype, shape, "z")
    count, length, at = _batch(offsets, dev, nseq, length, packed)
    heads = (code, 1 if softplus else 0, count, length, d, groups, n, at,
             _flat(A, dev, f32, (d, n), "A"), _flat(D, dev, f32, (d,), "D"),
             _flat(delta_bias, dev, f32, (d,), "delta_bias"),
             _flat(initial_state, dev, f32, (nseq, d, n), "initial_state"))
    desc = _SCAN.pack(*heads, *_seq(u, packed), *_seq(delta, packed), *_seq(B, packed),
                      *_seq(C, packed), *_seq(z, packed))
    return desc, dev, nseq, d, n


def selective_scan(u, delta, A, B, C, D=None, z=None, delta_bias=None, softplus=False,
                   initial_state=None, offsets=None, return_state=False, out=None, stream=None):
    """Selective state-space scan (fft_scan_forward): u, delta, z [..., channels], A [channels, n],
    B, C [..., groups, n] or [..., n], D, delta_bias [channels]; states [sequences, channels, n].
    A, D, delta_bias and states are float32.  out may be u or z and overlaps no other input.
    Returns out, or (out, final_state).  Not recorded for autograd: gradients come from
    selective_scan_backward."""
    desc, dev, nseq, d, n = _scan_desc(u, delta, A, B, C, D, z, delta_bias, softplus,
                                       initial_state, offsets)
    on, s = _stream(stream, dev)
    with on:
        out = _out(out, u, dev)
        state = u.new_empty((nseq, d, n), dtype=torch.float32) if return_state else None
        ws, wp, size = _workspace(_L.fft_scan_workspace, (desc, 0), u, "fft_scan_workspace")
        _check(_L.fft_scan_forward(desc, _SEQ.pack(*_seq(out, offsets is not None)), _ptr(state),
                                   wp, size, s), "fft_scan_forward")
    return (out, state) if return_state else out


def selective_scan_backward(dout, u, delta, A, B, C, D=None, z=None, delta_bias=None,
                            softplus=False, initial_state=None, offsets=None, dfinal_state=None,
                            stream=None):
    """Gradients of selective_scan from dout (and dfinal_state): ScanGrads."""
    desc, dev, nseq, d, n = _scan_desc(u, delta, A, B, C, D, z, delta_bias, softplus,
                                       initial_state, offsets)
    f32 = torch.float32
    _need(dout, dev, u.dtype, u.shape, "dout")
    packed, shape = offsets is not None, (nseq, d, n)
    dfin = _flat(dfinal_state, dev, f32, shape, "dfinal_state")
    on, s = _stream(stream, dev)
    with on:
        du, dd = u.new_empty(u.shape), u.new_empty(u.shape)
        dz = u.new_empty(u.shape) if z is not None else None
        dB, dC = u.new_empty(B.shape), u.new_empty(C.shape)
        dA = u.new_empty((d, n), dtype=f32)
        dD = u.new_empty((d,), dtype=f32) if D is not None else None
        db = u.new_empty((d,), dtype=f32) if delta_bias is not None else None
        di = u.new_empty(shape, dtype=f32) if initial_state is not None else None
        grads = _GRADS.pack(*_seq(dout, packed), dfin, *_seq(du, packed), *_seq(dd, packed),
                            *_seq(dB, packed), *_seq(dC, packed), *_seq(dz, packed),
                            *[_ptr(t) or 0 for t in (dA, dD, db, di)])
        ws, wp, size = _workspace(_L.fft_scan_workspace, (desc, 1), u, "fft_scan_workspace")
        _check(_L.fft_scan_backward(desc, grads, wp, size, s), "fft_scan_backward")
    return ScanGrads(du, dd, dA, dB, dC, dD, dz, db, di)


def selective_scan_step(state, u, delta, A, B, C, D=None, z=None, delta_bias=None, softplus=False,
                        slots=None, slots_out=None, out=None, stream=None):
    """One token for each sequence (fft_scan_step): u, delta, z [sequences, channels], B, C
    [sequences, groups, n] or [sequences, n], state the pool [pool, channels, n] float32, updated
    in place; slots, slots_out int64 [sequences] as in causal_conv_step.  out may be u, delta or z
    itself."""
    code, dev = _first(u, "u")
    f32, dtype, shape, bshape = torch.float32, u.dtype, u.shape, B.shape
    if len(shape) != 2 or len(bshape) not in (2, 3) or bshape[0] != shape[0]:
        raise ValueError("u: expected [sequences, channels], B: [sequences, groups, n]")
    nseq, d = shape
    groups, n = (1, bshape[1]) if len(bshape) == 2 else bshape[1:]
    desc = _SCAN.pack(code, 1 if softplus else 0, nseq, 1, d, groups, n, 0,
                      _flat(A, dev, f32, (d, n), "A"), _flat(D, dev, f32, (d,), "D"),
                      _flat(delta_bias, dev, f32, (d,), "delta_bias"), 0,
                      *_token(u, dev, dtype, shape, "u"), *_token(delta, dev, dtype, shape, "delta"),
                      *_token(B, dev, dtype, bshape, "B"), *_token(C, dev, dtype, bshape, "C"),
                      *(_token(z, dev, dtype, shape, "z") if z is not None else _NONE))
    size = state.shape[0]
    pool = _flat(state, dev, f32, (size, d, n), "state")
    src = _flat(slots, dev, torch.int64, (nseq,), "slots")
    dst = _flat(slots_out, dev, torch.int64, (nseq,), "slots_out")
    if nseq == 0:
        return _out(out, u, dev)
    if out is None and stream is None:  # the usual call
        out = u.new_empty(shape)
        _check(_L.fft_scan_step(desc, _SEQ.pack(out.data_ptr(), d, 0), pool, size, src, dst,
                                _raw_stream(dev)), "fft_scan_step")
        return out
    on, s = _stream(stream, dev)
    with on:
        out = _out(out, u, dev)
        _check(_L.fft_scan_step(desc, _SEQ.pack(*_row(out)), pool, size, src, dst, s),
               "fft_scan_step")
    return out


# ---- residual norm --------------------------------------------------------------------------


def _rows(t):
    """[..., columns] as rows of one stride: (rows, stride); the last axis is contiguous."""
    shape, st = t.shape, t.stride()
    if st[-1] != 1 and shape[-1] > 1:
        raise ValueError("expected rows whose last axis is contiguous")
    if len(shape) == 2:
        return shape[0], st[0]
    if len(shape) < 2:
        return 1, shape[-1]
    if 0 in shape[:-1]:
        return 0, shape[-1]
    rows, stride = shape[-2], st[-2]
    for k in range(len(shape) - 3, -1, -1):
        if shape[k] != 1 and rows != 1 and st[k] != rows * stride:
            raise ValueError("expected rows at one stride")
        if rows == 1:
            stride = st[k]
        rows *= shape[k]
    return rows, stride


def _norm_desc(x, res_dtype, weight, eps, e4m3, group):
    """(packed fft_norm_desc, device, columns, row stride of x)."""
    code, dev = _first(x, "x")
    rows, stride = _rows(x)
    d, ptype = x.shape[-1], weight.dtype
    if ptype is not x.dtype and ptype is not torch.float32:
        raise TypeError("weight: expected float32 or the type of x")
    desc = _NORM.pack(code, _CODES.get(res_dtype, -1), F32 if ptype is torch.float32 else code,
                      E4M3 if e4m3 else code, rows, d, group, eps,
                      _flat(weight, dev, ptype, (d,), "weight"))
    return desc, dev, d, stride


def residual_norm(x, weight, residual=None, eps=1e-6, out_dtype=None, group=0, out=None,
                  inplace_residual=False, stream=None):
    """Root-mean-square norm of x + residual (fft_norm_forward), rows along the last axis: NormOut.
    residual is of x's type or float32, and so is the sum that is returned (written over it with
    inplace_residual).  out_dtype torch.float8_e4m3fn: out in 8 bits with scale
    [..., ceil(columns / group)], group 32, 64 or 128 columns, or 0 for one scale per row.  Not
    recorded for autograd: gradients come from residual_norm_backward."""
    if _L is None:
        _setup()
    dtype, shape = x.dtype, x.shape
    otype = dtype if out_dtype is None else out_dtype
    e4m3 = otype is not dtype
    if e4m3 and otype is not torch.float8_e4m3fn:
        raise TypeError("out_dtype: expected the type of x or torch.float8_e4m3fn")
    res_dtype = dtype if residual is None else residual.dtype
    desc, dev, d, xs = _norm_desc(x, res_dtype, weight, eps, e4m3, group)
    rp = rs = 0
    if residual is not None:
        if residual.shape != shape or residual.get_device() != dev:
            _tell(residual, dev, res_dtype, shape, "residual")
        rp, rs = residual.data_ptr(), _rows(residual)[1]
    on, s = _stream(stream, dev)
    with on:
        if out is None:
            out, os = x.new_empty(shape, dtype=otype), d
        else:
            os = _rows(_need(out, dev, otype, shape, "out"))[1]
        scale = total = sp = tp = None
        ts = d
        if e4m3:
            groups = -(-d // group) if group > 0 else 1
            scale = x.new_empty((*shape[:-1], groups), dtype=torch.float32)
            sp = scale.data_ptr()
        if residual is not None:
            if inplace_residual:
                total, tp, ts = residual, rp, rs
            else:
                total = x.new_empty(shape, dtype=res_dtype)
                tp = total.data_ptr()
        rc = _L.fft_norm_forward(desc, x.data_ptr(), xs, rp, rs, out.data_ptr(), os, sp, tp, ts, s)
    _check(rc, "fft_norm_forward")
    return NormOut(out, scale, total)


def residual_norm_backward(dout, r, weight, dresidual=None, eps=1e-6, stream=None):
    """Gradients of residual_norm at its sum r (NormOut.residual, or x without a residual) from
    dout and from dresidual, the gradient that reaches the sum by itself: NormGrads."""
    desc, dev, d, gs = _norm_desc(dout, r.dtype, weight, eps, False, 0)
    shape = dout.shape
    _need(r, dev, r.dtype, shape, "r")
    if dresidual is not None:
        _need(dresidual, dev, r.dtype, shape, "dresidual")
    on, s = _stream(stream, dev)
    with on:
        dr = dout.new_empty(shape, dtype=r.dtype)
        dx = dr if r.dtype is dout.dtype else dout.new_empty(shape)
        dw = dout.new_empty((d,), dtype=torch.float32)
        ws, wp, size = _workspace(_L.fft_norm_workspace, (desc,), dout, "fft_norm_workspace")
        _check(_L.fft_norm_backward(
            desc, dout.data_ptr(), gs, r.data_ptr(), _rows(r)[1], _ptr(dresidual),
            _rows(dresidual)[1] if dresidual is not None else 0, dr.data_ptr(), _rows(dr)[1],
            None if dx is dr else dx.data_ptr(), _rows(dx)[1], dw.data_ptr(), wp, size, s),
            "fft_norm_backward")
    return NormGrads(dx, dr, dw)
