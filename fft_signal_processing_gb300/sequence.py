"""Sequence operators: short causal convolution, selective state-space scan, linear attention with
decays, residual norm, group norm.

Filters along the tokens of a sequence whose coefficients change from token to token (so that no
transform plan describes them), and the norm between two such layers; see include/gbfft.h for the
definitions.  Like the rest of the binding this marshals torch tensors to device pointers and the
current CUDA stream: every step runs in the library's kernels.

    out, state = causal_conv(x, weight, bias, silu=True, return_state=True)    # x [b, l, d]
    y, h = selective_scan(u, delta, A, B, C, D=D, z=z, softplus=True, return_state=True)
    o, S = linear_attention(q, k, v, decay, return_state=True)      # q, k [b, l, groups, dk]
    r = group_norm(x, groups, weight, bias, z=z)                    # r.out, r.mean, r.rstd
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
_HEADS = struct.Struct("@P3q")  # fft_heads
_ATTN = struct.Struct("@if6q2P" + "P3q" * 3 + "P2q")  # fft_linattn_desc
_ATTN_GRADS = struct.Struct("@P3qP" + "P3q" * 3 + "P2qP")  # fft_linattn_grads
_GNORM = struct.Struct("@3if4q3P" + "P2q" * 2)  # fft_gnorm_desc
_GNORM_GRADS = struct.Struct("@2P" + "P2q" * 3 + "2P")  # fft_gnorm_grads
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


class AttentionGrads(NamedTuple):
    dq: object
    dk: object
    dv: object
    ddecay: object
    dinitial_state: Optional[object]


class GroupNormOut(NamedTuple):
    out: object
    mean: object  # float32 [sequences, groups]
    rstd: object


class GroupNormGrads(NamedTuple):
    dx: object
    dz: Optional[object]
    dweight: Optional[object]  # float32 [channels]
    dbias: Optional[object]


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
    L.fft_linattn_workspace.argtypes = [desc, ctypes.c_int, ctypes.POINTER(sz)]
    L.fft_linattn_forward.argtypes = [desc, desc, vp, vp, sz, vp]
    L.fft_linattn_backward.argtypes = [desc, desc, vp, sz, vp]
    L.fft_linattn_check.argtypes = [vp]
    L.fft_linattn_set_wait_timeout.argtypes = [ctypes.c_uint64]
    L.fft_linattn_step.argtypes = [desc, desc, vp, i64, vp, vp, vp]
    L.fft_norm_forward.argtypes = [desc, vp, i64, vp, i64, vp, i64, vp, vp, i64, vp]
    L.fft_norm_workspace.argtypes = [desc, ctypes.POINTER(sz)]
    L.fft_norm_backward.argtypes = [desc, vp, i64, vp, i64, vp, i64, vp, i64, vp, i64, vp, vp, sz,
                                    vp]
    L.fft_gnorm_workspace.argtypes = [desc, ctypes.c_int, ctypes.POINTER(sz)]
    L.fft_gnorm_forward.argtypes = [desc, desc, vp, vp, vp, sz, vp]
    L.fft_gnorm_backward.argtypes = [desc, desc, vp, sz, vp]


SYMBOLS = ("fft_conv_forward", "fft_conv_workspace", "fft_conv_backward", "fft_conv_step",
           "fft_scan_workspace", "fft_scan_forward", "fft_scan_backward", "fft_scan_step",
           "fft_linattn_workspace", "fft_linattn_forward", "fft_linattn_backward",
           "fft_linattn_step", "fft_linattn_check", "fft_linattn_set_wait_timeout", "fft_norm_forward",
           "fft_norm_workspace", "fft_norm_backward",
           "fft_gnorm_workspace", "fft_gnorm_forward", "fft_gnorm_backward")


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


# ---- linear attention -----------------------------------------------------------------------


def _heads(t, packed):
    """The fields of an fft_heads."""
    st = t.stride()
    return (t.data_ptr(), 0, st[0], st[1]) if packed else (t.data_ptr(), st[0], st[1], st[2])


def _scale(scale, dk):
    """dk ** -0.5 unless given; rows without values are the library's to refuse."""
    return (dk or 1) ** -0.5 if scale is None else scale


def _attn_desc(q, k, v, decay, scale, initial_state, offsets):
    """(packed fft_linattn_desc, device, sequences, heads, dk, dv)."""
    code, dev = _first(q, "q")
    dtype, packed = q.dtype, offsets is not None
    if q.dim() != (3 if packed else 4) or v.dim() != q.dim():
        raise ValueError("q: expected [tokens, groups, dk] with offsets, [sequences, tokens, groups, dk] "
                         "without, and v [..., heads, dv]")
    lead, (groups, dk), (heads, dv) = q.shape[:-2], q.shape[-2:], v.shape[-2:]
    _need(q, dev, dtype, q.shape, "q")
    _need(k, dev, dtype, q.shape, "k")
    _need(v, dev, dtype, (*lead, heads, dv), "v")
    if decay.dtype is not dtype or decay.shape != (*lead, heads) or decay.get_device() != dev or (
            decay.stride(-1) != 1 and heads > 1 and decay.numel()):
        _tell(decay, dev, dtype, (*lead, heads), "decay")
    nseq, length = (offsets.numel() - 1, lead[0]) if packed else lead
    count, length, at = _batch(offsets, dev, nseq, length, packed)
    st = decay.stride()
    desc = _ATTN.pack(code, _scale(scale, dk), count, length, heads, groups, dk, dv,
                      at, _flat(initial_state, dev, torch.float32, (nseq, heads, dk, dv), "initial_state"),
                      *_heads(q, packed), *_heads(k, packed), *_heads(v, packed),
                      *((decay.data_ptr(), 0, st[0]) if packed else (decay.data_ptr(), st[0], st[1])))
    return desc, dev, nseq, heads, dk, dv


def linear_attention(q, k, v, decay, scale=None, initial_state=None, offsets=None, return_state=False,
                     out=None, stream=None):
    """Linear attention with a decay for each head (fft_linattn_forward): q, k [..., groups, dk],
    v [..., heads, dv], decay [..., heads] (logs, at most 0; of q's dtype; strides of 0 for decays that do
    not change), scale dk ** -0.5 unless given; states [sequences, heads, dk, dv] float32.  Any strides but
    of the last axis, so heads may lie beside tokens or around them.  out overlaps no input.  Returns out,
    or (out, final_state).  Not recorded for autograd: gradients come from linear_attention_backward."""
    desc, dev, nseq, heads, dk, dv = _attn_desc(q, k, v, decay, scale, initial_state, offsets)
    on, s = _stream(stream, dev)
    with on:
        out = v.new_empty(v.shape) if out is None else _need(out, dev, v.dtype, v.shape, "out")
        state = v.new_empty((nseq, heads, dk, dv), dtype=torch.float32) if return_state else None
        ws, wp, size = _workspace(_L.fft_linattn_workspace, (desc, 0), v, "fft_linattn_workspace")
        _check(_L.fft_linattn_forward(desc, _HEADS.pack(*_heads(out, offsets is not None)), _ptr(state),
                                      wp, size, s), "fft_linattn_forward")
    return (out, state) if return_state else out


def linear_attention_backward(dout, q, k, v, decay, scale=None, initial_state=None, offsets=None,
                              dfinal_state=None, stream=None):
    """Gradients of linear_attention from dout (and dfinal_state): AttentionGrads.  Those of queries and
    keys are sums over the heads that share them; ddecay has decay's shape, also where decay is a view
    whose strides are 0.  A value that is not finite may reach all of its sequence's and heads' gradients."""
    desc, dev, nseq, heads, dk, dv = _attn_desc(q, k, v, decay, scale, initial_state, offsets)
    _need(dout, dev, v.dtype, v.shape, "dout")
    packed, shape = offsets is not None, (nseq, heads, dk, dv)
    dfin = _flat(dfinal_state, dev, torch.float32, shape, "dfinal_state")
    on, s = _stream(stream, dev)
    with on:
        dq, dkey, dval = q.new_empty(q.shape), q.new_empty(q.shape), v.new_empty(v.shape)
        dg = v.new_empty(decay.shape)
        di = v.new_empty(shape, dtype=torch.float32) if initial_state is not None else None
        grads = _ATTN_GRADS.pack(*_heads(dout, packed), dfin, *_heads(dq, packed), *_heads(dkey, packed),
                                 *_heads(dval, packed), *_seq(dg, packed), _ptr(di) or 0)
        ws, wp, size = _workspace(_L.fft_linattn_workspace, (desc, 1), v, "fft_linattn_workspace")
        _check(_L.fft_linattn_backward(desc, grads, wp, size, s), "fft_linattn_backward")
    return AttentionGrads(dq, dkey, dval, dg, di)


def linear_attention_check(stream=None):
    """Synchronises the stream and raises GbfftError where a device-side wait of an earlier call of
    linear_attention or its gradients on the current device has run out (fft_linattn_check)."""
    if _L is None:
        _setup()
    _check(_L.fft_linattn_check(_stream(stream, _device())[1]), "fft_linattn_check")


def linear_attention_set_wait_timeout(ns=2 * 10 ** 9):
    """Time limit of the device-side waits of the calls that follow (fft_linattn_set_wait_timeout); 0: each
    gives up at once (a diagnostic hook)."""
    if _L is None:
        _setup()
    _check(_L.fft_linattn_set_wait_timeout(int(ns)), "fft_linattn_set_wait_timeout")


def linear_attention_step(state, q, k, v, decay, scale=None, slots=None, slots_out=None, out=None,
                          stream=None):
    """One token for each sequence (fft_linattn_step): q, k [sequences, groups, dk], v [sequences, heads,
    dv], decay [sequences, heads], state the pool [pool, heads, dk, dv] float32, updated in place; slots,
    slots_out int64 [sequences] as in causal_conv_step.  out overlaps no input."""
    code, dev = _first(q, "q")
    dtype, qs, vs = q.dtype, q.shape, v.shape
    if len(qs) != 3 or len(vs) != 3:
        raise ValueError("q: expected [sequences, groups, dk], v: [sequences, heads, dv]")
    nseq, groups, dk = qs
    heads, dv = vs[1:]
    _need(q, dev, dtype, qs, "q")
    _need(k, dev, dtype, qs, "k")
    _need(v, dev, dtype, (nseq, heads, dv), "v")
    qt, kt, vt = q.stride(), k.stride(), v.stride()
    desc = _ATTN.pack(code, _scale(scale, dk), nseq, 1, heads, groups, dk, dv, 0, 0,
                      q.data_ptr(), qt[0], 0, qt[1], k.data_ptr(), kt[0], 0, kt[1],
                      v.data_ptr(), vt[0], 0, vt[1], *_token(decay, dev, dtype, (nseq, heads), "decay"))
    size = state.shape[0]
    pool = _flat(state, dev, torch.float32, (size, heads, dk, dv), "state")
    src = _flat(slots, dev, torch.int64, (nseq,), "slots")
    dst = _flat(slots_out, dev, torch.int64, (nseq,), "slots_out")
    on, s = _stream(stream, dev)
    with on:
        out = v.new_empty(vs) if out is None else _need(out, dev, dtype, vs, "out")
        if nseq == 0:
            return out
        ot = out.stride()
        _check(_L.fft_linattn_step(desc, _HEADS.pack(out.data_ptr(), ot[0], 0, ot[1]), pool, size, src, dst, s),
               "fft_linattn_step")
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


# ---- group norm -----------------------------------------------------------------------------


def _gnorm_rows(t):
    """The fields of an fft_seq of [rows, channels] (sequences of one token), [sequences, tokens,
    channels] or, packed, [tokens, channels]."""
    st = t.stride()
    return (t.data_ptr(), st[0], st[1] if len(st) == 3 else 0)


def _gnorm_desc(x, groups, weight, bias, z, silu, eps, offsets):
    """(packed fft_gnorm_desc, device, sequences)."""
    code, dev = _first(x, "x")
    dtype, shape, packed = x.dtype, x.shape, offsets is not None
    if len(shape) != 2 and (packed or len(shape) != 3):
        raise ValueError("x: expected [tokens, channels] with offsets, [sequences, tokens, channels] or [rows, "
                         "channels] without")
    _need(x, dev, dtype, shape, "x")
    d = shape[-1]
    nseq = offsets.numel() - 1 if packed else shape[0]
    length = shape[0] if packed else (shape[1] if len(shape) == 3 else 1)
    ptype = torch.float32
    for t, what in ((weight, "weight"), (bias, "bias")):
        if t is not None:
            if t.dtype is not dtype and t.dtype is not torch.float32:
                raise TypeError(f"{what}: expected float32 or the type of x")
            ptype = t.dtype
    if z is not None:
        _need(z, dev, dtype, shape, "z")
    count, length, at = _batch(offsets, dev, nseq, length, packed)
    rows = _seq if packed else (lambda t, _: _gnorm_rows(t))
    desc = _GNORM.pack(code, F32 if ptype is torch.float32 else code, 1 if silu else 0, eps, count, length, d,
                       groups, at, _flat(weight, dev, ptype, (d,), "weight"),
                       _flat(bias, dev, ptype, (d,), "bias"), *rows(x, packed),
                       *(rows(z, packed) if z is not None else _NONE))
    return desc, dev, nseq, rows


def group_norm(x, groups, weight=None, bias=None, z=None, silu=False, eps=1e-5, offsets=None, out=None,
               stream=None):
    """Group norm, channels last (fft_gnorm_forward): x [sequences, tokens, channels], packed [tokens,
    channels] with offsets, or [rows, channels], each row by itself; weight, bias [channels], both
    float32 or of x's type; silu applies SiLU, z [like x] gates what comes out.  out may be x or z itself.
    Returns GroupNormOut: out, and mean and rstd [sequences, groups] for group_norm_backward.  Not
    recorded for autograd."""
    desc, dev, nseq, rows = _gnorm_desc(x, groups, weight, bias, z, silu, eps, offsets)
    on, s = _stream(stream, dev)
    with on:
        out = _out(out, x, dev)
        stats = x.new_empty((2, nseq, groups), dtype=torch.float32)
        mean, rstd = stats[0], stats[1]
        if nseq == 0:
            return GroupNormOut(out, mean, rstd)
        ws, wp, size = _workspace(_L.fft_gnorm_workspace, (desc, 0), x, "fft_gnorm_workspace")
        _check(_L.fft_gnorm_forward(desc, _SEQ.pack(*rows(out, offsets is not None)), mean.data_ptr(),
                                    rstd.data_ptr(), wp, size, s), "fft_gnorm_forward")
    return GroupNormOut(out, mean, rstd)


def group_norm_backward(dout, x, mean, rstd, weight=None, bias=None, z=None, silu=False, offsets=None,
                        stream=None):
    """Gradients of group_norm from dout and the forward call's mean and rstd: GroupNormGrads."""
    groups = mean.shape[-1]
    desc, dev, nseq, rows = _gnorm_desc(x, groups, weight, bias, z, silu, 0.0, offsets)
    _need(dout, dev, x.dtype, x.shape, "dout")
    packed, f32 = offsets is not None, torch.float32
    mp, rp = _flat(mean, dev, f32, (nseq, groups), "mean"), _flat(rstd, dev, f32, (nseq, groups), "rstd")
    on, s = _stream(stream, dev)
    with on:
        dx = x.new_empty(x.shape)
        dz = x.new_empty(x.shape) if z is not None else None
        # one behind the other, which takes one kernel less
        params = (x.new_empty if nseq else x.new_zeros)((2, x.shape[-1]), dtype=f32)
        dw = params[0] if weight is not None else None
        db = params[1] if bias is not None else None
        if nseq == 0:
            return GroupNormGrads(dx, dz, dw, db)
        grads = _GNORM_GRADS.pack(mp, rp, *rows(dout, packed), *rows(dx, packed),
                                  *(rows(dz, packed) if z is not None else _NONE), _ptr(dw) or 0, _ptr(db) or 0)
        ws, wp, size = _workspace(_L.fft_gnorm_workspace, (desc, 1), x, "fft_gnorm_workspace")
        _check(_L.fft_gnorm_backward(desc, grads, wp, size, s), "fft_gnorm_backward")
    return GroupNormGrads(dx, dz, dw, db)
