"""The operators at a block's edges and beside the recurrences on torch tensors
(include/tfla.h): rotary positions of queries and keys, the gated linear
recurrence of channels, and the residual sum with a layer or RMS norm;
:mod:`mlstm_sequence_amd.tfla` offers the same names.

Argument checks, output allocation and marshalling only, in the manner of
:mod:`mlstm_sequence_amd.blocks`: the work runs in the library's HIP kernels on
torch's current stream of the tensors' device, or with ``stream`` as under
``torch.cuda.stream(stream)``.  Channels are contiguous, other strides are
free; a tensor that does not fit is refused, never copied.
"""
from __future__ import annotations

import ctypes
import math
import struct
from typing import NamedTuple, Optional

import torch

from . import blocks as _blocks
from .blocks import _HEADS, _IO, _NO_HEADS, _NO_ROWS, _ROWS, Heads, Rows, _bad, _call, _current, _i, _ll, _p

ROTARY_HALVES, ROTARY_INTERLEAVED = 0, 0x4000   # pairs: channels j and j + R/2, or 2j and 2j + 1
DIAG_COUPLED, DIAG_SIGMOID, DIAG_DECAY = 0, 1, 2
DIAG_CHUNK = 128   # rows between the states that diag_forward leaves for diag_backward
_RMS, _SUM_FP32 = 0x8000, 0x10000

_fn = {}   # this module's entry points, once the library is loaded


def bind(L):
    """Argument types of this module's entry points, offered all at once."""
    global _fn
    vp, sz = ctypes.c_void_p, ctypes.c_size_t
    fn = {}
    for name, args, res in (
            ("tfla_rotary_fwd", [vp, vp], _i),
            ("tfla_rotary_bwd", [vp, vp], _i),
            ("tfla_diag_workspace_bytes", [_i] * 5, sz),
            ("tfla_diag_fwd", [vp, vp, sz, vp], _i),
            ("tfla_diag_bwd_workspace_bytes", [_i] * 5, sz),
            ("tfla_diag_bwd", [vp, vp, sz, vp], _i),
            ("tfla_addnorm_fwd", [vp, vp], _i),
            ("tfla_addnorm_bwd_workspace_bytes", [_i] * 4, sz),
            ("tfla_addnorm_bwd", [vp, vp, sz, vp], _i)):
        f = getattr(L, name)
        f.argtypes, f.restype = args, res
        fn[name] = f
    _fn = fn


def _entry(name):
    if not _fn:
        from . import tfla
        tfla.lib()
    return _fn[name]


class RotaryArgs(ctypes.Structure):
    """tfla_rotary_args."""
    _fields_ = [("B", _i), ("T", _i), ("H", _i), ("Hk", _i), ("C", _i), ("R", _i), ("flags", _i), ("scale", ctypes.c_float),
                ("freqs", _p), ("positions", _p), ("positions_batch", _ll), ("start", _p), ("lengths", _p),
                ("q", Heads), ("k", Heads), ("q_out", Heads), ("k_out", Heads)]


class DiagArgs(ctypes.Structure):
    """tfla_diag_args."""
    _fields_ = [("B", _i), ("T", _i), ("D", _i), ("kind", _i), ("flags", _i),
                ("x", Rows), ("fgate", Rows), ("igate", Rows), ("decay", _p), ("lengths", _p),
                ("state", _p), ("y", Rows), ("state_out", _p), ("starts", _p),
                ("dy", Rows), ("dstate_out", _p), ("dx", Rows), ("dfgate", Rows), ("digate", Rows), ("ddecay", _p),
                ("dstate", _p)]


class AddNormArgs(ctypes.Structure):
    """tfla_addnorm_args."""
    _fields_ = [("B", _i), ("T", _i), ("C", _i), ("flags", _i), ("eps", ctypes.c_float),
                ("x", Rows), ("residual", Rows), ("weight", _p), ("bias", _p), ("y", Rows), ("total", Rows),
                ("dy", Rows), ("dtotal", Rows), ("dx", Rows), ("dresidual", Rows), ("dweight", _p), ("dbias", _p)]


_ROTARY = struct.Struct("@7if2Pq2P" + _HEADS * 4)
_DIAG = struct.Struct("@5i" + _ROWS * 3 + "3P" + _ROWS + "2P" + _ROWS + "P" + _ROWS * 3 + "2P")
_ADDNORM = struct.Struct("@4if" + _ROWS * 2 + "2P" + _ROWS * 6 + "2P")


# ---- checks --------------------------------------------------------------------------
#
# As in blocks.py, each in one step: a call of single tokens spends most of its
# time here.

def _first(x, name, dims):
    """Checks the tensor that sets type and device; returns the device's index."""
    if isinstance(x, torch.Tensor) and x.dtype in _IO and x.dim() == dims and x.is_cuda and 0 < x.numel() <= 0x7FFFFFFF:
        return x.get_device()
    return _blocks._first(x, name, dims)   # says what does not fit, or that a large tensor does


def _new(x):
    """A contiguous tensor of the shape and type of ``x``."""
    return torch.empty_like(x) if x.is_contiguous() else torch.empty_like(x, memory_format=torch.contiguous_format)


def _out(t, name, like, dtype, dev):
    """An output [B,T,D], new where ``t`` is None, and its tfla_rows."""
    if t is not None:
        return t, _rows(t, name, like.shape, dtype, dev)
    t = _new(like)
    _, T, D = like.shape
    return t, (t.data_ptr(), T * D, D)


def _flat(t, name, shape, dtype, dev):
    """Pointer of a contiguous tensor (None: NULL)."""
    if t is None:
        return 0
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous():
        return t.data_ptr()
    _bad(t, name, shape, dtype, dev)


def _rows(t, name, shape, dtype, dev):
    """tfla_rows of a [B,T,D] tensor with contiguous channels."""
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.get_device() == dev:
        batch, row, one = t.stride()
        if one == 1 or shape[2] <= 1:
            return t.data_ptr(), batch, row
    _bad(t, name, shape, dtype, dev)


def _heads(t, name, shape, dtype, dev):
    """tfla_heads of a [B,T,G,C] tensor with contiguous channels."""
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.get_device() == dev:
        batch, row, group, one = t.stride()
        if one == 1 or shape[3] <= 1:
            return t.data_ptr(), batch, row, group
    _bad(t, name, shape, dtype, dev)


# ---- rotary positions ------------------------------------------------------------

def rotary_frequencies(dim: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
                       original_length: Optional[int] = None, slow: float = 1.0, fast: float = 32.0, device="cuda"):
    """Frequencies of ``dim`` rotated channels, fp64 [dim/2] on ``device``, and
    the factor of the rotated values: what :func:`rotary_forward` takes as
    ``freqs`` and ``scale``.

    ``base ** (-2 j / dim)``, for contexts ``factor`` times the trained length:
    "linear" divides all by the factor; "ntk" stretches the base to
    ``base factor ** (dim / (dim - 2))``, so the fastest stay and the slowest
    are divided by the factor; "yarn" divides those with fewer than ``slow``
    turns in ``original_length`` rows, keeps those with more than ``fast``,
    goes over linearly between, and scales by ``0.1 ln(factor) + 1``."""
    if dim < 0 or dim % 2:
        raise ValueError(f"dim must be even and not negative, got {dim}")
    if not (base > 0 and math.isfinite(base)):
        raise ValueError(f"base must be positive and finite, got {base}")
    if not (factor >= 1 and math.isfinite(factor)):
        raise ValueError(f"factor must be finite and at least 1, got {factor}")
    exponent = -2.0 * torch.arange(dim // 2, dtype=torch.float64) / max(dim, 1)
    scale = 1.0
    if scaling == "ntk" and dim > 2:
        base = base * factor ** (dim / (dim - 2))
    freqs = torch.pow(torch.tensor(float(base), dtype=torch.float64), exponent)
    if scaling == "linear":
        freqs = freqs / factor
    elif scaling == "yarn":
        if original_length is None or original_length < 1:
            raise ValueError("yarn needs original_length, the trained length in rows")
        if not fast > slow:
            raise ValueError(f"fast must be above slow, got {fast} and {slow}")
        keep = ((original_length * freqs / (2 * math.pi) - slow) / (fast - slow)).clamp(0.0, 1.0)
        freqs = (1.0 - keep) * freqs / factor + keep * freqs
        scale = 0.1 * math.log(factor) + 1.0
    elif scaling not in ("none", "ntk"):
        raise ValueError(f'scaling must be "none", "linear", "ntk" or "yarn", got {scaling!r}')
    return freqs.to(device), scale


def _rotary(name, q, k, freqs, layout, scale, positions, start, lengths, q_out, k_out, head_major, stream):
    if stream is not None:
        with _current(stream, q):
            return _rotary(name, q, k, freqs, layout, scale, positions, start, lengths, q_out, k_out, head_major, None)
    fn = _fn.get(name) or _entry(name)
    dev = _first(q, "q", 4)
    shape, dtype = q.shape, q.dtype
    B, T, H, C = shape
    if layout not in (ROTARY_HALVES, ROTARY_INTERLEAVED):
        raise ValueError(f"layout must be ROTARY_HALVES or ROTARY_INTERLEAVED, got {layout}")
    if not isinstance(freqs, torch.Tensor) or freqs.dim() != 1:
        raise ValueError("freqs must be a one-dimensional fp64 tensor")
    half = freqs.shape

    def out(t, name, like, n):   # a new tensor's strides are known
        if t is not None:
            return t, _heads(t, name, (B, T, n, C), dtype, dev)
        if head_major:
            t = like.new_empty((B, n, T, C)).transpose(1, 2)
            return t, (t.data_ptr(), n * T * C, C, T * C)
        t = _new(like)
        return t, (t.data_ptr(), T * n * C, n * C, C)

    q_out, queries_out = out(q_out, "q_out", q, H)
    Hk, keys, keys_out = 0, _NO_HEADS, _NO_HEADS
    if k is not None:
        if not isinstance(k, torch.Tensor) or k.dim() != 4:
            raise ValueError("k must be a [B,T,Hk,C] tensor")
        Hk = k.shape[2]
        kshape = (B, T, Hk, C)
        keys = _heads(k, "k", kshape, dtype, dev)
        k_out, keys_out = out(k_out, "k_out", k, Hk)
    elif k_out is not None:
        raise ValueError("k_out is given without k")
    at = stride = 0
    if positions is not None:
        shared = isinstance(positions, torch.Tensor) and positions.dim() == 1
        want = (T,) if shared else (B, T)
        if not isinstance(positions, torch.Tensor) or positions.dtype is not torch.int32 or positions.shape != want \
                or positions.get_device() != dev or (T > 1 and positions.stride(-1) != 1):
            _bad(positions, "positions", want, torch.int32, dev)
        at, stride = positions.data_ptr(), 0 if shared else positions.stride(0)
    packed = _ROTARY.pack(B, T, H, Hk, C, 2 * half[0], _IO[dtype] | layout, scale,
                          _flat(freqs, "freqs", half, torch.float64, dev), at, stride,
                          _flat(start, "start", (B,), torch.int32, dev), _flat(lengths, "lengths", (B,), torch.int32, dev),
                          *_heads(q, "q", shape, dtype, dev), *keys, *queries_out, *keys_out)
    _call(name, packed, dev, None, None, fn)
    return q_out, k_out


def rotary_forward(q, k, freqs, layout: int = ROTARY_HALVES, scale: float = 1.0, positions=None, start=None, lengths=None,
                   q_out=None, k_out=None, head_major: bool = False, stream=None):
    """Rotary positions of q [B,T,H,C] and k [B,T,Hk,C] (or None): the first
    2 len(freqs) channels of each head turn by ``position * freqs``, times
    ``scale``; the others pass.  Returns ``(q_out, k_out)``.

    ``freqs`` fp64 [R/2] (:func:`rotary_frequencies`); positions are
    ``positions`` int32 [B,T] or [T], else ``start`` int32 [B] plus the row,
    else the row.  ``head_major`` allocates outputs whose memory is [B,H,T,C],
    so that ``q_out.transpose(1, 2)`` is what :func:`forward` takes; ``q_out``
    may be q itself.  ``lengths`` int32 [B]: valid rows of a padded batch."""
    return _rotary("tfla_rotary_fwd", q, k, freqs, layout, scale, positions, start, lengths, q_out, k_out, head_major, stream)


def rotary_backward(dq, dk, freqs, layout: int = ROTARY_HALVES, scale: float = 1.0, positions=None, start=None,
                    lengths=None, q_out=None, k_out=None, head_major: bool = False, stream=None):
    """Gradients of :func:`rotary_forward`'s q and k from those of its outputs
    (dk None: of q alone), the other arguments being the forward pass's;
    ``q_out`` and ``k_out`` receive them where given."""
    return _rotary("tfla_rotary_bwd", dq, dk, freqs, layout, scale, positions, start, lengths, q_out, k_out, head_major, stream)


# ---- gated linear recurrence of channels --------------------------------------------

class DiagGrads(NamedTuple):
    """Gradients of :func:`diag_forward`; None where the input was None."""
    dx: torch.Tensor
    dfgate: torch.Tensor
    digate: Optional[torch.Tensor]
    ddecay: Optional[torch.Tensor]
    dstate: Optional[torch.Tensor]


def _diag_args(x, fgate, igate, decay, kind, lengths):
    """(fields shared by both directions, sizes of the workspace calls, device)"""
    dev = _first(x, "x", 3)
    shape, dtype = x.shape, x.dtype
    B, T, D = shape
    if kind not in (DIAG_COUPLED, DIAG_SIGMOID, DIAG_DECAY):
        raise ValueError(f"kind must be DIAG_COUPLED, DIAG_SIGMOID or DIAG_DECAY, got {kind}")
    if (igate is None) != (kind == DIAG_COUPLED):
        raise ValueError("igate must be given exactly for DIAG_SIGMOID and DIAG_DECAY")
    if (decay is None) != (kind != DIAG_DECAY):
        raise ValueError("decay must be given exactly for DIAG_DECAY")
    sizes = (B, T, D, kind, _IO[dtype])
    return (*sizes, *_rows(x, "x", shape, dtype, dev), *_rows(fgate, "fgate", shape, dtype, dev),
            *(_NO_ROWS if igate is None else _rows(igate, "igate", shape, dtype, dev)),
            _flat(decay, "decay", (D,), torch.float32, dev), _flat(lengths, "lengths", (B,), torch.int32, dev)), sizes, dev


def _chunks(shape):
    B, T, D = shape
    return B, -(-T // DIAG_CHUNK), D


def diag_forward(x, fgate, igate=None, decay=None, kind: int = DIAG_COUPLED, state=None, lengths=None,
                 want_state: bool = False, want_starts: bool = False, y=None, state_out=None, starts=None, workspace=None,
                 stream=None):
    """Gated linear recurrence ``y = h = f h + i x`` of x [B,T,D], a state a
    channel; returns ``(y, state_out, starts)``.

    Gates from pre-activations [B,T,D]: DIAG_COUPLED ``f = sigmoid(fgate)``,
    ``i = 1 - f``; DIAG_SIGMOID the same f and ``i = sigmoid(igate)``;
    DIAG_DECAY ``f = exp(-decay sigmoid(fgate))``,
    ``i = sqrt(1 - f^2) sigmoid(igate)`` with decay fp32 [D], not negative.
    ``state`` fp32 [B,D] is the state before the first row; ``state_out``
    (allocated with ``want_state``, may be ``state`` itself) the one after the
    last; ``starts`` (allocated with ``want_starts``) fp32
    [B, ceil(T / DIAG_CHUNK), D] the states that :func:`diag_backward` needs.
    ``lengths`` int32 [B]: valid rows of a padded batch."""
    if stream is not None:
        with _current(stream, x):
            return diag_forward(x, fgate, igate, decay, kind, state, lengths, want_state, want_starts, y, state_out, starts,
                                workspace)
    need = _fn.get("tfla_diag_workspace_bytes") or _entry("tfla_diag_workspace_bytes")
    fields, sizes, dev = _diag_args(x, fgate, igate, decay, kind, lengths)
    shape, dtype, f32 = x.shape, x.dtype, torch.float32
    bd = (shape[0], shape[2])
    y, yr = _out(y, "y", x, dtype, dev)
    if state_out is None and want_state:
        state_out = x.new_empty(bd, dtype=f32)
    if starts is None and want_starts:
        starts = x.new_empty(_chunks(shape), dtype=f32)
    packed = _DIAG.pack(*fields, _flat(state, "state", bd, f32, dev), *yr,
                        _flat(state_out, "state_out", bd, f32, dev),
                        0 if starts is None else _flat(starts, "starts", _chunks(shape), f32, dev),
                        *_NO_ROWS, 0, *_NO_ROWS * 3, 0, 0)
    _call("tfla_diag_fwd", packed, dev, need(*sizes), workspace, _fn["tfla_diag_fwd"])
    return y, state_out, starts


def diag_backward(x, fgate, dy, starts, igate=None, decay=None, kind: int = DIAG_COUPLED, lengths=None, dstate_out=None,
                  want_dstate: bool = False, dx=None, dfgate=None, digate=None, workspace=None, stream=None) -> DiagGrads:
    """Gradients of :func:`diag_forward` for ``dy`` and (with carried states)
    ``dstate_out``, from the ``starts`` it left; dx, dfgate and digate may be
    given, as parts of a projection's gradient for instance.  The gradient of
    the state before the first row comes with ``want_dstate``."""
    if stream is not None:
        with _current(stream, x):
            return diag_backward(x, fgate, dy, starts, igate, decay, kind, lengths, dstate_out, want_dstate, dx, dfgate,
                                 digate, workspace)
    need = _fn.get("tfla_diag_bwd_workspace_bytes") or _entry("tfla_diag_bwd_workspace_bytes")
    fields, sizes, dev = _diag_args(x, fgate, igate, decay, kind, lengths)
    shape, dtype, f32 = x.shape, x.dtype, torch.float32
    bd = (shape[0], shape[2])
    if starts is None:
        raise ValueError("starts is needed: the states that diag_forward leaves with want_starts")
    dx, dxr = _out(dx, "dx", x, dtype, dev)
    dfgate, dur = _out(dfgate, "dfgate", x, dtype, dev)
    dvr = _NO_ROWS
    if igate is not None:
        digate, dvr = _out(digate, "digate", x, dtype, dev)
    elif digate is not None:
        raise ValueError("digate is given without igate")
    ddecay = None if decay is None else torch.empty_like(decay)
    dstate = x.new_empty(bd, dtype=f32) if want_dstate else None
    packed = _DIAG.pack(*fields, 0, *_NO_ROWS, 0, _flat(starts, "starts", _chunks(shape), f32, dev),
                        *_rows(dy, "dy", shape, dtype, dev), _flat(dstate_out, "dstate_out", bd, f32, dev),
                        *dxr, *dur, *dvr,
                        0 if ddecay is None else ddecay.data_ptr(), 0 if dstate is None else dstate.data_ptr())
    _call("tfla_diag_bwd", packed, dev, need(*sizes), workspace, _fn["tfla_diag_bwd"])
    return DiagGrads(dx, dfgate, digate, ddecay, dstate)


# ---- residual sum with a norm ---------------------------------------------------------

def _stream_type(t, name, dtype):
    """Type of a tensor of the residual stream: the activations' or fp32."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor, got {type(t).__name__}")
    if t.dtype not in (dtype, torch.float32):
        raise TypeError(f"{name} must be {dtype} or torch.float32, got {t.dtype}")
    return t.dtype


def addnorm_forward(x, residual=None, weight=None, bias=None, eps: float = 1e-5, rms: bool = False, y=None, total=None,
                    stream=None):
    """Residual sum ``total = x + residual`` of [B,T,C] and its layer norm (or,
    with ``rms``, RMS norm) ``y = norm(total) weight + bias``; returns
    ``(y, total)``, total None without a residual.

    residual and total are of x's type or fp32; ``total`` may be ``residual``
    itself.  y comes from the sum before it is rounded to total's type.
    weight, bias are fp32 [C]."""
    if stream is not None:
        with _current(stream, x):
            return addnorm_forward(x, residual, weight, bias, eps, rms, y, total)
    fn = _fn.get("tfla_addnorm_fwd") or _entry("tfla_addnorm_fwd")
    dev = _first(x, "x", 3)
    shape, dtype, f32 = x.shape, x.dtype, torch.float32
    flags, c = _IO[dtype] | (_RMS if rms else 0), shape[2:]
    res = tot = _NO_ROWS
    y, yr = _out(y, "y", x, dtype, dev)
    if residual is not None:
        st = _stream_type(residual, "residual", dtype)
        if st is not dtype:
            flags |= _SUM_FP32
        res = _rows(residual, "residual", shape, st, dev)
        total, tot = _out(total, "total", residual, st, dev)
    elif total is not None:
        raise ValueError("total is given without a residual")
    packed = _ADDNORM.pack(*shape, flags, eps, *_rows(x, "x", shape, dtype, dev), *res,
                           _flat(weight, "weight", c, f32, dev), _flat(bias, "bias", c, f32, dev),
                           *yr, *tot, *_NO_ROWS * 4, 0, 0)
    _call("tfla_addnorm_fwd", packed, dev, None, None, fn)
    return y, total


def addnorm_backward(total, dy, weight=None, bias: bool = False, eps: float = 1e-5, rms: bool = False, dtotal=None, dx=None,
                     dresidual=None, workspace=None, stream=None):
    """Gradients of :func:`addnorm_forward` from its ``total`` (x where there
    was no residual), ``dy`` and ``dtotal``, the gradient of total from behind
    (or None); returns ``(dx, dresidual, dweight, dbias)``.

    The gradient of the sum, in dy's type and in total's: one tensor where
    these are the same.  dweight comes where weight is given, dbias with
    ``bias``."""
    if stream is not None:
        with _current(stream, dy):
            return addnorm_backward(total, dy, weight, bias, eps, rms, dtotal, dx, dresidual, workspace)
    need = _fn.get("tfla_addnorm_bwd_workspace_bytes") or _entry("tfla_addnorm_bwd_workspace_bytes")
    dev = _first(dy, "dy", 3)
    shape, dtype, f32 = dy.shape, dy.dtype, torch.float32
    flags, c = _IO[dtype] | (_RMS if rms else 0), shape[2:]
    st = _stream_type(total, "total", dtype)
    res = _NO_ROWS
    dx, dxr = _out(dx, "dx", dy, dtype, dev)
    if st is dtype:
        if dresidual is not None and dresidual is not dx:
            raise ValueError("dresidual is dx where dy and total have one type")
        dresidual = dx
    else:
        flags |= _SUM_FP32
        _rows(total, "total", shape, st, dev)   # before an output takes its shape
        dresidual, res = _out(dresidual, "dresidual", total, st, dev)
    dweight = None if weight is None else torch.empty_like(weight)
    dbias = None if not bias else dy.new_empty(c, dtype=f32) if weight is None else torch.empty_like(weight)
    packed = _ADDNORM.pack(*shape, flags, eps, *_NO_ROWS * 2, _flat(weight, "weight", c, f32, dev), 0, *_NO_ROWS,
                           *_rows(total, "total", shape, st, dev), *_rows(dy, "dy", shape, dtype, dev),
                           *(_NO_ROWS if dtotal is None else _rows(dtotal, "dtotal", shape, st, dev)),
                           *dxr, *res,
                           0 if dweight is None else dweight.data_ptr(), 0 if dbias is None else dbias.data_ptr())
    wanted = need(*shape, flags) if weight is not None or bias else None
    _call("tfla_addnorm_bwd", packed, dev, wanted or 0, workspace if wanted else None, _fn["tfla_addnorm_bwd"])
    return dx, dresidual, dweight, dbias
