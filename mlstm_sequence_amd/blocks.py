"""The operators around the recurrences on torch tensors (include/tfla.h):
causal depthwise convolution, selective state space scan, and group norm with
an activation or a gate; :mod:`mlstm_sequence_amd.tfla` offers the same names.

Argument checks, output allocation and marshalling only; the work runs in the
library's HIP kernels on torch's current stream of the tensors' device, or with
``stream`` as under ``torch.cuda.stream(stream)``: outputs and workspaces are
allocated there, and the caller orders what other streams do with the tensors
(and records those streams on them).  Activations are [B,T,...] with contiguous
channels and any batch and row strides, so views of projections need no copy; a
tensor that does not fit is refused, never copied.
"""
from __future__ import annotations

import contextlib
import ctypes
import struct
from typing import NamedTuple, Optional

import torch

ACT_NONE, ACT_SILU, ACT_SIGMOID = 0, 1, 2

SCAN_SOFTPLUS = 0x1000
NORM_TOKEN, NORM_SEQUENCE = 0, 0x2000   # statistics of a group: per token, or over the whole sequence

_IO = {torch.bfloat16: 0x100, torch.float32: 0}
_i, _p, _ll = ctypes.c_int, ctypes.c_void_p, ctypes.c_longlong


class Rows(ctypes.Structure):
    """tfla_rows: data pointer, batch and row strides in elements."""
    _fields_ = [("data", _p), ("batch", _ll), ("row", _ll)]


class ConvArgs(ctypes.Structure):
    """tfla_conv_args."""
    _fields_ = [("B", _i), ("T", _i), ("D", _i), ("K", _i), ("flags", _i), ("act", _i),
                ("x", Rows), ("weight", _p), ("bias", _p), ("state", _p), ("lengths", _p),
                ("y", Rows), ("state_out", _p),
                ("dy", Rows), ("dstate_out", _p), ("dx", Rows), ("dweight", _p), ("dbias", _p), ("dstate", _p)]


class ScanArgs(ctypes.Structure):
    """tfla_scan_args."""
    _fields_ = [("B", _i), ("T", _i), ("D", _i), ("N", _i), ("G", _i), ("flags", _i),
                ("x", Rows), ("dt", Rows), ("z", Rows), ("bmat", Rows), ("cmat", Rows),
                ("a", _p), ("skip", _p), ("dt_bias", _p), ("state", _p), ("lengths", _p),
                ("y", Rows), ("state_out", _p),
                ("dy", Rows), ("dstate_out", _p), ("dx", Rows), ("ddt", Rows), ("dz", Rows), ("dbmat", Rows),
                ("dcmat", Rows), ("da", _p), ("dskip", _p), ("ddt_bias", _p), ("dstate", _p)]


class Heads(ctypes.Structure):
    """tfla_heads: data pointer, batch, row and group strides in elements."""
    _fields_ = [("data", _p), ("batch", _ll), ("row", _ll), ("group", _ll)]


class NormArgs(ctypes.Structure):
    """tfla_norm_args."""
    _fields_ = [("B", _i), ("T", _i), ("G", _i), ("C", _i), ("flags", _i), ("act", _i), ("eps", ctypes.c_float),
                ("x", Heads), ("gate", Heads), ("weight", _p), ("bias", _p), ("mean", _p), ("rstd", _p),
                ("y", Heads), ("dy", Heads), ("dx", Heads), ("dgate", Heads), ("dweight", _p), ("dbias", _p)]


_fn = {}   # this module's entry points, once the library is loaded


def bind(L):
    """Argument types of this module's entry points, which are offered all at
    once: another thread may be on its first call."""
    global _fn
    vp, sz = ctypes.c_void_p, ctypes.c_size_t
    fn = {}
    for name, args, res in (
            ("tfla_conv_fwd", [vp, vp], _i),
            ("tfla_conv_bwd_workspace_bytes", [_i] * 5, sz),
            ("tfla_conv_bwd", [vp, vp, sz, vp], _i),
            ("tfla_scan_workspace_bytes", [_i] * 6, sz),
            ("tfla_scan_fwd", [vp, vp, sz, vp], _i),
            ("tfla_scan_bwd_workspace_bytes", [_i] * 6, sz),
            ("tfla_scan_bwd", [vp, vp, sz, vp], _i),
            ("tfla_norm_workspace_bytes", [_i] * 5, sz),
            ("tfla_norm_fwd", [vp, vp, sz, vp], _i),
            ("tfla_norm_bwd_workspace_bytes", [_i] * 5, sz),
            ("tfla_norm_bwd", [vp, vp, sz, vp], _i)):
        f = getattr(L, name)
        f.argtypes, f.restype = args, res
        fn[name] = f
    _fn = fn


def _entry(name):
    if not _fn:
        from . import tfla
        tfla.lib()
    return _fn[name]


# The argument structures as the calls below fill them: a tuple of their
# fields in order, packed at once (a ctypes structure filled field by field
# takes most of a small call's time).
_ROWS, _HEADS = "Pqq", "Pqqq"
_CONV = struct.Struct("@6i" + _ROWS + "4P" + _ROWS + "P" + _ROWS + "P" + _ROWS + "3P")
_SCAN = struct.Struct("@6i" + _ROWS * 5 + "5P" + _ROWS + "P" + _ROWS + "P" + _ROWS * 5 + "4P")
_NORM = struct.Struct("@6if" + _HEADS * 2 + "4P" + _HEADS * 4 + "2P")
_NO_ROWS, _NO_HEADS = (0, 0, 0), (0, 0, 0, 0)


# ---- checks ------------------------------------------------------------------

def _first(x, name, dims):
    """Checks the tensor that sets type and device; returns the device's index."""
    if not isinstance(x, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor, got {type(x).__name__}")
    if x.dtype not in _IO:
        raise TypeError(f"{name} must be bfloat16 or float32, got {x.dtype}")
    if x.dim() != dims:
        raise ValueError(f"{name} must have {dims} dimensions, got shape {tuple(x.shape)}")
    if max(x.shape, default=0) > 0x7FFFFFFF:
        raise ValueError(f"{name}: dimensions above 2^31 - 1 are not supported, got {tuple(x.shape)}")
    if not x.is_cuda:
        raise ValueError(f"tensors must live in GPU memory, got {name} on {x.device}")
    return x.get_device()


def _bad(t, name, shape, dtype, dev):
    """Raises for the first thing about ``t`` that does not fit."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor, got {type(t).__name__}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, other tensors on cuda:{dev}")
    raise ValueError(f"{name} has strides {t.stride()}: its innermost dimensions must be contiguous")


def _fits(t, shape, dtype, dev):
    return isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.get_device() == dev


def _flat(t, name, shape, dtype, dev):
    """Pointer of a contiguous tensor (None: NULL)."""
    if t is None:
        return 0
    if not _fits(t, shape, dtype, dev) or not t.is_contiguous():
        _bad(t, name, shape, dtype, dev)
    return t.data_ptr()


def _rows(t, name, shape, dtype, dev):
    """tfla_rows of a [B,T,D] tensor with contiguous channels."""
    if not _fits(t, shape, dtype, dev):
        _bad(t, name, shape, dtype, dev)
    st = t.stride()
    if st[2] != 1 and shape[2] > 1:
        _bad(t, name, shape, dtype, dev)
    return t.data_ptr(), st[0], st[1]


# the current stream's handle without a Stream object around it, where torch offers that
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda dev: torch.cuda.current_stream(dev).cuda_stream)

# the current device, which tensors in GPU memory have initialised, without the checks around it
_this_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device

_HERE = contextlib.nullcontext()


def _current(stream, x):
    """Context with ``stream`` (a torch stream, a raw handle, or None for the
    current one) as the current stream of the device of ``x``, for all that a
    call allocates: memory of another stream could still be in use by that
    stream's pending work when a kernel writes it, and be handed out there
    again before the kernel is done."""
    if stream is None or not getattr(x, "is_cuda", False):   # tensors elsewhere are refused by the checks
        return _HERE
    dev = x.get_device()
    handle = stream if isinstance(stream, int) else stream.cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        if stream.device_index != dev:
            raise ValueError(f"stream is on {stream.device}, tensors on cuda:{dev}")
    elif handle <= 1:   # the null stream's two names
        stream = torch.cuda.default_stream(dev)
        handle = stream.cuda_stream
    else:
        stream = torch.cuda.ExternalStream(handle, device=dev)
    return _HERE if handle == _raw_stream(dev) else torch.cuda.stream(stream)


def _call(name, packed, dev, nbytes=None, workspace=None, fn=None):
    """Calls entry point ``name`` (of this module, or ``fn``) on the current
    stream of the tensors' device with that device current; ``nbytes``: the
    workspace it needs."""
    if dev != _this_device():
        with torch.cuda.device(dev):
            return _call(name, packed, dev, nbytes, workspace, fn)
    fn = fn or _fn[name]
    s = _raw_stream(dev)
    if nbytes is None:
        rc = fn(packed, s)
    else:
        at = size = 0
        if workspace is not None:
            from . import tfla
            tfla._check_workspace(workspace, nbytes, torch.device("cuda", dev))
            at, size = workspace.data_ptr(), workspace.numel() * workspace.element_size()
        elif nbytes:
            workspace = torch.empty(nbytes, dtype=torch.uint8, device=dev)
            at, size = workspace.data_ptr(), nbytes
        rc = fn(packed, at, size, s)
    if rc:
        from . import tfla
        tfla._check(rc, name)


# ---- causal convolution --------------------------------------------------------

def _conv_args(x, weight, bias, act, state, lengths):
    """(fields shared by both directions, device, K)"""
    dev = _first(x, "x", 3)
    shape, dtype = x.shape, x.dtype
    B, T, D = shape
    if act not in (ACT_NONE, ACT_SILU):
        raise ValueError(f"act must be ACT_NONE or ACT_SILU, got {act}")
    if not isinstance(weight, torch.Tensor) or weight.dim() != 2:
        raise ValueError("weight must be a [D,K] tensor")
    K = weight.shape[1]
    return (B, T, D, K, _IO[dtype], act, *_rows(x, "x", shape, dtype, dev),
            _flat(weight, "weight", (D, K), torch.float32, dev), _flat(bias, "bias", (D,), torch.float32, dev),
            _flat(state, "state", (B, K - 1, D), dtype, dev), _flat(lengths, "lengths", (B,), torch.int32, dev)), dev, K


def conv_forward(x, weight, bias=None, act: int = ACT_SILU, state=None, lengths=None, want_state: bool = False,
                 y=None, state_out=None, stream=None):
    """Causal depthwise convolution of x [B,T,D] with weight [D,K] (fp32),
    ``y = act(conv(x) + bias)``; returns ``(y, state_out)``.

    ``state`` [B,K-1,D] holds the inputs before the first row (None: zeros);
    ``state_out`` (allocated with ``want_state``, may be ``state`` itself)
    receives the last K-1 inputs, what the next call continues from.
    ``lengths`` int32 [B]: valid rows of each sequence of a padded batch."""
    _entry("tfla_conv_fwd")
    with _current(stream, x):
        a, dev, K = _conv_args(x, weight, bias, act, state, lengths)
        shape, dtype = x.shape, x.dtype
        B, _, D = shape
        if y is None:
            y = x.new_empty(shape)
        if state_out is None and want_state:
            state_out = x.new_empty((B, K - 1, D))
        packed = _CONV.pack(*a, *_rows(y, "y", shape, dtype, dev),
                            _flat(state_out, "state_out", (B, K - 1, D), dtype, dev), *_NO_ROWS, 0, *_NO_ROWS, 0, 0, 0)
        _call("tfla_conv_fwd", packed, dev)
        return y, state_out


def conv_backward(x, weight, dy, bias=None, act: int = ACT_SILU, state=None, lengths=None, dstate_out=None, dx=None,
                  workspace=None, stream=None):
    """Gradients of :func:`conv_forward` for ``dy`` and (with carried states)
    ``dstate_out``; returns ``(dx, dweight, dbias, dstate)``, dbias None
    without bias, dstate None without state."""
    need = _entry("tfla_conv_bwd_workspace_bytes")
    with _current(stream, x):
        a, dev, K = _conv_args(x, weight, bias, act, state, lengths)
        shape, dtype = x.shape, x.dtype
        B, T, D = shape
        if dx is None:
            dx = x.new_empty(shape)
        dweight = torch.empty_like(weight)
        dbias = None if bias is None else torch.empty_like(bias)
        dstate = None if state is None else torch.empty_like(state)
        packed = _CONV.pack(*a, *_NO_ROWS, 0, *_rows(dy, "dy", shape, dtype, dev),
                            _flat(dstate_out, "dstate_out", (B, K - 1, D), dtype, dev),
                            *_rows(dx, "dx", shape, dtype, dev), *map(_ptr, (dweight, dbias, dstate)))
        _call("tfla_conv_bwd", packed, dev, need(B, T, D, K, _IO[dtype]), workspace)
        return dx, dweight, dbias, dstate


def _ptr(t):
    return 0 if t is None else t.data_ptr()


# ---- selective scan ------------------------------------------------------------------

class ScanGrads(NamedTuple):
    """Gradients of :func:`scan_forward`; None where the input was None."""
    dx: torch.Tensor
    ddt: torch.Tensor
    da: torch.Tensor
    dbmat: torch.Tensor
    dcmat: torch.Tensor
    dskip: Optional[torch.Tensor]
    dz: Optional[torch.Tensor]
    ddt_bias: Optional[torch.Tensor]
    dstate: Optional[torch.Tensor]


def _group_rows(t, name, shape, dtype, dev):
    """tfla_rows of a [B,T,G,N] tensor whose last two dimensions are contiguous."""
    if not _fits(t, shape, dtype, dev):
        _bad(t, name, shape, dtype, dev)
    st = t.stride()
    if (st[3] != 1 and shape[3] > 1) or (st[2] != shape[3] and shape[2] > 1):
        _bad(t, name, shape, dtype, dev)
    return t.data_ptr(), st[0], st[1]


def _scan_args(x, dt, a, bmat, cmat, skip, z, dt_bias, softplus, state, lengths):
    """(fields shared by both directions, sizes of the workspace calls, device)"""
    dev = _first(x, "x", 3)
    shape, dtype, f32 = x.shape, x.dtype, torch.float32
    B, T, D = shape
    if not isinstance(bmat, torch.Tensor) or bmat.dim() != 4:
        raise ValueError("bmat and cmat must be [B,T,G,N] tensors")
    G, N = bmat.shape[2:]
    sizes = (B, T, D, N, G, _IO[dtype] | (SCAN_SOFTPLUS if softplus else 0))
    return (*sizes, *_rows(x, "x", shape, dtype, dev), *_rows(dt, "dt", shape, dtype, dev),
            *(_NO_ROWS if z is None else _rows(z, "z", shape, dtype, dev)),
            *_group_rows(bmat, "bmat", (B, T, G, N), dtype, dev), *_group_rows(cmat, "cmat", (B, T, G, N), dtype, dev),
            _flat(a, "a", (D, N), f32, dev), _flat(skip, "skip", (D,), f32, dev),
            _flat(dt_bias, "dt_bias", (D,), f32, dev), _flat(state, "state", (B, D, N), f32, dev),
            _flat(lengths, "lengths", (B,), torch.int32, dev)), sizes, dev


def scan_forward(x, dt, a, bmat, cmat, skip=None, z=None, dt_bias=None, softplus: bool = True, state=None, lengths=None,
                 want_state: bool = False, y=None, state_out=None, workspace=None, stream=None):
    """Selective state space scan of x [B,T,D]: ``delta = softplus(dt + dt_bias)``,
    ``h = exp(delta a) h + delta x bmat``, ``y = cmat . h + skip x``, times
    ``z sigmoid(z)`` when z is given; returns ``(y, state_out)``.

    a [D,N], skip and dt_bias [D] are fp32; bmat, cmat [B,T,G,N] serve D/G
    channels each.  ``state`` fp32 [B,D,N] is the state before the first row;
    ``state_out`` (allocated with ``want_state``, may be ``state`` itself) the
    one after the last.  ``lengths`` int32 [B]: valid rows of a padded batch."""
    need = _entry("tfla_scan_workspace_bytes")
    with _current(stream, x):
        fields, sizes, dev = _scan_args(x, dt, a, bmat, cmat, skip, z, dt_bias, softplus, state, lengths)
        B, T, D, N = sizes[:4]
        if y is None:
            y = x.new_empty(x.shape)
        if state_out is None and want_state:
            state_out = a.new_empty((B, D, N))
        packed = _SCAN.pack(*fields, *_rows(y, "y", x.shape, x.dtype, dev),
                            _flat(state_out, "state_out", (B, D, N), torch.float32, dev), *_NO_ROWS, 0,
                            *_NO_ROWS * 5, 0, 0, 0, 0)
        _call("tfla_scan_fwd", packed, dev, need(*sizes), workspace)
        return y, state_out


def scan_backward(x, dt, a, bmat, cmat, dy, skip=None, z=None, dt_bias=None, softplus: bool = True, state=None,
                  lengths=None, dstate_out=None, dx=None, ddt=None, dz=None, dbmat=None, dcmat=None, workspace=None,
                  stream=None) -> ScanGrads:
    """Gradients of :func:`scan_forward` for ``dy`` and (with carried states)
    ``dstate_out``.  dx, ddt, dz, dbmat and dcmat may be given, as parts of
    a projection's gradient for instance."""
    need = _entry("tfla_scan_bwd_workspace_bytes")
    with _current(stream, x):
        fields, sizes, dev = _scan_args(x, dt, a, bmat, cmat, skip, z, dt_bias, softplus, state, lengths)
        shape, dtype, bc = x.shape, x.dtype, bmat.shape
        B, T, D, N = sizes[:4]
        dx, ddt = (x.new_empty(shape) if t is None else t for t in (dx, ddt))
        dbmat, dcmat = (x.new_empty(bc) if t is None else t for t in (dbmat, dcmat))
        dz = None if z is None else x.new_empty(shape) if dz is None else dz
        da = torch.empty_like(a)
        dskip = None if skip is None else torch.empty_like(skip)
        ddt_bias = None if dt_bias is None else torch.empty_like(dt_bias)
        dstate = None if state is None else torch.empty_like(state)
        packed = _SCAN.pack(*fields, *_NO_ROWS, 0, *_rows(dy, "dy", shape, dtype, dev),
                            _flat(dstate_out, "dstate_out", (B, D, N), torch.float32, dev),
                            *_rows(dx, "dx", shape, dtype, dev), *_rows(ddt, "ddt", shape, dtype, dev),
                            *(_NO_ROWS if z is None else _rows(dz, "dz", shape, dtype, dev)),
                            *_group_rows(dbmat, "dbmat", bc, dtype, dev), *_group_rows(dcmat, "dcmat", bc, dtype, dev),
                            *map(_ptr, (da, dskip, ddt_bias, dstate)))
        _call("tfla_scan_bwd", packed, dev, need(*sizes), workspace)
        return ScanGrads(dx, ddt, da, dbmat, dcmat, dskip, dz, ddt_bias, dstate)


# ---- group norm --------------------------------------------------------------------------

def _heads(t, name, shape, dtype, dev):
    """tfla_heads of a [B,T,G,C] tensor with contiguous channels."""
    if not _fits(t, shape, dtype, dev):
        _bad(t, name, shape, dtype, dev)
    st = t.stride()
    if st[3] != 1 and shape[3] > 1:
        _bad(t, name, shape, dtype, dev)
    return t.data_ptr(), st[0], st[1], st[2]


def _norm_args(x, weight, bias, act, gate, over, eps):
    """(fields up to bias, sizes of the workspace calls, device)"""
    dev = _first(x, "x", 4)
    shape, dtype = x.shape, x.dtype
    if over not in (NORM_TOKEN, NORM_SEQUENCE):
        raise ValueError(f"over must be NORM_TOKEN or NORM_SEQUENCE, got {over}")
    if act not in (ACT_NONE, ACT_SILU, ACT_SIGMOID):
        raise ValueError(f"act must be ACT_NONE, ACT_SILU or ACT_SIGMOID, got {act}")
    sizes = (*shape, _IO[dtype] | over)
    gc = shape[2:]
    return (*sizes, act, float(eps), *_heads(x, "x", shape, dtype, dev),
            *(_NO_HEADS if gate is None else _heads(gate, "gate", shape, dtype, dev)),
            _flat(weight, "weight", gc, torch.float32, dev), _flat(bias, "bias", gc, torch.float32, dev)), sizes, dev


def norm_forward(x, weight=None, bias=None, eps: float = 1e-5, act: int = ACT_NONE, gate=None, over: int = NORM_TOKEN,
                 y=None, workspace=None, stream=None):
    """Group norm of x [B,T,G,C] over the channels of each group, per token or
    (``over=NORM_SEQUENCE``) over all T rows, then ``y = act(u)`` or, with a
    gate, ``y = u act(gate)``; returns ``(y, mean, rstd)``.

    weight, bias are fp32 [G,C]; mean, rstd fp32 [B,T,G] or [B,G].  The
    recurrences' head-major output h [B,H,T,d] goes in as
    ``h.transpose(1, 2)``; y is contiguous [B,T,G,C] unless given."""
    need = _entry("tfla_norm_workspace_bytes")
    with _current(stream, x):
        fields, sizes, dev = _norm_args(x, weight, bias, act, gate, over, eps)
        B, T, G, C = shape = x.shape
        if y is None:
            y = x.new_empty(shape)
        stats = (B, G) if over else (B, T, G)
        mean = torch.empty(stats, dtype=torch.float32, device=x.device)
        rstd = torch.empty_like(mean)
        packed = _NORM.pack(*fields, mean.data_ptr(), rstd.data_ptr(), *_heads(y, "y", shape, x.dtype, dev),
                            *_NO_HEADS * 3, 0, 0)
        _call("tfla_norm_fwd", packed, dev, need(*sizes), workspace)
        return y, mean, rstd


def norm_backward(x, dy, mean, rstd, weight=None, bias=None, act: int = ACT_NONE, gate=None, over: int = NORM_TOKEN,
                  dx=None, dgate=None, workspace=None, stream=None):
    """Gradients of :func:`norm_forward` for ``dy`` from its mean and rstd;
    returns ``(dx, dgate, dweight, dbias)``, None where the input was None."""
    need = _entry("tfla_norm_bwd_workspace_bytes")
    with _current(stream, x):
        fields, sizes, dev = _norm_args(x, weight, bias, act, gate, over, 0.0)
        B, T, G, C = shape = x.shape
        dtype = x.dtype
        if dx is None:
            dx = x.new_empty(shape)
        dgate = None if gate is None else x.new_empty(shape) if dgate is None else dgate
        dweight = None if weight is None else torch.empty_like(weight)
        dbias = None if bias is None else torch.empty_like(bias)
        stats = (B, G) if over else (B, T, G)
        packed = _NORM.pack(*fields, _flat(mean, "mean", stats, torch.float32, dev),
                            _flat(rstd, "rstd", stats, torch.float32, dev), *_NO_HEADS,
                            *_heads(dy, "dy", shape, dtype, dev), *_heads(dx, "dx", shape, dtype, dev),
                            *(_NO_HEADS if gate is None else _heads(dgate, "dgate", shape, dtype, dev)),
                            _ptr(dweight), _ptr(dbias))
        _call("tfla_norm_bwd", packed, dev, need(*sizes), workspace)
        return dx, dgate, dweight, dbias
