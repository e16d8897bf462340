"""The operators around the recurrences on torch tensors (include/tfla.h):
causal depthwise convolution, selective state space scan, and group norm with
an activation or a gate; :mod:`mlstm_sequence_amd.tfla` offers the same names.

Argument checks, output allocation and marshalling only; the work runs in the
library's HIP kernels on torch's current stream of the tensors' device (or the
given one).  Activations are [B,T,...] with contiguous channels and any batch
and row strides, so views of projections need no copy; a tensor that does not
fit is refused, never copied.
"""
from __future__ import annotations

import ctypes
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


def bind(L):
    """Argument types of this module's entry points."""
    vp, sz = ctypes.c_void_p, ctypes.c_size_t
    for name, args, res in (
            ("tfla_conv_fwd", [ctypes.POINTER(ConvArgs), vp], _i),
            ("tfla_conv_bwd_workspace_bytes", [_i] * 5, sz),
            ("tfla_conv_bwd", [ctypes.POINTER(ConvArgs), vp, sz, vp], _i),
            ("tfla_scan_workspace_bytes", [_i] * 6, sz),
            ("tfla_scan_fwd", [ctypes.POINTER(ScanArgs), vp, sz, vp], _i),
            ("tfla_scan_bwd_workspace_bytes", [_i] * 6, sz),
            ("tfla_scan_bwd", [ctypes.POINTER(ScanArgs), vp, sz, vp], _i),
            ("tfla_norm_workspace_bytes", [_i] * 5, sz),
            ("tfla_norm_fwd", [ctypes.POINTER(NormArgs), vp, sz, vp], _i),
            ("tfla_norm_bwd_workspace_bytes", [_i] * 5, sz),
            ("tfla_norm_bwd", [ctypes.POINTER(NormArgs), vp, sz, vp], _i)):
        f = getattr(L, name)
        f.argtypes, f.restype = args, res


def _lib():
    from . import tfla
    return tfla.lib()


# ---- checks ------------------------------------------------------------------

def _first(x, name, dims):
    """The tensor that sets type and device."""
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
    return x.device


def _like(t, name, shape, dtype, dev):
    """Shape, type and device of ``t``; whether its last dimension is contiguous is left to the caller."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor, got {type(t).__name__}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.device != dev:
        raise ValueError(f"{name} is on {t.device}, other tensors on {dev}")


def _flat(t, name, shape, dtype, dev):
    """Pointer of a contiguous tensor (None: NULL)."""
    if t is None:
        return None
    _like(t, name, shape, dtype, dev)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous (row-major), got strides {t.stride()}")
    return t.data_ptr()


def _rows(t, name, shape, dtype, dev):
    """tfla_rows of a [B,T,D] tensor with contiguous channels."""
    _like(t, name, shape, dtype, dev)
    st = t.stride()
    if st[2] != 1 and shape[2] > 1:
        raise ValueError(f"{name} must have contiguous channels (last stride 1), got strides {st}")
    return Rows(t.data_ptr(), st[0], st[1])


def _call(name, args, dev, stream, nbytes=None, workspace=None):
    """Calls entry point ``name`` on ``stream`` (None: the device's current
    one) with the tensors' device current; ``nbytes``: the workspace it needs."""
    from . import tfla
    if dev.index != torch.cuda.current_device():
        with torch.cuda.device(dev):
            return _call(name, args, dev, stream, nbytes, workspace)
    current = torch.cuda.current_stream().cuda_stream
    s = current if stream is None else stream if isinstance(stream, int) else stream.cuda_stream
    fn = getattr(tfla.lib(), name)
    if nbytes is None:
        rc = fn(ctypes.byref(args), s)
    else:
        if workspace is not None:
            tfla._check_workspace(workspace, nbytes, dev)
            size = workspace.numel() * workspace.element_size()
        elif nbytes and s == current:
            workspace = torch.empty(nbytes, dtype=torch.uint8, device=dev)
            size = nbytes
        else:
            size = 0   # another stream than torch's current one: the library allocates in that stream's order
        rc = fn(ctypes.byref(args), None if workspace is None else workspace.data_ptr(), size, s)
    if rc:
        tfla._check(rc, name)


# ---- causal convolution --------------------------------------------------------

def _conv_args(x, weight, bias, act, state, lengths):
    dev = _first(x, "x", 3)
    B, T, D = x.shape
    if not isinstance(weight, torch.Tensor) or weight.dim() != 2:
        raise ValueError("weight must be a [D,K] tensor")
    K = weight.shape[1]
    a = ConvArgs()
    a.B, a.T, a.D, a.K, a.flags, a.act = B, T, D, K, _IO[x.dtype], act
    a.x = _rows(x, "x", x.shape, x.dtype, dev)
    a.weight = _flat(weight, "weight", (D, K), torch.float32, dev)
    a.bias = _flat(bias, "bias", (D,), torch.float32, dev)
    a.state = _flat(state, "state", (B, K - 1, D), x.dtype, dev)
    a.lengths = _flat(lengths, "lengths", (B,), torch.int32, dev)
    return a, dev


def conv_forward(x, weight, bias=None, act: int = ACT_SILU, state=None, lengths=None, want_state: bool = False,
                 y=None, state_out=None, stream=None):
    """Causal depthwise convolution of x [B,T,D] with weight [D,K] (fp32),
    ``y = act(conv(x) + bias)``; returns ``(y, state_out)``.

    ``state`` [B,K-1,D] holds the inputs before the first row (None: zeros);
    ``state_out`` (allocated with ``want_state``, may be ``state`` itself)
    receives the last K-1 inputs, what the next call continues from.
    ``lengths`` int32 [B]: valid rows of each sequence of a padded batch."""
    a, dev = _conv_args(x, weight, bias, act, state, lengths)
    if y is None:
        y = torch.empty(x.shape, dtype=x.dtype, device=dev)
    if state_out is None and want_state:
        state_out = torch.empty((a.B, a.K - 1, a.D), dtype=x.dtype, device=dev)
    a.y = _rows(y, "y", x.shape, x.dtype, dev)
    a.state_out = _flat(state_out, "state_out", (a.B, a.K - 1, a.D), x.dtype, dev)
    _call("tfla_conv_fwd", a, dev, stream)
    return y, state_out


def conv_backward(x, weight, dy, bias=None, act: int = ACT_SILU, state=None, lengths=None, dstate_out=None, dx=None,
                  workspace=None, stream=None):
    """Gradients of :func:`conv_forward` for ``dy`` and (with carried states)
    ``dstate_out``; returns ``(dx, dweight, dbias, dstate)``, dbias None
    without bias, dstate None without state."""
    a, dev = _conv_args(x, weight, bias, act, state, lengths)
    if dx is None:
        dx = torch.empty(x.shape, dtype=x.dtype, device=dev)
    dweight = torch.empty_like(weight)
    dbias = None if bias is None else torch.empty_like(bias)
    dstate = None if state is None else torch.empty_like(state)
    a.dy = _rows(dy, "dy", x.shape, x.dtype, dev)
    a.dx = _rows(dx, "dx", x.shape, x.dtype, dev)
    a.dstate_out = _flat(dstate_out, "dstate_out", (a.B, a.K - 1, a.D), x.dtype, dev)
    a.dweight = dweight.data_ptr()
    a.dbias = None if dbias is None else dbias.data_ptr()
    a.dstate = None if dstate is None else dstate.data_ptr()
    _call("tfla_conv_bwd", a, dev, stream, _lib().tfla_conv_bwd_workspace_bytes(a.B, a.T, a.D, a.K, a.flags), workspace)
    return dx, dweight, dbias, dstate


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
    _like(t, name, shape, dtype, dev)
    st = t.stride()
    if (st[3] != 1 and shape[3] > 1) or (st[2] != shape[3] and shape[2] > 1):
        raise ValueError(f"{name} must have its last two dimensions contiguous, got strides {st}")
    return Rows(t.data_ptr(), st[0], st[1])


def _scan_args(x, dt, a, bmat, cmat, skip, z, dt_bias, softplus, state, lengths):
    dev = _first(x, "x", 3)
    shape, dtype = x.shape, x.dtype
    B, T, D = shape
    if not isinstance(bmat, torch.Tensor) or bmat.dim() != 4:
        raise ValueError("bmat and cmat must be [B,T,G,N] tensors")
    G, N = bmat.shape[2:]
    s = ScanArgs()
    s.B, s.T, s.D, s.N, s.G, s.flags = B, T, D, N, G, _IO[dtype] | (SCAN_SOFTPLUS if softplus else 0)
    s.x = _rows(x, "x", shape, dtype, dev)
    s.dt = _rows(dt, "dt", shape, dtype, dev)
    if z is not None:
        s.z = _rows(z, "z", shape, dtype, dev)
    s.bmat = _group_rows(bmat, "bmat", (B, T, G, N), dtype, dev)
    s.cmat = _group_rows(cmat, "cmat", (B, T, G, N), dtype, dev)
    s.a = _flat(a, "a", (D, N), torch.float32, dev)
    s.skip = _flat(skip, "skip", (D,), torch.float32, dev)
    s.dt_bias = _flat(dt_bias, "dt_bias", (D,), torch.float32, dev)
    s.state = _flat(state, "state", (B, D, N), torch.float32, dev)
    s.lengths = _flat(lengths, "lengths", (B,), torch.int32, dev)
    return s, dev


def scan_forward(x, dt, a, bmat, cmat, skip=None, z=None, dt_bias=None, softplus: bool = True, state=None, lengths=None,
                 want_state: bool = False, y=None, state_out=None, workspace=None, stream=None):
    """Selective state space scan of x [B,T,D]: ``delta = softplus(dt + dt_bias)``,
    ``h = exp(delta a) h + delta x bmat``, ``y = cmat . h + skip x``, times
    ``z sigmoid(z)`` when z is given; returns ``(y, state_out)``.

    a [D,N], skip and dt_bias [D] are fp32; bmat, cmat [B,T,G,N] serve D/G
    channels each.  ``state`` fp32 [B,D,N] is the state before the first row;
    ``state_out`` (allocated with ``want_state``, may be ``state`` itself) the
    one after the last.  ``lengths`` int32 [B]: valid rows of a padded batch."""
    s, dev = _scan_args(x, dt, a, bmat, cmat, skip, z, dt_bias, softplus, state, lengths)
    if y is None:
        y = torch.empty(x.shape, dtype=x.dtype, device=dev)
    if state_out is None and want_state:
        state_out = torch.empty((s.B, s.D, s.N), dtype=torch.float32, device=dev)
    s.y = _rows(y, "y", x.shape, x.dtype, dev)
    s.state_out = _flat(state_out, "state_out", (s.B, s.D, s.N), torch.float32, dev)
    n = _lib().tfla_scan_workspace_bytes(s.B, s.T, s.D, s.N, s.G, s.flags)
    _call("tfla_scan_fwd", s, dev, stream, n, workspace)
    return y, state_out


def scan_backward(x, dt, a, bmat, cmat, dy, skip=None, z=None, dt_bias=None, softplus: bool = True, state=None,
                  lengths=None, dstate_out=None, dx=None, ddt=None, dz=None, dbmat=None, dcmat=None, workspace=None,
                  stream=None) -> ScanGrads:
    """Gradients of :func:`scan_forward` for ``dy`` and (with carried states)
    ``dstate_out``.  dx, ddt, dz, dbmat and dcmat may be given, as parts of
    a projection's gradient for instance."""
    s, dev = _scan_args(x, dt, a, bmat, cmat, skip, z, dt_bias, softplus, state, lengths)
    shape, dtype, bc = x.shape, x.dtype, bmat.shape
    new = lambda like, t: torch.empty(like, dtype=dtype, device=dev) if t is None else t  # noqa: E731
    dx, ddt, dbmat, dcmat = new(shape, dx), new(shape, ddt), new(bc, dbmat), new(bc, dcmat)
    dz = None if z is None else new(shape, dz)
    da = torch.empty_like(a)
    dskip = None if skip is None else torch.empty_like(skip)
    ddt_bias = None if dt_bias is None else torch.empty_like(dt_bias)
    dstate = None if state is None else torch.empty_like(state)
    s.dy = _rows(dy, "dy", shape, dtype, dev)
    s.dstate_out = _flat(dstate_out, "dstate_out", (s.B, s.D, s.N), torch.float32, dev)
    s.dx = _rows(dx, "dx", shape, dtype, dev)
    s.ddt = _rows(ddt, "ddt", shape, dtype, dev)
    if z is not None:
        s.dz = _rows(dz, "dz", shape, dtype, dev)
    s.dbmat = _group_rows(dbmat, "dbmat", bc, dtype, dev)
    s.dcmat = _group_rows(dcmat, "dcmat", bc, dtype, dev)
    s.da = da.data_ptr()
    s.dskip = None if dskip is None else dskip.data_ptr()
    s.ddt_bias = None if ddt_bias is None else ddt_bias.data_ptr()
    s.dstate = None if dstate is None else dstate.data_ptr()
    n = _lib().tfla_scan_bwd_workspace_bytes(s.B, s.T, s.D, s.N, s.G, s.flags)
    _call("tfla_scan_bwd", s, dev, stream, n, workspace)
    return ScanGrads(dx, ddt, da, dbmat, dcmat, dskip, dz, ddt_bias, dstate)


# ---- group norm --------------------------------------------------------------------------

def _heads(t, name, shape, dtype, dev):
    """tfla_heads of a [B,T,G,C] tensor with contiguous channels."""
    _like(t, name, shape, dtype, dev)
    st = t.stride()
    if st[3] != 1 and shape[3] > 1:
        raise ValueError(f"{name} must have contiguous channels (last stride 1), got strides {st}")
    return Heads(t.data_ptr(), st[0], st[1], st[2])


def _norm_args(x, weight, bias, act, gate, over):
    dev = _first(x, "x", 4)
    shape, dtype = x.shape, x.dtype
    if over not in (NORM_TOKEN, NORM_SEQUENCE):
        raise ValueError(f"over must be NORM_TOKEN or NORM_SEQUENCE, got {over}")
    a = NormArgs()
    a.B, a.T, a.G, a.C = shape
    a.flags, a.act = _IO[dtype] | over, act
    a.x = _heads(x, "x", shape, dtype, dev)
    if gate is not None:
        a.gate = _heads(gate, "gate", shape, dtype, dev)
    a.weight = _flat(weight, "weight", shape[2:], torch.float32, dev)
    a.bias = _flat(bias, "bias", shape[2:], torch.float32, dev)
    return a, dev


def norm_forward(x, weight=None, bias=None, eps: float = 1e-5, act: int = ACT_NONE, gate=None, over: int = NORM_TOKEN,
                 y=None, workspace=None, stream=None):
    """Group norm of x [B,T,G,C] over the channels of each group, per token or
    (``over=NORM_SEQUENCE``) over all T rows, then ``y = act(u)`` or, with a
    gate, ``y = u act(gate)``; returns ``(y, mean, rstd)``.

    weight, bias are fp32 [G,C]; mean, rstd fp32 [B,T,G] or [B,G].  The
    recurrences' head-major output h [B,H,T,d] goes in as
    ``h.transpose(1, 2)``; y is contiguous [B,T,G,C] unless given."""
    a, dev = _norm_args(x, weight, bias, act, gate, over)
    if y is None:
        y = torch.empty(x.shape, dtype=x.dtype, device=dev)
    a.eps = eps
    a.y = _heads(y, "y", x.shape, x.dtype, dev)
    stats = (a.B, a.G) if over else (a.B, a.T, a.G)
    mean = torch.empty(stats, dtype=torch.float32, device=dev)
    rstd = torch.empty(stats, dtype=torch.float32, device=dev)
    a.mean, a.rstd = mean.data_ptr(), rstd.data_ptr()
    n = _lib().tfla_norm_workspace_bytes(a.B, a.T, a.G, a.C, a.flags)
    _call("tfla_norm_fwd", a, dev, stream, n, workspace)
    return y, mean, rstd


def norm_backward(x, dy, mean, rstd, weight=None, bias=None, act: int = ACT_NONE, gate=None, over: int = NORM_TOKEN,
                  dx=None, dgate=None, workspace=None, stream=None):
    """Gradients of :func:`norm_forward` for ``dy`` from its mean and rstd;
    returns ``(dx, dgate, dweight, dbias)``, None where the input was None."""
    a, dev = _norm_args(x, weight, bias, act, gate, over)
    shape, dtype = x.shape, x.dtype
    if dx is None:
        dx = torch.empty(shape, dtype=dtype, device=dev)
    if gate is None:
        dgate = None
    else:
        if dgate is None:
            dgate = torch.empty(shape, dtype=dtype, device=dev)
        a.dgate = _heads(dgate, "dgate", shape, dtype, dev)
    dweight = None if weight is None else torch.empty_like(weight)
    dbias = None if bias is None else torch.empty_like(bias)
    stats = (a.B, a.G) if over else (a.B, a.T, a.G)
    a.dy = _heads(dy, "dy", shape, dtype, dev)
    a.dx = _heads(dx, "dx", shape, dtype, dev)
    a.mean = _flat(mean, "mean", stats, torch.float32, dev)
    a.rstd = _flat(rstd, "rstd", stats, torch.float32, dev)
    a.dweight = None if dweight is None else dweight.data_ptr()
    a.dbias = None if dbias is None else dbias.data_ptr()
    n = _lib().tfla_norm_bwd_workspace_bytes(a.B, a.T, a.G, a.C, a.flags)
    _call("tfla_norm_bwd", a, dev, stream, n, workspace)
    return dx, dgate, dweight, dbias
