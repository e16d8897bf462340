"""Refusals of the operators around the recurrences, on the CPU: bad
arguments are answered by the host checks, before any HIP call.  Pointers are
fake aligned device addresses that no check follows."""
import ctypes

import pytest
import torch

tfla = pytest.importorskip("mlstm_sequence_amd.tfla")
from mlstm_sequence_amd import blocks  # noqa: E402

BF16 = 0x100
INVALID, UNSUPPORTED, OOM = 1, 2, 4


def at(n):
    return 0x100000000 * (n + 1)


@pytest.fixture(scope="module", autouse=True)
def _built():
    import os
    if not os.path.exists(tfla.LIB_PATH):
        pytest.skip("libtfla.so not built")
    tfla.lib()


def put(args, kw):
    """Sets fields; "x.row" names a field of a field."""
    for k, v in kw.items():
        o = args
        *path, last = k.split(".")
        for name in path:
            o = getattr(o, name)
        setattr(o, last, v)
    return args


# ---- convolution -------------------------------------------------------------------

def conv_args(**kw):
    B, T, D, K = 2, 300, 64, 4
    a = blocks.ConvArgs(B=B, T=T, D=D, K=K, flags=BF16, act=1)
    rows = lambda p: blocks.Rows(p, T * D, D)  # noqa: E731
    a.x, a.y, a.dy, a.dx = rows(at(0)), rows(at(1)), rows(at(2)), rows(at(3))
    a.weight, a.bias, a.state, a.state_out, a.lengths = at(4), at(5), at(6), at(7), at(8)
    a.dstate_out, a.dweight, a.dbias, a.dstate = at(9), at(10), at(11), at(12)
    return put(a, kw)


CONV_BOTH = [
    ({"B": 0}, INVALID), ({"T": 0}, INVALID), ({"D": -1}, INVALID), ({"K": 0}, INVALID), ({"K": 9}, UNSUPPORTED),
    ({"flags": 0x200}, INVALID), ({"act": 2}, INVALID), ({"act": -1}, INVALID),
    ({"B": 1 << 16, "T": 1 << 15}, UNSUPPORTED), ({"D": (1 << 24) + 1}, UNSUPPORTED),
    ({"x.data": None}, INVALID), ({"weight": None}, INVALID), ({"x.data": at(0) + 1}, INVALID),
    ({"weight": at(4) + 2}, INVALID), ({"bias": at(5) + 1}, INVALID), ({"lengths": at(8) + 2}, INVALID),
    ({"state": at(6) + 1}, INVALID), ({"x.row": -1}, INVALID), ({"x.batch": -64}, INVALID),
    ({"x.row": 1 << 62}, INVALID), ({"x.batch": 1 << 50}, INVALID),
]


@pytest.mark.parametrize("kw,code", CONV_BOTH + [
    ({"y.data": None}, INVALID), ({"y.row": 63}, INVALID), ({"y.batch": 0}, INVALID), ({"y.batch": 64}, INVALID),
    ({"y.data": at(0)}, INVALID), ({"y.data": at(4)}, INVALID), ({"state_out": at(0) + 128}, INVALID),
    ({"state_out": at(6) + 2}, INVALID), ({"state_out": at(1)}, INVALID), ({"y.data": at(8) - 2}, INVALID),
])
def test_conv_fwd_refuses(kw, code):
    assert tfla.lib().tfla_conv_fwd(ctypes.byref(conv_args(**kw)), None) == code
    assert tfla.tfla_last_error()


@pytest.mark.parametrize("kw,code", CONV_BOTH + [
    ({"dy.data": None}, INVALID), ({"dx.data": None}, INVALID), ({"dweight": None}, INVALID), ({"dbias": None}, INVALID),
    ({"bias": None}, INVALID), ({"dx.row": 32}, INVALID), ({"dx.data": at(2)}, INVALID), ({"dx.data": at(0)}, INVALID),
    ({"dstate": at(9)}, INVALID), ({"dstate": at(6)}, INVALID), ({"dweight": at(10) + 2}, INVALID),
    ({"dbias": at(10)}, INVALID),
])
def test_conv_bwd_refuses(kw, code):
    a = conv_args(**kw)
    assert tfla.lib().tfla_conv_bwd(ctypes.byref(a), None, 0, None) == code
    assert tfla.tfla_last_error()


def test_conv_bwd_workspace():
    L = tfla.lib()
    n = L.tfla_conv_bwd_workspace_bytes(2, 300, 64, 4, BF16)
    assert n > 0
    for bad in ((0, 300, 64, 4, BF16), (2, 300, 64, 9, BF16), (2, 300, 64, 4, 0x400)):
        assert L.tfla_conv_bwd_workspace_bytes(*bad) == 0
    a = conv_args()
    assert L.tfla_conv_bwd(ctypes.byref(a), at(20), n - 1, None) == OOM
    assert L.tfla_conv_bwd(ctypes.byref(a), at(20) + 16, n, None) == INVALID
    assert L.tfla_conv_bwd(ctypes.byref(a), at(2), n, None) == INVALID     # on top of dy
    assert "workspace overlaps dy" in tfla.tfla_last_error()


def test_null_args():
    L = tfla.lib()
    assert L.tfla_conv_fwd(None, None) == INVALID
    assert L.tfla_conv_bwd(None, None, 0, None) == INVALID


def test_injected_allocation_failure(set_knob):
    set_knob(tfla.KNOB_FAULT_ALLOC, 1)
    a = conv_args()
    assert tfla.lib().tfla_conv_bwd(ctypes.byref(a), None, 0, None) == OOM
    assert "injected" in tfla.tfla_last_error()


def test_python_checks_refuse():
    x, w = torch.zeros(2, 5, 8), torch.zeros(8, 4)
    with pytest.raises(ValueError, match="GPU memory"):
        tfla.conv_forward(x, w)
    with pytest.raises(TypeError):
        tfla.conv_forward(x.half(), w)
    with pytest.raises(ValueError, match="3 dimensions"):
        tfla.conv_forward(x[0], w)
    with pytest.raises(TypeError):
        tfla.conv_forward(None, w)


# ---- scan ------------------------------------------------------------------------------

def scan_args(**kw):
    B, T, D, N, G = 2, 300, 128, 16, 2
    a = blocks.ScanArgs(B=B, T=T, D=D, N=N, G=G, flags=BF16 | blocks.SCAN_SOFTPLUS)
    rows = lambda n, w=D: blocks.Rows(at(n), T * w, w)  # noqa: E731
    a.x, a.dt, a.z, a.y, a.dy = rows(0), rows(1), rows(2), rows(3), rows(4)
    a.bmat, a.cmat, a.dbmat, a.dcmat = rows(5, G * N), rows(6, G * N), rows(7, G * N), rows(8, G * N)
    a.dx, a.ddt, a.dz = rows(9), rows(10), rows(11)
    for i, k in enumerate(("a", "skip", "dt_bias", "state", "lengths", "state_out", "dstate_out", "da", "dskip",
                           "ddt_bias", "dstate")):
        setattr(a, k, at(12 + i))
    return put(a, kw)


SCAN_BOTH = [
    ({"B": 0}, INVALID), ({"T": -1}, INVALID), ({"D": 0}, INVALID), ({"G": 0}, INVALID), ({"G": 3}, INVALID),
    ({"N": 0}, INVALID), ({"N": 65}, UNSUPPORTED), ({"N": 1 << 20}, UNSUPPORTED), ({"flags": 0x200}, INVALID),
    ({"B": 1 << 16, "T": 1 << 15}, UNSUPPORTED), ({"D": 1 << 26}, UNSUPPORTED),
    ({"x.data": None}, INVALID), ({"dt.data": None}, INVALID), ({"bmat.data": None}, INVALID), ({"a": None}, INVALID),
    ({"bmat.data": at(5) + 1}, INVALID), ({"cmat.row": -2}, INVALID), ({"bmat.batch": 1 << 55}, INVALID),
    ({"a": at(12) + 2}, INVALID), ({"state": at(15) + 1}, INVALID), ({"z.row": -1}, INVALID), ({"dt.batch": 1 << 60}, INVALID),
]


@pytest.mark.parametrize("kw,code", SCAN_BOTH + [
    ({"y.data": None}, INVALID), ({"y.row": 127}, INVALID), ({"y.data": at(1)}, INVALID), ({"y.data": at(5)}, INVALID),
    ({"state_out": at(15) + 4}, INVALID), ({"state_out": at(3)}, INVALID),
])
def test_scan_fwd_refuses(kw, code):
    assert tfla.lib().tfla_scan_fwd(ctypes.byref(scan_args(**kw)), None, 0, None) == code
    assert tfla.tfla_last_error()


@pytest.mark.parametrize("kw,code", SCAN_BOTH + [
    ({"dy.data": None}, INVALID), ({"dx.data": None}, INVALID), ({"da": None}, INVALID), ({"dz.data": None}, INVALID),
    ({"z.data": None}, INVALID), ({"dskip": None}, INVALID), ({"dt_bias": None}, INVALID), ({"dx.data": at(4)}, INVALID),
    ({"ddt.data": at(9)}, INVALID), ({"dbmat.data": at(5)}, INVALID), ({"dcmat.row": 31}, INVALID),
    ({"dstate": at(15)}, INVALID), ({"dbmat.data": None}, INVALID),
])
def test_scan_bwd_refuses(kw, code):
    assert tfla.lib().tfla_scan_bwd(ctypes.byref(scan_args(**kw)), None, 0, None) == code
    assert tfla.tfla_last_error()


@pytest.mark.parametrize("B,D,G,fits", [
    (1, (1 << 24), 1, True), (8, (1 << 24), 1, False), (7, (1 << 24), 1, True),
    (1, (1 << 21) - 1, (1 << 21) - 1, True), (1, 1 << 21, 1 << 21, False),   # one channel a group: a block each
    (4, 65 << 13, 1 << 13, True), (128, 65 << 13, 1 << 13, False),           # 65 channels a group: two blocks each
])
def test_scan_blocks_of_channels(B, D, G, fits):
    L = tfla.lib()
    assert (L.tfla_scan_bwd_workspace_bytes(B, 64, D, 4, G, BF16) > 0) == fits
    if not fits:
        assert L.tfla_scan_fwd(ctypes.byref(scan_args(B=B, D=D, G=G)), None, 0, None) == UNSUPPORTED


def test_scan_workspace():
    L = tfla.lib()
    n = L.tfla_scan_bwd_workspace_bytes(2, 300, 128, 16, 2, BF16)
    assert n > 0
    for bad in ((2, 300, 128, 65, 2, BF16), (2, 300, 128, 16, 3, BF16), (0, 300, 128, 16, 2, BF16), (2, 300, 128, 16, 2, 1)):
        assert L.tfla_scan_bwd_workspace_bytes(*bad) == 0 and L.tfla_scan_workspace_bytes(*bad) == 0
    a = scan_args()
    n = L.tfla_scan_bwd_workspace_bytes(2, 300, 128, 16, 2, a.flags)
    assert L.tfla_scan_bwd(ctypes.byref(a), at(30), n - 1, None) == OOM
    assert L.tfla_scan_bwd(ctypes.byref(a), at(30) + 64, n, None) == INVALID
    assert L.tfla_scan_bwd(ctypes.byref(a), at(9), n, None) == INVALID
    assert L.tfla_scan_fwd(None, None, 0, None) == INVALID
    assert L.tfla_scan_bwd(None, None, 0, None) == INVALID


def test_interleaved_views_are_told_apart():
    """Two halves of one row share no element; a byte more and they do."""
    a = scan_args()
    a.dx, a.dz = blocks.Rows(at(40), 300 * 256, 256), blocks.Rows(at(40) + 256, 300 * 256, 256)
    a.T, a.B = 300, 2
    # the checks pass up to the workspace, which is refused as too small
    assert tfla.lib().tfla_scan_bwd(ctypes.byref(a), at(60), 256, None) == OOM
    a.dz = blocks.Rows(at(40) + 254, 300 * 256, 256)
    assert tfla.lib().tfla_scan_bwd(ctypes.byref(a), at(60), 256, None) == INVALID
    assert "overlaps" in tfla.tfla_last_error()


# ---- norm --------------------------------------------------------------------------------

def norm_args(**kw):
    B, T, G, C = 2, 100, 4, 64
    a = blocks.NormArgs(B=B, T=T, G=G, C=C, flags=BF16, act=1, eps=1e-5)
    heads = lambda n: blocks.Heads(at(n), T * G * C, G * C, C)  # noqa: E731
    a.x, a.gate, a.y, a.dy, a.dx, a.dgate = (heads(i) for i in range(6))
    for i, k in enumerate(("weight", "bias", "mean", "rstd", "dweight", "dbias")):
        setattr(a, k, at(10 + i))
    return put(a, kw)


NORM_BOTH = [
    ({"B": 0}, INVALID), ({"T": 0}, INVALID), ({"G": -1}, INVALID), ({"C": 0}, INVALID), ({"flags": 0x1000}, INVALID),
    ({"act": 3}, INVALID), ({"act": -1}, INVALID), ({"B": 1 << 16, "T": 1 << 15}, UNSUPPORTED),
    ({"G": 1 << 13, "C": 1 << 12}, UNSUPPORTED), ({"x.data": None}, INVALID), ({"x.data": at(0) + 1}, INVALID),
    ({"gate.data": at(1) + 1}, INVALID), ({"weight": at(10) + 2}, INVALID), ({"x.group": -1}, INVALID),
    ({"x.group": 1 << 61}, INVALID), ({"mean": at(12) + 1}, INVALID),
]


@pytest.mark.parametrize("kw,code", NORM_BOTH + [
    ({"y.data": None}, INVALID), ({"eps": 0.0}, INVALID), ({"eps": -1.0}, INVALID), ({"eps": float("nan")}, INVALID),
    ({"y.group": 32}, INVALID), ({"y.row": 64}, INVALID), ({"y.data": at(0)}, INVALID), ({"y.data": at(1)}, INVALID),
    ({"mean": at(2)}, INVALID), ({"rstd": at(12)}, INVALID),
])
def test_norm_fwd_refuses(kw, code):
    assert tfla.lib().tfla_norm_fwd(ctypes.byref(norm_args(**kw)), None, 0, None) == code
    assert tfla.tfla_last_error()


@pytest.mark.parametrize("kw,code", NORM_BOTH + [
    ({"dy.data": None}, INVALID), ({"dx.data": None}, INVALID), ({"mean": None}, INVALID), ({"rstd": None}, INVALID),
    ({"dgate.data": None}, INVALID), ({"gate.data": None}, INVALID), ({"dweight": None}, INVALID), ({"bias": None}, INVALID),
    ({"dx.data": at(3)}, INVALID), ({"dgate.data": at(4)}, INVALID), ({"dweight": at(10)}, INVALID),
])
def test_norm_bwd_refuses(kw, code):
    assert tfla.lib().tfla_norm_bwd(ctypes.byref(norm_args(**kw)), None, 0, None) == code
    assert tfla.tfla_last_error()


def test_norm_workspace():
    L = tfla.lib()
    assert L.tfla_norm_bwd_workspace_bytes(2, 100, 4, 64, BF16) > 0
    for bad in ((0, 100, 4, 64, 0), (2, 100, 4, 64, 0x1000), (2, 100, 1 << 13, 1 << 12, 0)):
        assert L.tfla_norm_bwd_workspace_bytes(*bad) == 0 and L.tfla_norm_workspace_bytes(*bad) == 0
    assert L.tfla_norm_fwd(None, None, 0, None) == INVALID
    assert L.tfla_norm_bwd(None, None, 0, None) == INVALID
    n = L.tfla_norm_bwd_workspace_bytes(2, 100, 4, 64, BF16)
    a = norm_args()
    assert L.tfla_norm_bwd(ctypes.byref(a), at(30), n - 1, None) == OOM
    assert L.tfla_norm_bwd(ctypes.byref(a), at(4), n, None) == INVALID


def test_head_major_and_interleaved_heads_are_told_apart():
    """Two outputs interleaved head by head, and one written head-major."""
    a = norm_args()
    a.dx, a.dgate = blocks.Heads(at(40), 100 * 512, 512, 128), blocks.Heads(at(40) + 128, 100 * 512, 512, 128)
    assert tfla.lib().tfla_norm_bwd(ctypes.byref(a), at(60), 0, None) == OOM
    a.dgate = blocks.Heads(at(40) + 126, 100 * 512, 512, 128)
    assert tfla.lib().tfla_norm_bwd(ctypes.byref(a), at(60), 0, None) == INVALID
    a = norm_args()
    a.dx = blocks.Heads(at(40), 100 * 256, 64, 100 * 64)
    assert tfla.lib().tfla_norm_bwd(ctypes.byref(a), at(60), 0, None) == OOM


def test_packed_arguments_match_the_structures():
    for packed, fields in ((blocks._CONV, blocks.ConvArgs), (blocks._SCAN, blocks.ScanArgs), (blocks._NORM, blocks.NormArgs)):
        assert packed.size == ctypes.sizeof(fields)
        # every value lands in the field of its place
        flat = []

        def walk(s, base):
            for name, kind in s._fields_:
                off = base + getattr(s, name).offset
                if issubclass(kind, ctypes.Structure):
                    walk(kind, off)
                else:
                    flat.append((off, kind))

        walk(fields, 0)
        values = [float(i) if k is ctypes.c_float else i + 1 for i, (_, k) in enumerate(flat)]
        raw = packed.pack(*values)
        for v, (off, kind) in zip(values, flat):
            assert kind.from_buffer_copy(raw, off).value == v


class _OnGpu:
    """What the stream rule asks of a tensor."""
    is_cuda = True

    def get_device(self):
        return 0


def test_a_given_stream_becomes_the_current_one(monkeypatch):
    """All that a call allocates and launches follows: see tests/test_gpu_streams.py for the memory itself."""
    import contextlib
    entered = []

    @contextlib.contextmanager
    def on(s):
        entered.append(s)
        yield

    class Stream:
        def __init__(self, handle, device_index=0):
            self.cuda_stream, self.device_index, self.device = handle, device_index, f"cuda:{device_index}"

    monkeypatch.setattr(blocks, "_raw_stream", lambda dev: 0x50)
    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda dev: Stream(0))
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device: Stream(handle, device))
    x, side = _OnGpu(), Stream(0x90)
    for given, handle in ((None, None), (0x50, None), (Stream(0x50), None), (side, 0x90), (0x90, 0x90), (0, 0), (1, 0)):
        with blocks._current(given, x):
            assert [s.cuda_stream for s in entered] == ([] if handle is None else [handle])
        entered.clear()
    with pytest.raises(ValueError, match="stream is on cuda:1"):
        blocks._current(Stream(0x90, 1), x)
    with pytest.raises(ValueError, match="GPU memory"):
        tfla.conv_forward(torch.zeros(2, 5, 8), torch.zeros(8, 4), stream=side)
    assert not entered


def test_first_use_from_two_threads(monkeypatch):
    """A thread that comes while another is still filling in the entry points finds none, or all."""
    import threading
    real, half, go = tfla.lib(), threading.Event(), threading.Event()

    class Slow:
        def __getattr__(self, name):
            if name == "tfla_scan_bwd":
                half.set()
                go.wait(20)
            return getattr(real, name)

    monkeypatch.setattr(blocks, "_fn", {})
    monkeypatch.setattr(tfla, "_lib", None)
    first = threading.Thread(target=blocks.bind, args=(Slow(),))
    first.start()
    try:
        assert half.wait(20)
        assert blocks._entry("tfla_norm_bwd").restype is ctypes.c_int
        assert blocks._fn["tfla_norm_fwd"] and blocks._fn["tfla_conv_fwd"]
    finally:
        go.set()
        first.join()
    assert len(blocks._fn) == 11
