"""Refusals of rotary positions, the gated linear recurrence of channels and
the residual sum with a norm, on the CPU: bad arguments are answered by the
host checks, before any HIP call.  Pointers are fake aligned device addresses
that no check follows."""
import ctypes

import pytest
import torch

tfla = pytest.importorskip("mlstm_sequence_amd.tfla")
from mlstm_sequence_amd import edges  # noqa: E402
from mlstm_sequence_amd.blocks import Heads, Rows  # noqa: E402
from test_abi_blocks import at, put  # noqa: E402

BF16 = 0x100
INVALID, UNSUPPORTED, OOM = 1, 2, 4


@pytest.fixture(scope="module", autouse=True)
def _built():
    import os
    if not os.path.exists(tfla.LIB_PATH):
        pytest.skip("libtfla.so not built")
    tfla.lib()


# ---- rotary positions ------------------------------------------------------------------

def rotary_args(**kw):
    B, T, H, Hk, C = 2, 30, 4, 2, 64
    a = edges.RotaryArgs(B=B, T=T, H=H, Hk=Hk, C=C, R=32, flags=BF16, scale=1.0)
    heads = lambda p, n: Heads(p, T * n * C, n * C, C)  # noqa: E731
    a.q, a.k, a.q_out, a.k_out = heads(at(0), H), heads(at(1), Hk), heads(at(2), H), heads(at(3), Hk)
    a.freqs, a.positions, a.positions_batch, a.lengths = at(4), at(5), T, at(6)
    return put(a, kw)


@pytest.mark.parametrize("fn", ["tfla_rotary_fwd", "tfla_rotary_bwd"])
@pytest.mark.parametrize("kw,code", [
    ({"B": 0}, INVALID), ({"T": 0}, INVALID), ({"H": 0}, INVALID), ({"Hk": -1}, INVALID), ({"C": 0}, INVALID),
    ({"R": 31}, INVALID), ({"R": -2}, INVALID), ({"R": 66}, INVALID), ({"C": 1025}, UNSUPPORTED),
    ({"B": 1 << 16, "T": 1 << 15}, UNSUPPORTED), ({"H": 1 << 18}, UNSUPPORTED), ({"H": 0x7fffffff}, UNSUPPORTED),
    ({"flags": 0x2000}, INVALID), ({"flags": 0x8000}, INVALID),
    ({"q.data": None}, INVALID), ({"k.data": None}, INVALID), ({"q_out.data": None}, INVALID), ({"k_out.data": None}, INVALID),
    ({"freqs": None}, INVALID), ({"freqs": at(4) + 4}, INVALID), ({"q.data": at(0) + 1}, INVALID), ({"lengths": at(6) + 2}, INVALID),
    ({"positions": at(5) + 2}, INVALID), ({"positions_batch": -1}, INVALID), ({"positions_batch": 1 << 61}, INVALID),
    ({"start": at(7)}, INVALID), ({"start": at(7) + 1, "positions": None}, INVALID),
    ({"q.group": -64}, INVALID), ({"q.row": 1 << 62}, INVALID), ({"k.batch": 1 << 47}, INVALID),
    ({"q_out.group": 32}, INVALID), ({"q_out.row": 64}, INVALID), ({"q_out.batch": 0}, INVALID),
    ({"q_out.data": at(0) + 2}, INVALID), ({"q_out.data": at(1)}, INVALID), ({"k_out.data": at(0)}, INVALID),
    ({"k_out.data": at(2) + 128}, INVALID), ({"q_out.data": at(4)}, INVALID), ({"k_out.data": at(5)}, INVALID),
    ({"q_out.data": at(6) - 16}, INVALID),
    ({"k": Heads(at(0), 30 * 256, 256, 64), "q_out.data": at(0)}, INVALID),   # in place over q, which k reads too
    ({"q_out": Heads(at(0), 30 * 256, 64, 30 * 64)}, INVALID),                 # q's memory in another order
])
def test_rotary_refuses(fn, kw, code):
    assert getattr(tfla.lib(), fn)(ctypes.byref(rotary_args(**kw)), None) == code
    assert tfla.tfla_last_error()


def test_rotary_start_overlap():
    a = rotary_args(positions=None, start=at(2))
    assert tfla.lib().tfla_rotary_fwd(ctypes.byref(a), None) == INVALID
    assert "overlaps start" in tfla.tfla_last_error()


# ---- gated linear recurrence of channels ------------------------------------------------

def diag_args(**kw):
    B, T, D = 2, 300, 64
    a = edges.DiagArgs(B=B, T=T, D=D, kind=2, flags=BF16)
    rows = lambda p: Rows(p, T * D, D)  # noqa: E731
    a.x, a.fgate, a.igate, a.y = rows(at(0)), rows(at(1)), rows(at(2)), rows(at(3))
    a.dy, a.dx, a.dfgate, a.digate = rows(at(4)), rows(at(5)), rows(at(6)), rows(at(7))
    a.decay, a.lengths, a.state, a.state_out, a.starts = at(8), at(9), at(10), at(11), at(12)
    a.dstate_out, a.ddecay, a.dstate = at(13), at(14), at(15)
    return put(a, kw)


DIAG_BOTH = [
    ({"B": 0}, INVALID), ({"T": -1}, INVALID), ({"D": 0}, INVALID), ({"kind": 3}, INVALID), ({"kind": -1}, INVALID),
    ({"flags": 0x1000}, INVALID), ({"B": 1 << 16, "T": 1 << 15}, UNSUPPORTED), ({"D": (1 << 24) + 1}, UNSUPPORTED),
    ({"x.data": None}, INVALID), ({"fgate.data": None}, INVALID), ({"igate.data": None}, INVALID),
    ({"igate.data": None, "kind": 1}, INVALID), ({"decay": None}, INVALID), ({"decay": at(8) + 2}, INVALID),
    ({"lengths": at(9) + 1}, INVALID), ({"x.data": at(0) + 1}, INVALID), ({"fgate.row": -1}, INVALID),
    ({"igate.batch": 1 << 50}, INVALID), ({"x.row": 1 << 62}, INVALID), ({"starts": at(12) + 2}, INVALID),
]


@pytest.mark.parametrize("kw,code", DIAG_BOTH + [
    ({"y.data": None}, INVALID), ({"y.row": 63}, INVALID), ({"y.batch": 0}, INVALID), ({"y.data": at(0)}, INVALID),
    ({"y.data": at(2)}, INVALID), ({"state": at(10) + 1}, INVALID), ({"state_out": at(11) + 2}, INVALID),
    ({"state_out": at(10) + 4}, INVALID), ({"state_out": at(3)}, INVALID), ({"starts": at(10)}, INVALID),
    ({"starts": at(11) - 256}, INVALID), ({"starts": at(3) - 1536 + 4}, INVALID), ({"y.data": at(9) - 2}, INVALID),
    ({"y.data": at(8)}, INVALID),
])
def test_diag_fwd_refuses(kw, code):
    assert tfla.lib().tfla_diag_fwd(ctypes.byref(diag_args(**kw)), None, 0, None) == code
    assert tfla.tfla_last_error()


@pytest.mark.parametrize("kw,code", DIAG_BOTH + [
    ({"starts": None}, INVALID), ({"dy.data": None}, INVALID), ({"dx.data": None}, INVALID), ({"dfgate.data": None}, INVALID),
    ({"digate.data": None}, INVALID), ({"ddecay": None}, INVALID), ({"ddecay": at(14) + 2}, INVALID),
    ({"dstate": at(15) + 1}, INVALID), ({"dstate_out": at(13) + 1}, INVALID), ({"dx.row": 32}, INVALID),
    ({"dx.data": at(4)}, INVALID), ({"dfgate.data": at(5)}, INVALID), ({"digate.data": at(6)}, INVALID),
    ({"dfgate.data": at(12)}, INVALID), ({"dstate": at(13)}, INVALID), ({"ddecay": at(8)}, INVALID),
])
def test_diag_bwd_refuses(kw, code):
    a = diag_args(**kw)
    assert tfla.lib().tfla_diag_bwd(ctypes.byref(a), at(30), 1 << 30, None) == code
    assert tfla.tfla_last_error()


def test_diag_workspaces():
    L = tfla.lib()
    for f in (L.tfla_diag_workspace_bytes, L.tfla_diag_bwd_workspace_bytes):
        for bad in ((0, 300, 64, 0, BF16), (2, 300, 64, 3, BF16), (2, 300, 64, 0, 0x400), (2, 300, (1 << 24) + 1, 0, 0)):
            assert f(*bad) == 0
    n = L.tfla_diag_bwd_workspace_bytes(2, 300, 64, 2, BF16)
    assert n > 0
    a = diag_args()
    assert L.tfla_diag_bwd(ctypes.byref(a), at(30), n - 1, None) == OOM
    assert L.tfla_diag_bwd(ctypes.byref(a), at(30) + 16, n, None) == INVALID
    assert L.tfla_diag_bwd(ctypes.byref(a), at(4), n, None) == INVALID
    assert "workspace overlaps dy" in tfla.tfla_last_error()
    n = L.tfla_diag_workspace_bytes(1, 65536, 64, 0, BF16)
    if n:
        a = diag_args(B=1, T=65536, kind=0, starts=None, lengths=None)
        assert L.tfla_diag_fwd(ctypes.byref(a), at(30), n - 1, None) == OOM


def test_diag_fields_that_a_kind_does_not_have_are_not_looked_at():
    """They would be refused otherwise; the call gets as far as its missing workspace."""
    a = diag_args(kind=1, decay=at(8) + 1, ddecay=at(14) + 1)
    L, need = tfla.lib(), tfla.lib().tfla_diag_bwd_workspace_bytes(2, 300, 64, 1, BF16)
    if need:
        assert L.tfla_diag_bwd(ctypes.byref(a), at(30), need - 1, None) == OOM
    a.x.row = -1
    assert L.tfla_diag_bwd(ctypes.byref(a), at(30), 1 << 30, None) == INVALID
    assert "x: strides" in tfla.tfla_last_error()


# ---- residual sum with a norm --------------------------------------------------------------

def addnorm_args(**kw):
    B, T, C = 2, 30, 64
    a = edges.AddNormArgs(B=B, T=T, C=C, flags=BF16 | 0x10000, eps=1e-5)
    rows = lambda p: Rows(p, T * C, C)  # noqa: E731
    a.x, a.residual, a.y, a.total = rows(at(0)), rows(at(1)), rows(at(2)), rows(at(3))
    a.dy, a.dtotal, a.dx, a.dresidual = rows(at(4)), rows(at(5)), rows(at(6)), rows(at(7))
    a.weight, a.bias, a.dweight, a.dbias = at(8), at(9), at(10), at(11)
    return put(a, kw)


ADDNORM_BOTH = [
    ({"B": 0}, INVALID), ({"T": 0}, INVALID), ({"C": -4}, INVALID), ({"flags": 0x4000}, INVALID), ({"flags": 0x20000}, INVALID),
    ({"B": 1 << 16, "T": 1 << 15}, UNSUPPORTED), ({"C": (1 << 24) + 1}, UNSUPPORTED), ({"eps": 0.0}, INVALID),
    ({"eps": -1.0}, INVALID), ({"eps": float("nan")}, INVALID), ({"weight": at(8) + 2}, INVALID),
    ({"total.data": at(3) + 2}, INVALID), ({"total.row": -1}, INVALID),
]


@pytest.mark.parametrize("kw,code", ADDNORM_BOTH + [
    ({"x.data": None}, INVALID), ({"y.data": None}, INVALID), ({"total.data": None}, INVALID), ({"residual.data": None}, INVALID),
    ({"bias": at(9) + 1}, INVALID), ({"residual.data": at(1) + 2}, INVALID), ({"y.row": 32}, INVALID),
    ({"y.data": at(0)}, INVALID), ({"y.data": at(1)}, INVALID), ({"y.data": at(3)}, INVALID), ({"total.data": at(0)}, INVALID),
    ({"total.data": at(1) + 4}, INVALID), ({"total": Rows(at(1), 30 * 64, 128)}, INVALID), ({"y.data": at(8)}, INVALID),
    ({"x.row": 1 << 62}, INVALID),
])
def test_addnorm_fwd_refuses(kw, code):
    assert tfla.lib().tfla_addnorm_fwd(ctypes.byref(addnorm_args(**kw)), None) == code
    assert tfla.tfla_last_error()


@pytest.mark.parametrize("kw,code", ADDNORM_BOTH + [
    ({"dy.data": None}, INVALID), ({"dx.data": None}, INVALID), ({"total.data": None}, INVALID), ({"dtotal.data": at(5) + 2}, INVALID),
    ({"flags": BF16}, INVALID), ({"dx.data": at(4)}, INVALID), ({"dx.data": at(3)}, INVALID), ({"dresidual.data": at(5)}, INVALID),
    ({"dresidual.data": at(6)}, INVALID), ({"dweight": at(8)}, INVALID), ({"dbias": at(10) + 4}, INVALID),
    ({"dbias": at(11) + 2}, INVALID), ({"dx.row": 63}, INVALID),
])
def test_addnorm_bwd_refuses(kw, code):
    assert tfla.lib().tfla_addnorm_bwd(ctypes.byref(addnorm_args(**kw)), at(30), 1 << 30, None) == code
    assert tfla.tfla_last_error()


def test_addnorm_workspace():
    L = tfla.lib()
    n = L.tfla_addnorm_bwd_workspace_bytes(2, 30, 64, BF16 | 0x10000)
    assert n > 0
    for bad in ((0, 30, 64, BF16), (2, 30, 64, 0x4000), (2, 30, (1 << 24) + 1, 0)):
        assert L.tfla_addnorm_bwd_workspace_bytes(*bad) == 0
    a = addnorm_args()
    assert L.tfla_addnorm_bwd(ctypes.byref(a), at(30), n - 1, None) == OOM
    assert L.tfla_addnorm_bwd(ctypes.byref(a), at(30) + 8, n, None) == INVALID
    assert L.tfla_addnorm_bwd(ctypes.byref(a), at(3), n, None) == INVALID
    assert "workspace overlaps total" in tfla.tfla_last_error()


# ---- all of them ------------------------------------------------------------------------------

def test_null_args():
    L = tfla.lib()
    for f in (L.tfla_rotary_fwd, L.tfla_rotary_bwd, L.tfla_addnorm_fwd):
        assert f(None, None) == INVALID
    for f in (L.tfla_diag_fwd, L.tfla_diag_bwd, L.tfla_addnorm_bwd):
        assert f(None, None, 0, None) == INVALID


def test_injected_allocation_failure(set_knob):
    set_knob(tfla.KNOB_FAULT_ALLOC, 1)
    for f, a in ((tfla.lib().tfla_diag_bwd, diag_args()), (tfla.lib().tfla_addnorm_bwd, addnorm_args())):
        assert f(ctypes.byref(a), None, 0, None) == OOM
        assert "injected" in tfla.tfla_last_error()


def test_packed_arguments_match_the_structures():
    for packed, fields in ((edges._ROTARY, edges.RotaryArgs), (edges._DIAG, edges.DiagArgs), (edges._ADDNORM, edges.AddNormArgs)):
        assert packed.size == ctypes.sizeof(fields)
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


def test_structures_match_the_header(tmp_path):
    """Sizes and last offsets as a C compiler sees them."""
    import os
    import subprocess
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    last = {"rotary": ("k_out", edges.RotaryArgs), "diag": ("dstate", edges.DiagArgs), "addnorm": ("dbias", edges.AddNormArgs)}
    body = "".join(f'printf("%zu %zu\\n", sizeof(tfla_{n}_args), offsetof(tfla_{n}_args, {f}));' for n, (f, _) in last.items())
    src = tmp_path / "sizes.c"
    src.write_text('#include <stdio.h>\n#include "tfla.h"\nint main(void) {' + body + f'printf("%d\\n", TFLA_DIAG_CHUNK); return 0; }}')
    subprocess.run(["gcc", "-I", os.path.join(root, "include"), str(src), "-o", str(tmp_path / "sizes")], check=True)
    got = subprocess.run([str(tmp_path / "sizes")], capture_output=True, text=True, check=True).stdout.split()
    want = [str(v) for f, c in last.values() for v in (ctypes.sizeof(c), getattr(c, f).offset)] + [str(tfla.DIAG_CHUNK)]
    assert got == want


def test_python_checks_refuse():
    x, g, q = torch.zeros(2, 5, 8), torch.zeros(2, 5, 8), torch.zeros(2, 5, 2, 8)
    f = torch.zeros(2, dtype=torch.float64)
    for call in (lambda: tfla.diag_forward(x, g), lambda: tfla.rotary_forward(q, None, f), lambda: tfla.addnorm_forward(x),
                 lambda: tfla.addnorm_backward(x, x)):
        with pytest.raises(ValueError, match="GPU memory"):
            call()
    for call in (lambda: tfla.diag_forward(x.half(), g), lambda: tfla.rotary_forward(None, None, f),
                 lambda: tfla.addnorm_forward(x.double())):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: tfla.diag_forward(x[0], g), lambda: tfla.rotary_forward(x, None, f), lambda: tfla.addnorm_forward(q)):
        with pytest.raises(ValueError, match="dimensions"):
            call()
