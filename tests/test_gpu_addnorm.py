"""Residual sum with a layer or RMS norm against the 64-bit reference.

Error bounds as in the group norm's tests, with U half a step of fp32, n = C
values of a row, A their mean magnitude, N = n + 60, and a sum t = x + residual
that is itself off by U |t|:
  m       (N + 2) U A
  s^2     2 N U s^2 + 4 s (N + 2) U A
  rstd    half of that over s^2 + eps, and 4 U, relative
and through th and the gradient's formula term by term (RMS: m = 0 exactly,
s^2 the mean square, (N + 4) U relative)."""
import numpy as np
import pytest
import torch

from blocks_helpers import HALF, U, as_view, randn, within
from mlstm_sequence_amd import tfla
from oracle import edges as O

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
NAN = float("nan")
EPS = 1e-5
TYPES = [(BF, BF), (BF, F32), (F32, F32)]   # activations, stream


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    tfla.lib()


def statistics(t, rms, extra):
    """(m, r, error of m, relative error of r); extra: of the values, relative, in U"""
    n = t.shape[-1]
    N = (n + 60 + extra) * U
    A = np.abs(t).mean(-1, keepdims=True)
    m = np.zeros_like(A) if rms else t.mean(-1, keepdims=True)
    var = ((t - m) ** 2).mean(-1, keepdims=True)
    em = np.zeros_like(A) if rms else N * A
    evar = 2 * N * var + 4 * np.sqrt(var) * (em + extra * U * A) + em ** 2
    return m, 1.0 / np.sqrt(var + EPS), em, 0.5 * evar / (var + EPS) + 4 * U


def check(act, stream, B, T, C, rms=False, residual=True, affine=True, bias=True, view="plain", scale=2.0, shift=0.5, behind=True):
    print("addnorm", act, stream, B, T, C, rms, residual, affine, bias, view, scale, shift, behind, flush=True)
    rng = np.random.default_rng(T + 7 * C)
    tx, x = randn(rng, (B, T, C), act, scale, shift)
    tr, r = randn(rng, (B, T, C), stream, scale) if residual else (None, None)
    tw, w = randn(rng, (C,), F32, 0.3, 1.0) if affine else (None, None)
    tb, b = randn(rng, (C,), F32, 0.3) if bias else (None, None)
    cu = lambda t: None if t is None else t.cuda()  # noqa: E731
    new = lambda dt: as_view(torch.full((B, T, C), NAN, dtype=dt), view)  # noqa: E731
    y, total = tfla.addnorm_forward(as_view(tx, view), as_view(tr, view), cu(tw), cu(tb), eps=EPS, rms=rms, y=new(act),
                                    total=new(stream) if residual else None)
    torch.cuda.synchronize()
    wy, wt = O.addnorm(x, r, w, b, EPS, rms)
    W, Bb = 1.0 if w is None else np.abs(w), 0.0 if b is None else np.abs(b)
    m, rs, em, er = statistics(wt, rms, 2)
    th = (wt - m) * rs
    eth = rs * (3 * U * (np.abs(wt) + np.abs(m)) + em) + np.abs(th) * er
    within("y", y, wy, HALF[act] * np.abs(wy) + W * eth + 4 * U * (np.abs(th) * W + Bb) + 1e-37)
    if residual:
        # the sum in fp32, then rounded to the stream's type
        within("total", total, wt, (HALF[stream] + U * 1.01) * np.abs(wt) + 1e-37)
    else:
        assert total is None

    # backward from the sum as it is kept
    kept = total if residual else as_view(tx, view)
    t64 = kept.double().cpu().numpy()
    tg, dy = randn(rng, (B, T, C), act)
    te, de = randn(rng, (B, T, C), kept.dtype) if behind else (None, None)
    two = kept.dtype != act
    dx, dr, dw, db = tfla.addnorm_backward(kept, as_view(tg, view), cu(tw), bias=bias, eps=EPS, rms=rms, dtotal=as_view(te, view),
                                           dx=new(act), dresidual=new(kept.dtype) if two else None)
    torch.cuda.synchronize()
    wdt, wdw, wdb = O.addnorm_grads(t64, dy, w, EPS, rms, de)
    m, rs, em, er = statistics(t64, rms, 0)
    th = (t64 - m) * rs
    eth = rs * (2 * U * (np.abs(t64) + np.abs(m)) + em) + np.abs(th) * er
    v = dy * (1.0 if w is None else w)
    ev, N = U * np.abs(v), (C + 60) * U
    mv, mvt = v.mean(-1, keepdims=True), (v * th).mean(-1, keepdims=True)
    emv = N * np.abs(v).mean(-1, keepdims=True)
    emvt = (ev * np.abs(th) + np.abs(v) * eth).mean(-1, keepdims=True) + N * np.abs(v * th).mean(-1, keepdims=True)
    if rms:
        mv, emv = np.zeros_like(mv), np.zeros_like(emv)
    edt = rs * (ev + emv + np.abs(th) * emvt + eth * np.abs(mvt)) + (2 * er + 8 * U) * rs * (np.abs(v) + np.abs(mv) + np.abs(th * mvt))
    edt = edt + U * (np.abs(wdt) + (0.0 if de is None else np.abs(de)))
    within("dx", dx, wdt, HALF[act] * np.abs(wdt) + edt + 1e-37)
    if two:
        within("dresidual", dr, wdt, HALF[kept.dtype] * np.abs(wdt) + edt + 1e-37)
    else:
        assert dr is dx
    rows = (B * T + 60) * U
    if affine:
        within("dweight", dw, wdw, (np.abs(dy) * eth).sum((0, 1)) + rows * np.abs(dy * th).sum((0, 1)) + 1e-37)
    else:
        assert dw is None
    if bias:
        within("dbias", db, wdb, rows * np.abs(dy).sum((0, 1)) + 1e-37)
    else:
        assert db is None


@pytest.mark.parametrize("act,stream", TYPES)
@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("C", [1, 2, 3, 7, 8, 40, 64, 65, 128, 200, 256, 512, 520, 1000, 1001, 1024, 2048, 4096, 5000])
def test_widths(act, stream, rms, C):
    check(act, stream, 2, 5, C, rms)


@pytest.mark.parametrize("act,stream", TYPES)
@pytest.mark.parametrize("C", [8192, 8193, 16384, 16392, 20000])
def test_wide_rows(act, stream, C):
    check(act, stream, 1, 3, C)
    check(act, stream, 1, 2, C, rms=True, bias=False)


@pytest.mark.parametrize("act,stream", TYPES)
@pytest.mark.parametrize("view", ["half", "odd", "wide", "time"])
def test_views(act, stream, view):
    check(act, stream, 3, 11, 72, view=view)
    check(act, stream, 2, 5, 640, rms=True, view=view)


@pytest.mark.parametrize("act,stream", TYPES)
@pytest.mark.parametrize("T", [1, 2, 63, 64, 65, 700])
def test_rows(act, stream, T):
    check(act, stream, 3, T, 96)


@pytest.mark.parametrize("act,stream", TYPES)
@pytest.mark.parametrize("rms", [False, True])
def test_parts_left_out(act, stream, rms):
    check(act, stream, 2, 30, 128, rms, affine=False, bias=False)
    check(act, stream, 2, 30, 128, rms, affine=False)
    check(act, stream, 2, 30, 128, rms, bias=False, behind=False)
    check(act, act, 2, 30, 128, rms, residual=False)


@pytest.mark.parametrize("act,stream", TYPES)
def test_large_means(act, stream):
    """A mean far above the spread: the second pass subtracts it first."""
    check(act, stream, 2, 9, 512, scale=0.5, shift=40.0)


def test_constant_rows():
    """No spread at all: rstd is 1 / sqrt(eps), y the bias."""
    x, r = torch.full((1, 3, 64), 2.0, device="cuda"), torch.full((1, 3, 64), -0.5, device="cuda")
    w, b = torch.randn(64, device="cuda"), torch.randn(64, device="cuda")
    y, t = tfla.addnorm_forward(x, r, w, b)
    dx, _, dw, db = tfla.addnorm_backward(t, torch.ones_like(x), w, bias=True)
    z, _ = tfla.addnorm_forward(torch.zeros_like(x), None, w, None, rms=True)
    torch.cuda.synchronize()
    assert torch.equal(y, b.expand_as(y)) and bool((t == 1.5).all()) and bool((dw == 0).all()) and bool((db == 3).all())
    assert bool(torch.isfinite(dx).all()) and bool((z == 0).all())


def test_nan_stays_in_its_row():
    x, r = torch.randn(2, 6, 96, device="cuda"), torch.randn(2, 6, 96, device="cuda")
    want, _ = tfla.addnorm_forward(x, r)
    x[1, 3, 5] = NAN
    x[0, 2, 7] = float("inf")
    y, _ = tfla.addnorm_forward(x, r)
    torch.cuda.synchronize()
    bad = torch.zeros(2, 6, dtype=torch.bool, device="cuda")
    bad[1, 3] = bad[0, 2] = True
    assert torch.equal(y[~bad], want[~bad]) and bool(torch.isnan(y[1, 3]).all()) and bool(torch.isnan(y[0, 2, 7]))


@pytest.mark.parametrize("act,stream", TYPES)
@pytest.mark.parametrize("C", [96, 1024, 1001, 20000])
def test_stream_updated_in_place(act, stream, C):
    x, r = torch.randn(2, 7, C, device="cuda").to(act), torch.randn(2, 7, C, device="cuda").to(stream)
    wy, wt = tfla.addnorm_forward(x, r, rms=True)
    y, t = tfla.addnorm_forward(x, r, rms=True, total=r)
    torch.cuda.synchronize()
    assert t is r and torch.equal(y, wy) and torch.equal(r, wt)


def test_broadcast_inputs():
    """A row that every token adds (strides of 0)."""
    x, r = torch.randn(2, 9, 64, device="cuda"), torch.randn(64, device="cuda").expand(2, 9, 64)
    got, want = tfla.addnorm_forward(x, r), tfla.addnorm_forward(x, r.contiguous())
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_refusals_on_tensors():
    x, r, w = torch.randn(2, 10, 32, device="cuda").to(BF), torch.randn(2, 10, 32, device="cuda"), torch.randn(32, device="cuda")
    for bad in (dict(residual=r.double()), dict(residual=r[:1]), dict(weight=w[:8]), dict(weight=w.to(BF)), dict(bias=w[None]),
                dict(total=x), dict(residual=None, total=r), dict(y=x), dict(y=r), dict(eps=0.0), dict(x=x.transpose(1, 2)),
                dict(total=r[:, :1].expand_as(r))):
        kw = dict(x=x, residual=r, weight=w)
        kw.update(bad)
        with pytest.raises((TypeError, ValueError, tfla.TflaError)):
            tfla.addnorm_forward(**kw)
    for bad in (dict(total=r.to(torch.float16)), dict(dy=x[:, :4]), dict(dtotal=x), dict(dx=x), dict(weight=w[:4]),
                dict(total=x, dresidual=torch.empty_like(x)), dict(workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))):
        kw = dict(total=r, dy=x, weight=w)
        kw.update(bad)
        with pytest.raises((TypeError, ValueError, tfla.TflaError)):
            tfla.addnorm_backward(**kw)


def test_stream_workspace_and_repeat():
    x, r, w, dy = (torch.randn(3, 333, 264, device="cuda") for _ in range(4))
    w = w[0, 0].contiguous()

    def step(**k):
        y, t = tfla.addnorm_forward(x, r, w, **{n: v for n, v in k.items() if n != "workspace"})
        return [y, t, *tfla.addnorm_backward(t, dy, w, bias=True, dtotal=r, **k)]

    want = step()
    ws = torch.empty(tfla.lib().tfla_addnorm_bwd_workspace_bytes(3, 333, 264, 0), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        a = step()
    b, c = step(workspace=ws), step(stream=side)
    torch.cuda.synchronize()
    for got in (a, b, c):
        assert all(torch.equal(p, q) for p, q in zip(got, want))


def test_captured_and_replayed():
    x, r, dy = (torch.randn(2, 40, 512, device="cuda").to(BF) for _ in range(3))
    w = torch.randn(512, device="cuda")

    def step():
        y, t = tfla.addnorm_forward(x, r, w)
        return [y, t, *tfla.addnorm_backward(t, dy, w, bias=True, dtotal=r)]

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(3):
        x.copy_(torch.randn_like(x))
        dy.copy_(torch.randn_like(dy))
        graph.replay()
        torch.cuda.synchronize()
        want = step()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, want))


def test_offsets_beyond_32_bits():
    far = (1 << 32) + 128
    view, out = (torch.as_strided(torch.empty(far + 9 * 128, dtype=BF, device="cuda"), (2, 9, 128), (far, 128, 1)) for _ in range(2))
    x, w = torch.randn(2, 9, 128, device="cuda").to(BF), torch.randn(128, device="cuda")
    view.copy_(x)
    got, want = tfla.addnorm_forward(view, view, w, y=out), tfla.addnorm_forward(x, x, w)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    got, want = tfla.addnorm_backward(view, view, w, dx=out), tfla.addnorm_backward(x, x, w)
    assert torch.equal(got[0], want[0]) and torch.equal(got[2], want[2])
    torch.cuda.synchronize()


@pytest.mark.parametrize("act,stream", TYPES)
def test_many_rows(act, stream):
    """More rows than workgroups take at once, and parts of the weights' gradients that add up many of them."""
    check(act, stream, 3, 7001, 40, rms=True)
    check(act, stream, 1, 3001, 520)


@pytest.mark.parametrize("act,stream", TYPES)
@pytest.mark.parametrize("C", [9, 41, 521, 2047])
def test_many_rows_of_odd_widths(act, stream, C):
    check(act, stream, 2, 1703, C)


@pytest.mark.parametrize("act,stream", TYPES)
@pytest.mark.parametrize("C", [8, 40, 382, 4096, 5761])
@pytest.mark.parametrize("T", [1, 4, 8, 9])
def test_few_rows(act, stream, T, C):
    """One workgroup for all rows, and more."""
    check(act, stream, 1, T, C)
    check(act, stream, 1, T, C, bias=False)
    check(act, stream, 1, T, C, affine=False)


@pytest.mark.parametrize("act,stream", TYPES)
@pytest.mark.parametrize("C", [3, 8, 13, 269, 1025])
def test_what_lies_between_rows(act, stream, C):
    """Columns beside the rows: NaN read from there would show, and what lies there stays."""
    B, T, L, R = 2, 37, 3, 5
    g = torch.Generator().manual_seed(C)

    def inside(dt, fill):
        big = torch.full((B, T, L + C + R), fill, device="cuda", dtype=dt)
        return big, big[..., L:L + C]

    def data(dt):
        big, v = inside(dt, NAN)
        v.copy_(torch.randn(B, T, C, generator=g))
        return v

    x, r, dy, de, w = data(act), data(stream), data(act), data(stream), torch.randn(C, generator=g).cuda()
    (by, y), (bt, total), (bx, dx) = (inside(dt, 7.0) for dt in (act, stream, act))
    br, dr = inside(stream, 7.0) if act != stream else (None, None)
    tfla.addnorm_forward(x, r, w, y=y, total=total)
    _, _, dw, _ = tfla.addnorm_backward(total, dy, w, dtotal=de, dx=dx, dresidual=dr)
    torch.cuda.synchronize()
    for out in (y, total, dx, dw) + ((dr,) if br is not None else ()):
        assert torch.isfinite(out).all() and not bool((out == 7).all(-1).any())   # read within the rows, all of them written
    for b in (by, bt, bx) + ((br,) if br is not None else ()):
        assert bool((b[..., :L] == 7).all()) and bool((b[..., L + C:] == 7).all())


def test_a_call_that_streams():
    """Large enough for loads past the caches; against the same rows in two smaller calls."""
    B, T, C = 2, 20000, 2048
    t, dy, dt = (torch.randn(B, T, C, device="cuda").to(BF) for _ in range(3))
    w = torch.randn(C, device="cuda")
    dx, _, dw, db = tfla.addnorm_backward(t, dy, w, bias=True, dtotal=dt)
    parts = [tfla.addnorm_backward(t[:, a:b], dy[:, a:b], w, bias=True, dtotal=dt[:, a:b]) for a, b in ((0, 3000), (3000, 20000))]
    torch.cuda.synchronize()
    assert torch.equal(dx, torch.cat([p[0] for p in parts], 1))
    mag = dy.double().abs()
    # sums of 40000 terms in two orders; |th| is at most 6 here
    assert bool(((dw - sum(p[2] for p in parts)).abs() <= 2 * 40100 * U * 6 * mag.sum((0, 1))).all())
    assert bool(((db - sum(p[3] for p in parts)).abs() <= 2 * 40100 * U * mag.sum((0, 1))).all())


@pytest.mark.parametrize("act,stream", TYPES)
@pytest.mark.parametrize("B,T,C", [(2, 1100, 2560), (2, 1100, 4096), (3, 700, 4099), (3, 700, 5120), (2, 600, 8192), (2, 600, 8199),
                                   (2, 560, 16384)])
def test_many_wide_rows(act, stream, B, T, C):
    """Rows of several waves, more of them than workgroups take at once in either direction."""
    check(act, stream, B, T, C, rms=C == 5120)


@pytest.mark.parametrize("act,stream", TYPES)
@pytest.mark.parametrize("C", [4096, 5120, 5125, 10000])
def test_wide_calls_that_stream(act, stream, C):
    """Wide rows in calls large enough for loads past the caches, against the same rows in calls that are not."""
    T = (36 << 20) // C                                  # 8 to 16 bytes an element are read and written: above 256 MiB
    t, dt = (torch.randn(1, T, C, device="cuda").to(stream) for _ in range(2))
    dy, w = torch.randn(1, T, C, device="cuda").to(act), torch.randn(C, device="cuda")
    dx, dr, dw, db = tfla.addnorm_backward(t, dy, w, bias=True, dtotal=dt)
    parts = [tfla.addnorm_backward(t[:, a:b], dy[:, a:b], w, bias=True, dtotal=dt[:, a:b])
             for a, b in zip(range(0, T, T // 4), [*range(T // 4, T, T // 4), T])]
    torch.cuda.synchronize()
    assert torch.equal(dx, torch.cat([p[0] for p in parts], 1)) and torch.equal(dr, torch.cat([p[1] for p in parts], 1))
    mag, n = dy.double().abs().sum((0, 1)), T + 100
    # sums of T terms in two orders; |th| is at most 6 here
    assert bool(((dw - sum(p[2] for p in parts)).abs() <= 2 * n * U * 6 * mag).all())
    assert bool(((db - sum(p[3] for p in parts)).abs() <= 2 * n * U * mag).all())
