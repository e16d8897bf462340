"""Gated linear recurrence of channels against the 64-bit reference.

Relative errors of the gates, u and v their pre-activations, U half a step of
fp32: an exponential e^-u is within (4 + 2 |u|) U (bf16 data takes it without
the low part of u log2 e), so s(u) within rs = (8 + 2 |u|) U; w = decay s(u)
within rs + U; f = e^-w within rf = w (rs + 2 U) + (4 + 2 w) U; 1 - f^2 by its
series within 6 U and the error of w, by the difference (w above 1/4, where it
is above 0.39) within 2 rf f^2 / 0.39 + 2 U, its root half of that and 2 U:
rm = rs + 2.6 rf + 6 U.

The recurrence E_t = f (E_{t-1} + rf H_{t-1}) + ri |i x| + 6 U H_t, H_t the
recurrence of the magnitudes, bounds the error of h however products of f are
put together (a factor's product, a term's sum: 6 U a step); the adjoint's
likewise from the end.  The gradients follow term by term."""
import numpy as np
import pytest
import torch

from blocks_helpers import HALF, U, as_view, randn, within
from mlstm_sequence_amd import tfla
from oracle import edges as O
from oracle.blocks import sigmoid

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
NAN = float("nan")
KIND = {"coupled": tfla.DIAG_COUPLED, "sigmoid": tfla.DIAG_SIGMOID, "decay": tfla.DIAG_DECAY}
KINDS = list(KIND)


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    tfla.lib()


def cuda(t):
    return None if t is None else t.cuda()


def make(dtype, kind, B, T, D, state=True, lengths=None, seed=0, shift=2.0):
    rng = np.random.default_rng(seed + 13 * T + D)
    d = dict(x=randn(rng, (B, T, D), dtype), fg=randn(rng, (B, T, D), dtype, 1.5, shift),
             ig=None if kind == "coupled" else randn(rng, (B, T, D), dtype, 1.5), decay=None,
             state=randn(rng, (B, D), F32) if state else None, dy=randn(rng, (B, T, D), dtype),
             dend=randn(rng, (B, D), F32) if state else None)
    if kind == "decay":
        t = torch.from_numpy(np.exp(rng.uniform(np.log(1e-3), np.log(2.0), D))).float()
        d["decay"] = (t, t.double().numpy())
    dev = {k: None if v is None else v[0] for k, v in d.items()}
    ref = {k: None if v is None else v[1] for k, v in d.items()}
    if lengths is not None:
        for k in ("x", "fg", "ig", "dy"):
            if dev[k] is not None:
                for b, n in enumerate(lengths):
                    dev[k][b, max(0, n):] = NAN
    dev["lengths"] = None if lengths is None else torch.tensor(lengths, dtype=torch.int32)
    return dev, ref


def reference(ref, kind, lengths):
    """({name: value}, {name: bound without the rounding to the output's type})"""
    x, fg, ig, decay, dy = (ref[k] for k in ("x", "fg", "ig", "decay", "dy"))
    B, T, D = x.shape
    y, end, before = O.diag(x, fg, ig, decay, kind, ref["state"], lengths)
    want = O.diag_grads(x, fg, dy, ig, decay, kind, ref["state"], lengths, ref["dend"])
    want.update(y=y, end=end, before=before)
    f, i = O.diag_gates(fg, ig, decay, kind)
    r, rs = sigmoid(fg), (8 + 2 * np.abs(fg)) * U
    if kind == "coupled":
        rf, ri = rs, (8 + 2 * np.abs(fg)) * U + 2 * U
    else:
        s, rv = sigmoid(ig), (8 + 2 * np.abs(ig)) * U
        if kind == "sigmoid":
            rf, ri = rs, rv
        else:
            w = decay * r
            rf = w * (rs + 2 * U) + (4 + 2 * w) * U
            rm = rs + 2.6 * rf + 6 * U
            ri = rm + rv + U
    lens = [T] * B if lengths is None else [min(max(n, 0), T) for n in lengths]
    Hb, Eb, G, EG = (np.zeros((B, T, D)) for _ in range(4))
    tol = dict(y=np.zeros((B, T, D)), end=np.zeros((B, D)), dstate=np.zeros((B, D)))
    for b, n in enumerate(lens):
        H = np.zeros(D) if ref["state"] is None else np.abs(ref["state"][b])
        E = np.zeros(D)
        for t in range(n):
            Hb[b, t], Eb[b, t] = H, E
            add = i[b, t] * np.abs(x[b, t])
            E = f[b, t] * (E + rf[b, t] * H) + ri[b, t] * add
            H = f[b, t] * H + add
            E = E + 6 * U * H
            tol["y"][b, t] = E
        Hb[b, n:], Eb[b, n:] = H, E
        tol["end"][b] = E
        A = np.zeros(D) if ref["dend"] is None else np.abs(ref["dend"][b])
        E = np.zeros(D)
        for t in range(n - 1, -1, -1):
            G[b, t] = np.abs(dy[b, t]) + A
            EG[b, t] = E + U * G[b, t]
            E = f[b, t] * (EG[b, t] + (rf[b, t] + 6 * U) * G[b, t])
            A = f[b, t] * G[b, t]
        tol["dstate"][b] = E
    tol["before"] = Eb
    X = np.abs(x)
    df, edf = Hb * G, Eb * G + Hb * EG + U * Hb * G
    di, edi = X * G, X * EG + U * X * G
    tol["dx"] = i * (EG + (ri + 2 * U) * G)
    if kind == "coupled":
        tol["dfgate"] = f * i * (edf + edi + (df + di) * (rf + ri + 6 * U))
    elif kind == "sigmoid":
        tol["dfgate"] = f * (1 - f) * (edf + df * (rf + 6 * U)) + df * f * (f * rf + U)
        tol["digate"] = i * (1 - i) * (edi + di * (ri + 6 * U)) + di * i * (i * ri + U)
    else:
        m = np.sqrt(-np.expm1(-2 * w))
        with np.errstate(divide="ignore", invalid="ignore"):
            dm = np.where(m > 0, f * f / m, 0.0)
        dw = di * s * dm + df * f
        edw = s * dm * (edi + di * (rv + 2 * rf + rm + 8 * U)) + f * (edf + df * (rf + 3 * U)) + U * dw
        tol["dfgate"] = w * (1 - r) * (edw + dw * (rs + 8 * U)) + dw * w * (r * rs + U)
        tol["digate"] = i * (1 - s) * (edi + di * (ri + 6 * U)) + di * i * (s * rv + U)
        tol["ddecay"] = (r * (edw + dw * (rs + 2 * U))).sum((0, 1)) + (B * T + 10) * U * (dw * r).sum((0, 1))
    return want, tol


def check(dtype, kind, B, T, D, state=True, lengths=None, view="plain", seed=0, shift=2.0):
    print("diag", dtype, kind, B, T, D, state, lengths, view, shift, flush=True)
    dev, ref = make(dtype, kind, B, T, D, state, lengths, seed, shift)
    x, fg, ig, dy = (as_view(dev[k], view) for k in ("x", "fg", "ig", "dy"))
    dc, st, de, ln = (cuda(dev[k]) for k in ("decay", "state", "dend", "lengths"))
    new = lambda: as_view(torch.full((B, T, D), NAN, dtype=dtype), view)  # noqa: E731
    kw = dict(kind=KIND[kind], lengths=ln)
    y, end, starts = tfla.diag_forward(x, fg, ig, dc, state=st, want_state=True, want_starts=True, y=new(), **kw)
    y2, _, _ = tfla.diag_forward(x, fg, ig, dc, state=st, **kw)            # without states
    g = tfla.diag_backward(x, fg, dy, starts, ig, dc, dstate_out=de, want_dstate=True, dx=new(), dfgate=new(),
                           digate=None if ig is None else new(), **kw)
    torch.cuda.synchronize()
    assert torch.equal(y, y2)
    want, tol = reference(ref, kind, lengths)
    rows = np.arange(0, T, tfla.DIAG_CHUNK)
    within("starts", starts, want["before"][:, rows], tol["before"][:, rows] + 1e-37)
    half = HALF[dtype]
    for name, got in (("y", y), ("end", end), ("dx", g.dx), ("dfgate", g.dfgate), ("digate", g.digate), ("ddecay", g.ddecay),
                      ("dstate", g.dstate)):
        if got is None:
            assert kind != "decay" and name == "ddecay" or kind == "coupled" and name == "digate"
            continue
        h = half if got.dtype == dtype and name not in ("end", "ddecay", "dstate") else U
        # values below the smallest normal number may come out 0
        within(name, got, want[name], h * np.abs(want[name]) + tol[name] + 1e-36)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("T", [1, 2, 3, 4, 5, 15, 16, 17, 31, 33, 64, 127, 128, 129, 255, 256, 257, 300, 520])
def test_lengths_of_one_call(dtype, kind, T):
    check(dtype, kind, 2, T, 64)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D", [1, 2, 3, 63, 65, 66, 96, 130, 200])
def test_channels(dtype, kind, D):
    check(dtype, kind, 2, 70, D)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("view", ["half", "odd", "wide", "time"])
@pytest.mark.parametrize("T", [3, 140])
def test_views(dtype, view, T):
    for kind in KINDS:
        check(dtype, kind, 2, T, 72, view=view)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("kind", KINDS)
def test_padded_batches(dtype, kind):
    check(dtype, kind, 5, 300, 40, lengths=[300, 0, 1, 129, 260])
    check(dtype, kind, 4, 40, 66, lengths=[-2, 39, 50, 17], state=False)
    check(dtype, kind, 3, 2, 66, lengths=[2, 0, 1])


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_long_sequences(dtype, kind):
    """A long axis over few channels, cut over workgroups."""
    check(dtype, kind, 1, 5000, 6, shift=4.0)
    check(dtype, kind, 2, 3333, 64, lengths=[3333, 1500], state=False)


def test_many_short_sequences():
    check(BF, "decay", 300, 3, 70)
    check(F32, "sigmoid", 300, 6, 66, lengths=[6 * (i % 3 > 0) for i in range(300)])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("kind", KINDS)
def test_prompt_then_single_tokens(dtype, kind):
    """States carried in fp32 and updated in place, against the formula for the whole."""
    B, T, D = 3, 150, 66
    dev, ref = make(dtype, kind, B, T, D)
    x, fg, ig, dc, st = (cuda(dev[k]) for k in ("x", "fg", "ig", "decay", "state"))
    cut = lambda a, b: [None if t is None else t[:, a:b] for t in (x, fg, ig)]  # noqa: E731
    parts = []
    y, s, _ = tfla.diag_forward(*cut(0, 140), dc, kind=KIND[kind], state=st, want_state=True)
    parts.append(y)
    for a, b in [(140, 141), (141, 142), (142, 145), (145, 150)]:
        y, again, _ = tfla.diag_forward(*cut(a, b), dc, kind=KIND[kind], state=s, state_out=s)
        assert again is s
        parts.append(y)
    torch.cuda.synchronize()
    want, tol = reference(ref, kind, None)
    within("y", torch.cat(parts, 1), want["y"], HALF[dtype] * np.abs(want["y"]) + tol["y"] + 1e-36)
    within("state", s, want["end"], U * np.abs(want["end"]) + tol["end"] + 1e-36)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_extreme_gates(dtype):
    """Pre-activations where the exponential over- or underflows, gates of exactly 0 and 1, no decay."""
    B, T, D = 1, 40, 8
    big = torch.tensor([200.0, -200.0, 100.0, -100.0, 90.0, -90.0, float("inf"), -float("inf")])
    x = torch.randn(B, T, D, generator=torch.Generator().manual_seed(1)).to(dtype)
    dy = torch.randn(B, T, D, generator=torch.Generator().manual_seed(2)).to(dtype)
    st = torch.randn(B, D, generator=torch.Generator().manual_seed(3))
    gate = big.expand(B, T, D).contiguous().to(dtype)
    other = torch.randn(B, T, D, generator=torch.Generator().manual_seed(4)).to(dtype)
    f64 = lambda t: None if t is None else t.double().numpy()  # noqa: E731
    for kind, fg, ig, dc in (("coupled", gate, None, None), ("sigmoid", gate, other, None), ("sigmoid", other, gate, None),
                             ("decay", gate, other, torch.full((D,), 0.5)), ("decay", other, gate, torch.full((D,), 0.5)),
                             ("decay", other, other, torch.zeros(D)), ("decay", other, other, torch.full((D,), 300.0))):
        y, end, starts = tfla.diag_forward(x.cuda(), fg.cuda(), cuda(ig), cuda(dc), kind=KIND[kind], state=st.cuda(),
                                           want_state=True, want_starts=True)
        g = tfla.diag_backward(x.cuda(), fg.cuda(), dy.cuda(), starts, cuda(ig), cuda(dc), kind=KIND[kind], want_dstate=True)
        torch.cuda.synchronize()
        args = (f64(x), f64(fg))
        wy, wend, _ = O.diag(*args, f64(ig), f64(dc), kind, f64(st))
        with np.errstate(all="ignore"):
            wg = O.diag_grads(*args, f64(dy), f64(ig), f64(dc), kind, f64(st))
        for name, got, want in (("y", y, wy), ("end", end, wend), ("dx", g.dx, wg["dx"]), ("dfgate", g.dfgate, wg["dfgate"]),
                                ("digate", g.digate, wg["digate"]), ("dstate", g.dstate, wg["dstate"])):
            if got is not None:
                # gates are at their limits within 1e-30; h and g are sums of up to 40 terms of order 3
                within(f"{kind} {name}", got, want, HALF[dtype] * np.abs(want) + 40 * 40 * 3 * 20 * U)


def test_nan_stays_in_its_channel_and_behind_its_row():
    dev, _ = make(F32, "sigmoid", 2, 50, 70)
    x, fg, ig = (dev[k].cuda() for k in ("x", "fg", "ig"))
    want, _, _ = tfla.diag_forward(x, fg, ig, kind=tfla.DIAG_SIGMOID)
    x[1, 20, 33] = NAN
    y, _, _ = tfla.diag_forward(x, fg, ig, kind=tfla.DIAG_SIGMOID)
    torch.cuda.synchronize()
    bad = torch.zeros_like(y, dtype=torch.bool)
    bad[1, 20:, 33] = True
    assert torch.equal(torch.isnan(y), bad) and torch.equal(y[~bad], want[~bad])


def test_broadcast_inputs():
    """Rows and batches that share memory (strides of 0) are read like any other."""
    for dtype in (BF, F32):
        B, T, D = 2, 140, 64
        fg = torch.randn(D, device="cuda").to(dtype).expand(B, T, D)
        x = torch.randn(1, T, D, device="cuda").to(dtype).expand(B, T, D)
        dy = torch.randn(B, 1, D, device="cuda").to(dtype).expand(B, T, D)
        y, _, st = tfla.diag_forward(x, fg, want_starts=True)
        wy, _, ws = tfla.diag_forward(x.contiguous(), fg.contiguous(), want_starts=True)
        g = tfla.diag_backward(x, fg, dy, st)
        w = tfla.diag_backward(x.contiguous(), fg.contiguous(), dy.contiguous(), ws)
        torch.cuda.synchronize()
        eps = 8 * HALF[dtype]
        for a, b in ((y, wy), (g.dx, w.dx), (g.dfgate, w.dfgate)):
            assert torch.allclose(a.float(), b.float(), rtol=eps, atol=1e-4 if dtype == F32 else eps * 4)


def test_refusals_on_tensors():
    dev, _ = make(BF, "decay", 2, 10, 16)
    x, fg, ig, dc, st, dy = (dev[k].cuda() for k in ("x", "fg", "ig", "decay", "state", "dy"))
    for bad in (dict(decay=None), dict(igate=None), dict(kind=tfla.DIAG_COUPLED), dict(kind=tfla.DIAG_SIGMOID), dict(kind=5),
                dict(fgate=fg.float()), dict(fgate=fg[:, :5]), dict(decay=dc[:8]), dict(decay=dc.double()), dict(state=st[:1]),
                dict(state=st.to(BF)), dict(x=x.transpose(1, 2)), dict(y=x), dict(y=x.new_zeros(2, 10, 8)), dict(igate=ig.cpu()),
                dict(lengths=torch.zeros(2, device="cuda")), dict(starts=st), dict(state_out=st[:, :8])):
        kw = dict(x=x, fgate=fg, igate=ig, decay=dc, state=st, kind=tfla.DIAG_DECAY)
        kw.update(bad)
        with pytest.raises((TypeError, ValueError, tfla.TflaError)):
            tfla.diag_forward(**kw)
    _, _, starts = tfla.diag_forward(x, fg, ig, dc, kind=tfla.DIAG_DECAY, want_starts=True)
    for bad in (dict(starts=None), dict(starts=starts[:, 0]), dict(dy=dy[:, :4]), dict(dx=dy), dict(dstate_out=st.to(BF)),
                dict(workspace=torch.empty(16, dtype=torch.uint8, device="cuda")), dict(igate=None, kind=tfla.DIAG_COUPLED)):
        kw = dict(x=x, fgate=fg, dy=dy, starts=starts, igate=ig, decay=dc, kind=tfla.DIAG_DECAY)
        kw.update(bad)
        with pytest.raises((TypeError, ValueError, tfla.TflaError)):
            tfla.diag_backward(**kw)
    with pytest.raises(ValueError):
        tfla.diag_backward(x, fg, dy, starts, digate=torch.empty_like(x))


def test_gradients_into_a_projections_gradient():
    dev, _ = make(BF, "sigmoid", 2, 200, 64)
    x, fg, ig, dy = (dev[k].cuda() for k in ("x", "fg", "ig", "dy"))
    _, _, starts = tfla.diag_forward(x, fg, ig, kind=tfla.DIAG_SIGMOID, want_starts=True)
    want = tfla.diag_backward(x, fg, dy, starts, ig, kind=tfla.DIAG_SIGMOID)
    all_ = torch.full((2, 200, 4 * 64), 7.0, dtype=BF, device="cuda")
    got = tfla.diag_backward(x, fg, dy, starts, ig, kind=tfla.DIAG_SIGMOID, dx=all_[..., :64], dfgate=all_[..., 64:128],
                             digate=all_[..., 128:192])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got[:3], want[:3])) and bool((all_[..., 192:] == 7.0).all())


@pytest.mark.parametrize("T,D", [(333, 136), (4000, 64)])
def test_stream_workspace_and_repeat(T, D):
    """Another stream, the caller's workspaces and the library's own allocation give the same bits."""
    dev, _ = make(BF, "decay", 2, T, D)
    x, fg, ig, dc, st, dy, de = (dev[k].cuda() for k in ("x", "fg", "ig", "decay", "state", "dy", "dend"))

    def step(**k):
        y, end, starts = tfla.diag_forward(x, fg, ig, dc, kind=tfla.DIAG_DECAY, state=st, want_state=True, want_starts=True,
                                           workspace=k.pop("ws", None), **k)
        g = tfla.diag_backward(x, fg, dy, starts, ig, dc, kind=tfla.DIAG_DECAY, dstate_out=de, want_dstate=True,
                               workspace=k.pop("wb", None), **k)
        return [y, end, starts, *g]

    want = step()
    L = tfla.lib()
    size = lambda n: torch.empty(max(n, 256), dtype=torch.uint8, device="cuda")  # noqa: E731
    ws = size(L.tfla_diag_workspace_bytes(2, T, D, 2, 0x100))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        a = step()
    b = step(ws=ws)
    c = step(stream=side)
    torch.cuda.synchronize()
    for got in (a, b, c):
        assert all(torch.equal(p, q) for p, q in zip(got, want))


@pytest.mark.parametrize("T", [40, 3000])
def test_captured_and_replayed(T):
    dev, _ = make(BF, "decay", 2, T, 64)
    x, fg, ig, dc, st, dy = (dev[k].cuda() for k in ("x", "fg", "ig", "decay", "state", "dy"))

    def step():
        y, end, starts = tfla.diag_forward(x, fg, ig, dc, kind=tfla.DIAG_DECAY, state=st, want_state=True, want_starts=True)
        return [y, end, *tfla.diag_backward(x, fg, dy, starts, ig, dc, kind=tfla.DIAG_DECAY, want_dstate=True)]

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


@pytest.mark.parametrize("D", [64, 65])
def test_offsets_beyond_32_bits(D):
    """Batches 2^32 elements apart in one buffer, and rows 2^24 elements apart."""
    for T, far, row in ((9, (1 << 32) + 128, 128), (140, 0, 1 << 24)):
        n = 2 if far else 1
        full = torch.empty(far * (n - 1) + (T - 1) * row + D + 8, dtype=BF, device="cuda")
        view = torch.as_strided(full, (n, T, D), (far, row, 1))
        x, fg = torch.randn(n, T, D, device="cuda").to(BF), torch.randn(n, T, D, device="cuda").to(BF)
        want, _, ws = tfla.diag_forward(x, fg, want_starts=True)
        wg = tfla.diag_backward(x, fg, want, ws)
        tol = dict(rtol=2.0 ** -6, atol=1e-2)
        view.copy_(x)
        got, _, st = tfla.diag_forward(view, fg, want_starts=True)
        assert torch.allclose(got.float(), want.float(), **tol)
        g = tfla.diag_backward(view, fg, want, ws)
        assert torch.allclose(g.dx.float(), wg.dx.float(), **tol) and torch.allclose(g.dfgate.float(), wg.dfgate.float(), **tol)
        tfla.diag_forward(x, fg, y=view)
        assert torch.allclose(view.float(), want.float(), **tol)
        tfla.diag_backward(x, fg, want, ws, dfgate=view)
        assert torch.allclose(view.float(), wg.dfgate.float(), **tol)
        torch.cuda.synchronize()
        del full, view


def test_very_many_sequences():
    """More workgroups than one dimension of a grid holds."""
    B, T, D = (1 << 21) + 5, 5, 1
    x, fg, dy = (torch.randn(B, T, D, device="cuda") for _ in range(3))
    y, end, starts = tfla.diag_forward(x, fg, want_state=True, want_starts=True)
    g = tfla.diag_backward(x, fg, dy, starts, want_dstate=True)
    f = torch.sigmoid(fg.double())
    h, hs = torch.zeros(B, D, dtype=torch.float64, device="cuda"), []
    for t in range(T):
        hs.append(h)
        h = f[:, t] * h + (1 - f[:, t]) * x[:, t]
    a = torch.zeros_like(h)
    for t in reversed(range(T)):
        gt = dy[:, t] + a
        a = f[:, t] * gt
        # up to 5 terms of order 5, gates within 20 U
        assert float((g.dx[:, t] - (1 - f[:, t]) * gt).abs().max()) <= 5 * 5 * 40 * U
        assert float((g.dfgate[:, t] - f[:, t] * (1 - f[:, t]) * gt * (hs[t] - x[:, t])).abs().max()) <= 25 * 5 * 40 * U
    torch.cuda.synchronize()
    assert float((end - h).abs().max()) <= 5 * 5 * 40 * U and float((g.dstate - a).abs().max()) <= 5 * 5 * 40 * U


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("B,T,D", [(2, 700, 520), (9, 140, 1000), (3, 900, 1100), (33, 130, 520), (1, 2500, 64)])
def test_cuts(dtype, kind, B, T, D):
    """Blocks of 16, 32 and 64 channels, whole and in segments."""
    check(dtype, kind, B, T, D)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("B,T,D", [(40, 20, 512), (40, 21, 512), (3, 16, 70), (3, 17, 70)])
def test_short_axes(dtype, kind, B, T, D):
    """On both sides of where a thread takes a channel; padded, with sequences of no row and of one."""
    check(dtype, kind, B, T, D, lengths=[(0, 1, T, T // 2, T - 1)[i % 5] for i in range(B)])


@pytest.mark.parametrize("dtype,kind,B,T,D", [(F32, "coupled", 1030, 64, 3), (F32, "coupled", 1044, 65, 3), (BF, "coupled", 2050, 128, 1),
                                              (BF, "decay", 4100, 256, 1), (F32, "sigmoid", 2050, 129, 1)])
def test_short_axes_of_many_channels(dtype, kind, B, T, D):
    """Longer ones, over one chunk and more."""
    check(dtype, kind, B, T, D, lengths=[(0, 1, T, T // 2, T - 1)[i % 5] for i in range(B)])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("B,T,D", [(33, 130, 512), (33, 130, 528), (33, 130, 513), (2, 2500, 192), (2, 2500, 163),
                                   (5, 300, 1024), (5, 300, 1000), (70, 2100, 2), (40, 2300, 3)])
def test_rows_on_lines_and_off_them(dtype, kind, B, T, D):
    check(dtype, kind, B, T, D)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_state_in_place_of_a_long_call(dtype):
    """Cut into segments, every one of which starts from the state that the last one replaces."""
    dev, _ = make(dtype, "decay", 2, 3000, 200)
    x, fg, ig, dc, st = (dev[k].cuda() for k in ("x", "fg", "ig", "decay", "state"))
    kw = dict(kind=tfla.DIAG_DECAY, want_starts=True)
    assert tfla.lib().tfla_diag_workspace_bytes(2, 3000, 200, 2, 0x100 if dtype == BF else 0) > 0
    want, end, starts = tfla.diag_forward(x, fg, ig, dc, state=st, want_state=True, **kw)
    got, same, again = tfla.diag_forward(x, fg, ig, dc, state=st, state_out=st, **kw)
    torch.cuda.synchronize()
    assert same is st and torch.equal(got, want) and torch.equal(st, end) and torch.equal(again, starts)


def test_a_states_copy_serves_every_segment():
    """The workspace holds the state before the first row once a call is cut: what a workgroup that starts late reads."""
    dev, _ = make(F32, "coupled", 1, 3000, 64)
    x, fg, st = (dev[k].cuda() for k in ("x", "fg", "state"))
    n = tfla.lib().tfla_diag_workspace_bytes(1, 3000, 64, 0, 0)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    before = st.clone()
    tfla.diag_forward(x, fg, state=st, state_out=st, workspace=ws)
    torch.cuda.synchronize()
    pairs = ws.view(torch.float32).view(-1, 2)
    held = [i for i in range(0, pairs.shape[0] - 63, 64) if torch.equal(pairs[i:i + 64, 1], before[0])]
    assert held and not torch.equal(st, before)


def compare(dtype, kind, dev, ref, lengths=None, extra=0.0):
    """A forward and a backward call on the tensors of `dev` against the reference on `ref`; extra: added to every bound."""
    B, T, D = ref["x"].shape
    print("diag", dtype, kind, B, T, D, lengths, flush=True)
    d = {k: cuda(v) for k, v in dev.items()}
    kw = dict(kind=KIND[kind], lengths=d["lengths"])
    y, end, starts = tfla.diag_forward(d["x"], d["fg"], d["ig"], d["decay"], state=d["state"], want_state=True, want_starts=True,
                                       **kw)
    g = tfla.diag_backward(d["x"], d["fg"], d["dy"], starts, d["ig"], d["decay"], dstate_out=d["dend"], want_dstate=True, **kw)
    torch.cuda.synchronize()
    want, tol = reference(ref, kind, lengths)
    rows = np.arange(0, T, tfla.DIAG_CHUNK)
    within("starts", starts, want["before"][:, rows], tol["before"][:, rows] + 1e-37 + extra)
    for name, got, half in (("y", y, HALF[dtype]), ("end", end, U), ("dx", g.dx, HALF[dtype]), ("dfgate", g.dfgate, HALF[dtype]),
                            ("digate", g.digate, HALF[dtype]), ("ddecay", g.ddecay, U), ("dstate", g.dstate, U)):
        if got is not None:
            within(f"{kind} {name}", got, want[name], half * np.abs(want[name]) + tol[name] + 1e-36 + extra)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("T", [1, 12, 40, 140])
def test_gates_whose_reciprocal_is_below_the_smallest_number(dtype, kind, T):
    """Pre-activations around -88, where 1 / (1 + e^-u) is finite and below 2^-126, and as far on the other side: a single
    token, a short axis, tiles."""
    u = torch.tensor([87.0, 87.25, 87.5, 88.0, 88.5, 88.7, 88.75, 89.0])
    u = torch.cat([u, -u])
    D = 4 * len(u)
    for which in ("fg", "ig"):
        if which == "ig" and kind == "coupled":
            continue
        dev, ref = make(dtype, kind, 2, T, D)
        gate = u.repeat_interleave(4).expand(2, T, D).contiguous().to(dtype)
        gate[:, :, 3::4] = dev[which][:, :, 3::4]          # every fourth channel ordinary, and every third row of others
        gate[:, ::3, 2::4] = dev[which][:, ::3, 2::4]
        dev[which], ref[which] = gate, gate.double().numpy()
        # A sigmoid below 2^-126 may come out 0: f and i are off by that, and with a decay w by 2^-125, sqrt(1 - f^2) by
        # 2^-62 (decay <= 2), what the root's slope leaves out of du by sqrt(w / 2), of ddecay by sqrt(s(u) / 2 decay), at
        # most 2^-58 (decay >= 1e-3).  Each is met with |x g| at most: x and dy below 5, g a sum of T + 1 terms, T + 1 rows
        # of two sequences to a sum.
        compare(dtype, kind, dev, ref, extra=(2.0 ** -58 if kind == "decay" else 2.0 ** -126) * 25 * 2 * (T + 1) ** 2)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T", [1, 40])
def test_a_closed_coupled_gate_passes_its_input(dtype, T):
    """f below 2^-126 and i = 1: rows are their inputs and dx is dy, to the last bit."""
    x, dy = (torch.randn(2, T, 64, device="cuda").to(dtype) for _ in range(2))
    for u in (-87.5, -88.0, -88.5, -100.0, -float("inf")):
        fg = torch.full_like(x, u)
        y, end, starts = tfla.diag_forward(x, fg, state=torch.ones(2, 64, device="cuda"), want_state=True, want_starts=True)
        g = tfla.diag_backward(x, fg, dy, starts)
        torch.cuda.synchronize()
        assert torch.equal(y, x) and torch.equal(end, x[:, -1].float()) and torch.equal(g.dx, dy), u


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("B,T,D,lengths", [
    (2, 600, 4160, (600, 430)),          # 64 channels, whole axes of 5 tiles on lines
    (3, 640, 2816, (640, 512, 301)),     # the same, ending with a tile
    (2, 600, 4161, (513, 600)),          # off the lines
    (3, 5200, 512, (5200, 3000, 4480)),  # 64 channels in segments of 5 tiles
    (2, 2000, 520, (2000, 1300)),        # 16 channels forward, tiles of 512 rows
    (2, 1100, 2560, (1100, 900)),        # 32 channels, tiles of 256
    (2, 2100, 2560, (2100, 1025)),       # 32 forward; backward 32 in fp32, segments in bf16
    (1, 2100, 4096, (2100,)),            # 16 channels forward in fp32, segments else
])
def test_walks_of_several_tiles(dtype, kind, B, T, D, lengths):
    """Tiles whose loads were issued in the loop, not before it."""
    dev, ref = make(dtype, kind, B, T, D, lengths=lengths)
    compare(dtype, kind, dev, ref, lengths)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,T,D", [(2, 600, 4160), (1, 3000, 200)])
def test_walks_of_several_tiles_over_shared_rows(dtype, B, T, D):
    """Rows that share memory (a stride of 0) go by 64-bit addresses: whole axes and segments, ragged."""
    lengths = [T - 170 * b - 5 for b in range(B)]
    for kind in KINDS:
        dev, ref = make(dtype, kind, B, T, D)
        for k in ("fg", "dy"):
            dev[k] = dev[k][:, :1].cuda().expand(B, T, D)
            ref[k] = np.broadcast_to(ref[k][:, :1], (B, T, D))
        dev["lengths"] = torch.tensor(lengths, dtype=torch.int32)
        compare(dtype, kind, dev, ref, lengths)
