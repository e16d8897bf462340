"""Group norm with an activation or a gate against the 64-bit reference.

Error bounds, with U half a step of fp32, n the values of a set, A their mean
magnitude, m and s^2 their mean and variance, N = n + 60 (a sum of n terms in
any order, and the joining of partial means):
  m       N U A
  s^2     2 N U s^2 + 4 s N U A     (values minus the mean carry the mean's error)
  rstd    half of that over s^2 + eps, and 4 U, relative
and through xh, u, the activation (slope at most 1.1, second derivative at
most 0.5, its value within 12 U) and the gradient's formula term by term."""
import numpy as np
import pytest
import torch

from blocks_helpers import HALF, U, randn, within
from mlstm_sequence_amd import tfla
from oracle import blocks as O

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
NAN = float("nan")
EPS = 1e-5
ACT = {"none": tfla.ACT_NONE, "silu": tfla.ACT_SILU, "sigmoid": tfla.ACT_SIGMOID}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    tfla.lib()


def as_heads(t, layout):
    """The CPU tensor [B,T,G,C] on the GPU: "plain"; "heads" head-major
    memory; "half" the second half of rows twice as wide; "odd" rows one
    element longer; "time" time-major."""
    if t is None:
        return None
    t = t.cuda()
    B, T, G, C = t.shape
    if layout == "plain":
        return t
    if layout == "heads":
        return t.transpose(1, 2).contiguous().transpose(1, 2)
    if layout == "time":
        return t.transpose(0, 1).contiguous().transpose(0, 1)
    W = G * C
    pad, at = (W, W) if layout == "half" else (1, 1)
    full = torch.full((B, T, W + pad), NAN, dtype=t.dtype, device="cuda")
    full[..., at:at + W] = t.flatten(2)
    return full[..., at:at + W].unflatten(-1, (G, C))


def check(dtype, B, T, G, C, sequence=False, kind="silu", gated=False, affine=True, layout="plain", scale=2.0, shift=0.5):
    print("norm", dtype, B, T, G, C, sequence, kind, gated, affine, layout, scale, shift, flush=True)
    rng = np.random.default_rng(T + 7 * C + G)
    tx, x = randn(rng, (B, T, G, C), dtype, scale, shift)
    tw, w = randn(rng, (G, C), F32, 0.3, 1.0) if affine else (None, None)
    tb, b = randn(rng, (G, C), F32, 0.3) if affine else (None, None)
    tz, z = randn(rng, (B, T, G, C), dtype, 2.0) if gated else (None, None)
    tg, dy = randn(rng, (B, T, G, C), dtype)
    gx, gz, gdy = (as_heads(t, layout) for t in (tx, tz, tg))
    gw, gb = (None if t is None else t.cuda() for t in (tw, tb))
    new = lambda: as_heads(torch.full((B, T, G, C), NAN, dtype=dtype), layout)  # noqa: E731
    kw = dict(act=ACT[kind], gate=gz, over=tfla.NORM_SEQUENCE if sequence else tfla.NORM_TOKEN)
    y, mean, rstd = tfla.norm_forward(gx, gw, gb, eps=EPS, y=new(), **kw)
    dx, dz, dw, db = tfla.norm_backward(gx, gdy, mean, rstd, gw, gb, dx=new(), dgate=new() if gated else None, **kw)
    torch.cuda.synchronize()

    dims = (1, 3) if sequence else (3,)
    n = C * (T if sequence else 1)
    N = (n + 60) * U
    ek = dict(eps=EPS, kind=kind, gate=z, sequence=sequence)
    wy, wm, wr = O.norm(x, w, b, **ek)
    wdx, wdz, wdw, wdb = O.norm_grads(x, dy, w, b, **ek)
    ex = (lambda v: v[:, None, :, None]) if sequence else (lambda v: v[..., None])
    m, r = ex(wm), ex(wr)
    A = np.abs(x).mean(dims, keepdims=True)
    var = ((x - m) ** 2).mean(dims, keepdims=True)
    em = N * A
    evar = 2 * N * var + 4 * np.sqrt(var) * em + em ** 2
    er = 0.5 * evar / (var + EPS) + 4 * U
    sq = (lambda v: v[:, 0, :, 0]) if sequence else (lambda v: v[..., 0])
    within("mean", mean, wm, sq(em) + U * np.abs(wm))
    within("rstd", rstd, wr, sq(er) * wr + U * wr)

    W = 1.0 if w is None else np.abs(w)
    xh = (x - m) * r
    u = xh * (1.0 if w is None else w) + (0.0 if b is None else b)
    exh = r * (2 * U * (np.abs(x) + np.abs(m)) + em) + np.abs(xh) * er
    eu = W * exh + 3 * U * (np.abs(xh) * W + (0.0 if b is None else np.abs(b)))
    h = HALF[dtype]
    if gated:
        f, df = O.act(z, kind)
        ey = np.abs(f) * eu + 14 * U * np.abs(u * f)
        edu = 13 * U * np.abs(dy * f)
        edz = np.abs(dy * df) * eu + 16 * U * np.abs(dy * u) * 1.1
        within("dgate", dz, wdz, h * np.abs(wdz) + edz + 1e-37)
        du = dy * f
    else:
        assert dz is None
        f, df = O.act(u, kind)
        ey = 1.1 * eu + 12 * U * np.abs(f)
        du = dy * df
        edu = np.abs(dy) * ((0.5 * eu + 12 * U) if kind != "none" else U)
    within("y", y, wy, h * np.abs(wy) + ey + 1e-37)
    v, ev = du * (1.0 if w is None else w), W * edu + 2 * U * np.abs(du) * W
    mv, mvx = v.mean(dims, keepdims=True), (v * xh).mean(dims, keepdims=True)
    emv = ev.mean(dims, keepdims=True) + N * np.abs(v).mean(dims, keepdims=True)
    emvx = (ev * np.abs(xh) + np.abs(v) * exh).mean(dims, keepdims=True) + N * np.abs(v * xh).mean(dims, keepdims=True)
    edx = r * (ev + emv + np.abs(xh) * emvx + exh * np.abs(mvx)) + (er + 5 * U) * r * (np.abs(v) + np.abs(mv) + np.abs(xh * mvx))
    within("dx", dx, wdx, h * np.abs(wdx) + edx + 1e-37)
    if affine:
        rows = (B * T + 60) * U
        within("dweight", dw, wdw, (edu * np.abs(xh) + np.abs(du) * exh).sum((0, 1)) + rows * np.abs(du * xh).sum((0, 1)) + 1e-37)
        within("dbias", db, wdb, edu.sum((0, 1)) + rows * np.abs(du).sum((0, 1)) + 1e-37)
    else:
        assert dw is None and db is None


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("C", [1, 2, 7, 8, 12, 64, 96, 100, 128, 200, 256, 500, 512, 1000, 1024, 2048, 2056, 5000])
def test_token_widths(dtype, C):
    check(dtype, 2, 5, 3, C)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("kind", ["none", "silu", "sigmoid"])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("sequence", [False, True])
def test_activations(dtype, kind, gated, sequence):
    check(dtype, 2, 9, 4, 64, sequence=sequence, kind=kind, gated=gated)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("layout", ["heads", "half", "odd", "time"])
@pytest.mark.parametrize("sequence", [False, True])
@pytest.mark.parametrize("C", [64, 20, 7])
def test_layouts(dtype, layout, sequence, C):
    check(dtype, 3, 11, 4, C, sequence=sequence, gated=True, layout=layout)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,T,G", [(1, 1, 1), (1, 1, 8), (3, 1, 5), (1, 77, 1), (2, 130, 3), (5, 33, 16), (1, 300, 2)])
@pytest.mark.parametrize("C", [64, 24])
def test_token_rows_and_groups(dtype, B, T, G, C):
    check(dtype, B, T, G, C, gated=T % 2 == 1)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 64, 255, 1000])
@pytest.mark.parametrize("G,C", [(4, 16), (3, 27), (1, 8)])
def test_sequence_lengths(dtype, T, G, C):
    check(dtype, 2, T, G, C, sequence=True)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("G,C", [(64, 1), (2, 2048), (1, 5000), (5, 600), (300, 8)])
def test_sequence_widths(dtype, G, C):
    check(dtype, 2, 21, G, C, sequence=True, gated=G == 2)


@pytest.mark.parametrize("sequence", [False, True])
def test_without_weights(sequence):
    check(F32, 2, 6, 2, 32, sequence=sequence, affine=False)
    check(BF, 2, 6, 2, 33, sequence=sequence, affine=False, kind="sigmoid")


@pytest.mark.parametrize("sequence", [False, True])
def test_large_mean(sequence):
    """A mean 1000 times the spread: the variance is formed around it."""
    check(F32, 2, 40, 2, 64, sequence=sequence, scale=1.0, shift=1000.0)


@pytest.mark.parametrize("sequence", [False, True])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_constant_values(sequence, dtype):
    """No variance: xh is 0, y is act(bias), everything finite."""
    x = torch.full((2, 6, 2, 32), 3.0, dtype=dtype, device="cuda")
    b = torch.randn(2, 32, device="cuda")
    over = tfla.NORM_SEQUENCE if sequence else tfla.NORM_TOKEN
    y, mean, rstd = tfla.norm_forward(x, None, b, over=over)
    g = tfla.norm_backward(x, torch.ones_like(x), mean, rstd, None, b, over=over)
    torch.cuda.synchronize()
    assert torch.equal(y, b.to(dtype).expand_as(y)) and bool((mean == 3.0).all())
    assert all(bool(torch.isfinite(t).all()) for t in (rstd, g[0], g[3]))


def test_head_major_output_of_the_recurrence():
    """norm(h) of the forward pass's own output, seen as [B,T,H,d], laid out for a projection."""
    B, H, T, dqk, dhv = 2, 4, 150, 64, 128
    g = torch.Generator().manual_seed(3)
    q, k = (torch.randn(B, H, T, dqk, generator=g).bfloat16().cuda() for _ in range(2))
    v = torch.randn(B, H, T, dhv, generator=g).bfloat16().cuda()
    ig, fg = torch.randn(B, H, T, generator=g).cuda(), (torch.randn(B, H, T, generator=g) + 3).cuda()
    h = tfla.forward(q, k, v, ig, fg, tfla.MLSTM_SIG, 64)
    gate = torch.randn(B, T, H, dhv, generator=g).bfloat16().cuda()
    y, mean, rstd = tfla.norm_forward(h.transpose(1, 2), act=tfla.ACT_SIGMOID, gate=gate)
    torch.cuda.synchronize()
    assert y.is_contiguous() and y.shape == (B, T, H, dhv)
    x = h.transpose(1, 2).double().cpu().numpy()
    want, _, wr = O.norm(x, kind="sigmoid", gate=gate.double().cpu().numpy())
    xh = np.abs(O.norm(x, kind="none")[0])
    # as in check(): n = dhv values, no weights
    A = np.abs(x).mean(3, keepdims=True)
    s = x.std(3, keepdims=True)
    N = (dhv + 60) * U
    r = wr[..., None]
    er = 0.5 * (2 * N * s ** 2 + 4 * s * N * A) / (s ** 2 + EPS) + 4 * U
    eu = r * (2 * U * (np.abs(x) + A) + N * A) + xh * er + 3 * U * xh
    within("y", y, want, HALF[BF] * np.abs(want) + eu + 14 * U * xh + 1e-37)


def test_refusals_on_tensors():
    x = torch.randn(2, 5, 4, 32, device="cuda")
    w = torch.ones(4, 32, device="cuda")
    y, mean, rstd = tfla.norm_forward(x, w)
    for bad in (dict(weight=w.bfloat16()), dict(weight=w[:2]), dict(gate=x[:1]), dict(gate=x.bfloat16()), dict(x=x[0]),
                dict(x=x.transpose(2, 3)), dict(y=x), dict(over=7), dict(act=9), dict(eps=0.0), dict(gate=x.cpu())):
        kw = dict(x=x, weight=w)
        kw.update(bad)
        with pytest.raises((TypeError, ValueError, tfla.TflaError)):
            tfla.norm_forward(**kw)
    for bad in (dict(mean=mean[:1]), dict(rstd=rstd.double()), dict(dy=x[:, :2]), dict(dx=x)):
        kw = dict(x=x, dy=torch.ones_like(x), mean=mean, rstd=rstd, weight=w)
        kw.update(bad)
        with pytest.raises((TypeError, ValueError, tfla.TflaError)):
            tfla.norm_backward(**kw)


@pytest.mark.parametrize("over", [tfla.NORM_TOKEN, tfla.NORM_SEQUENCE])
def test_captured_replayed_streams_and_workspaces(over):
    x, dy, z = (torch.randn(2, 300, 4, 64, device="cuda").bfloat16() for _ in range(3))
    w, b = torch.randn(4, 64, device="cuda"), torch.randn(4, 64, device="cuda")
    kw = dict(act=tfla.ACT_SILU, gate=z, over=over)

    def both(**more):
        f = tfla.norm_forward(x, w, b, **kw, **more)
        return f + tfla.norm_backward(x, dy, f[1], f[2], w, b, **kw, **more)

    want = both()
    L = tfla.lib()
    n = max(256, L.tfla_norm_workspace_bytes(2, 300, 4, 64, 0x100 | over), L.tfla_norm_bwd_workspace_bytes(2, 300, 4, 64, 0x100 | over))
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = both()
    torch.cuda.synchronize()
    for g in (got, both(workspace=ws), both(stream=side)):
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(g, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = both()
    for _ in range(3):
        x.copy_(torch.randn_like(x))
        dy.copy_(torch.randn_like(dy))
        graph.replay()
        torch.cuda.synchronize()
        want = both()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(out, want))


def test_a_large_call_equals_its_halves():
    """Calls that move more than the caches hold load past them; rows are
    independent, so the two halves of the batch give the same bits."""
    B, T, G, C = 2, 8192, 32, 256
    x, dy = (torch.randn(B, T, G, C, device="cuda", dtype=BF) for _ in range(2))
    z = torch.randn(B, T, G, C, device="cuda", dtype=BF)
    w, b = torch.randn(G, C, device="cuda"), torch.randn(G, C, device="cuda")
    kw = dict(act=tfla.ACT_SILU)
    y, mean, rstd = tfla.norm_forward(x, w, b, gate=z, **kw)
    dx, dz, dw, db = tfla.norm_backward(x, dy, mean, rstd, w, b, gate=z, **kw)
    sums = [torch.zeros(G, C, dtype=torch.float64, device="cuda") for _ in range(2)]
    for i in range(2):
        h = slice(i, i + 1)
        yh, mh, rh = tfla.norm_forward(x[h], w, b, gate=z[h], **kw)
        gh = tfla.norm_backward(x[h], dy[h], mh, rh, w, b, gate=z[h], **kw)
        assert torch.equal(yh, y[h]) and torch.equal(mh, mean[h]) and torch.equal(rh, rstd[h])
        assert torch.equal(gh[0], dx[h]) and torch.equal(gh[1], dz[h])
        sums[0] += gh[2].double()
        sums[1] += gh[3].double()
    # du xh and du summed over 2^14 rows twice, in other orders: each within (n + 1) U of their magnitudes, which
    # are below 64 sqrt(n) here only on average, so bounded by the values' own: |dy| <= 7, |act| <= 7, |xh| <= 7
    tol = 2 * (B * T + 1) * U * B * T * 7.0 ** 3
    assert float((sums[0] - dw).abs().max()) <= tol and float((sums[1] - db).abs().max()) <= tol


def test_offsets_beyond_32_bits():
    """Batches 2^32 elements apart in one buffer."""
    T, G, C = 3, 4, 64
    far = (1 << 32) + 64
    buf = torch.empty(far + T * G * C, dtype=BF, device="cuda")
    view = torch.as_strided(buf, (2, T, G, C), (far, G * C, C, 1))
    out = torch.as_strided(torch.empty_like(buf), (2, T, G, C), (far, G * C, C, 1))
    x = torch.randn(2, T, G, C, device="cuda").to(BF)
    view.copy_(x)
    for over in (tfla.NORM_TOKEN, tfla.NORM_SEQUENCE):
        want, m, r = tfla.norm_forward(x, act=tfla.ACT_SILU, over=over)
        got, _, _ = tfla.norm_forward(view, act=tfla.ACT_SILU, over=over, y=out)
        assert torch.equal(got, want)
        g = tfla.norm_backward(x, x, m, r, act=tfla.ACT_SILU, over=over)[0]
        assert torch.equal(tfla.norm_backward(view, view, m, r, act=tfla.ACT_SILU, over=over, dx=out)[0], g)
    torch.cuda.synchronize()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_a_very_long_sequence(dtype):
    check(dtype, 1, 100000, 2, 8, sequence=True)


@pytest.mark.parametrize("gated", [False, True])
def test_parameter_gradients_of_a_large_call(gated):
    """dweight and dbias of a call whose loads go past the caches, against sums in 64 bits; bounds as in check()."""
    B, T, G, C = 2, 8192, 32, 256
    x, dy = (torch.randn(B, T, G, C, device="cuda", dtype=BF) for _ in range(2))
    z = torch.randn(B, T, G, C, device="cuda", dtype=BF) if gated else None
    w, b = torch.randn(G, C, device="cuda"), torch.randn(G, C, device="cuda")
    kw = dict(act=tfla.ACT_SILU, gate=z)
    _, mean, rstd = tfla.norm_forward(x, w, b, eps=EPS, **kw)
    got = tfla.norm_backward(x, dy, mean, rstd, w, b, **kw)[2:]
    want, off = (torch.zeros(2, G, C, dtype=torch.float64, device="cuda") for _ in range(2))
    N, rows = (C + 60) * U, (B * T + 60) * U
    W, bias = w.double(), b.double()
    for i in range(B):
        v, g = x[i].double(), dy[i].double()
        m = v.mean(-1, keepdim=True)
        var = ((v - m) ** 2).mean(-1, keepdim=True)
        r = 1.0 / (var + EPS).sqrt()
        xh = (v - m) * r
        em = N * v.abs().mean(-1, keepdim=True)
        er = 0.5 * (2 * N * var + 4 * var.sqrt() * em + em ** 2) / (var + EPS) + 4 * U
        exh = r * (2 * U * (v.abs() + m.abs()) + em) + xh.abs() * er
        u = xh * W + bias
        at = z[i].double() if gated else u
        s = torch.sigmoid(at)
        if gated:
            du = g * at * s
            edu = 13 * U * du.abs()
        else:
            du = g * s * (1 + at * (1 - s))
            edu = g.abs() * (0.5 * (W.abs() * exh + 3 * U * ((xh * W).abs() + bias.abs())) + 12 * U)
        want[0] += (du * xh).sum(0)
        want[1] += du.sum(0)
        off[0] += (edu * xh.abs() + du.abs() * exh + rows * (du * xh).abs()).sum(0)
        off[1] += (edu + rows * du.abs()).sum(0)
    torch.cuda.synchronize()
    for name, p, q, tol in zip(("dweight", "dbias"), got, want, off):
        assert float(tol.max()) < 0.1 * float(q.abs().max()), name   # the bound tells a wrong sum from a right one
        within(name, p, q.cpu().numpy(), tol.cpu().numpy())


# rows of more than 1024 vectors, or single elements, go through memory; their weights' gradients in runs of 64 tokens
@pytest.mark.parametrize("dtype,C", [(BF, 1025), (BF, 1031), (BF, 8200), (F32, 1031), (F32, 4100)])
@pytest.mark.parametrize("kind,gated", [("none", False), ("sigmoid", False), ("silu", True), ("sigmoid", True), ("none", True)])
@pytest.mark.parametrize("B,T", [(1, 64), (1, 65), (2, 65)])
def test_rows_walked_from_memory(dtype, C, kind, gated, B, T):
    check(dtype, B, T, 2, C, kind=kind, gated=gated)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("C", [1024, 1032, 2048])
@pytest.mark.parametrize("gated", [False, True])
def test_wide_rows_without_wide_alignment(dtype, C, gated):
    """Single elements where rows are one element longer: a workgroup's registers up to 1024, memory beyond."""
    check(dtype, 2, 33, 2, C, gated=gated, layout="odd")


@pytest.mark.parametrize("dtype", [BF, F32])
def test_rows_walked_from_memory_without_weights(dtype):
    check(dtype, 2, 40, 1, 8200, affine=False, gated=dtype == BF)
