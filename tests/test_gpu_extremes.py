"""The operators around the recurrences at gates, pre-activations and steps
where the activations' exponential over- or underflows, against the 64-bit
reference.

Error bounds, with U half a step of fp32.  The sigmoid s of u: the
exponential's argument is rounded (|u| U relative, of e^-u) and 1 + e^-u, its
reciprocal and the exponential are off by 6 U; from u = 17 on fp32 holds 1,
which e^-u is then the distance from; a result below 2^-125 may be 0.  So

  es  = (|u| + 6) U min(s, 2^25 e^-u) + s where s < 2^-125
  SiLU u s:              |u| es + 2 U |u s|
  its slope s + u s (1 - s), 1 - s exact from s = 1/2 on:
                         es (1 + |u|) + |u| s (es + U where s < 1/2) + 4 U (s + |u| s (1 - s))
  sigmoid's slope:       es + s (es + U where s < 1/2) + 2 U s (1 - s)

and an error du of u itself changes a value by at most its slope's largest
absolute value within du, e^-w (1 + |u| + du) for the side below zero, a
slope by e^-w (2 + |u| + du) with w = |u| - du, both at most about 1."""
import numpy as np
import pytest
import torch

from blocks_helpers import HALF, U, randn, within
from mlstm_sequence_amd import tfla
from oracle import blocks as O

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
ACT = {"none": tfla.ACT_NONE, "silu": tfla.ACT_SILU, "sigmoid": tfla.ACT_SIGMOID}
# e^-u overflows fp32 from u = -88.8 on; near there, its double and far beyond
NEGATIVE = [-80.0, -87.0, -88.0, -88.5, -89.0, -95.0, -100.0, -120.0, -150.0, -177.0, -178.0, -200.0, -1000.0, -1e4]
TINY = 2.0 ** -126   # fp32 results below may be 0


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    tfla.lib()


def extremes(dtype, signs):
    """Values to plant: "negative" with the lowest finite one, "both" with their mirrors instead of it."""
    low = torch.finfo(dtype).min
    return NEGATIVE + [low] if signs == "negative" else NEGATIVE + [-v for v in NEGATIVE]


def act_bounds(u, kind, du=0.0):
    """(f, f', error of f, error of f') at the computed u, off by up to `du`."""
    if kind == "none":
        return u, np.ones_like(u), np.zeros_like(u) + du, np.zeros_like(u)
    with np.errstate(all="ignore"):
        s = O.sigmoid(u)
        a = np.abs(u)
        far = np.minimum(s, 2.0 ** 25 * np.exp(-u))
        es = np.where(far > 0, (a + 6) * U * far, 0.0) + np.where(s < 2.0 ** -125, s, 0.0)
        low = np.where(s < 0.5, U, 0.0)
        w = np.exp(-np.maximum(a - du, 0.0))
        us, ues = np.where(s > 0, a * s, 0.0), np.where(es > 0, a * es, 0.0)   # 0 where u is -inf
        if kind == "sigmoid":
            f, df = s, s * (1 - s)
            ef = es + np.where(w > 0, np.minimum(0.25, w) * du, 0.0)
            edf = es + s * (es + low) + 2 * U * df + np.where(w > 0, np.minimum(0.1, w) * du, 0.0)
        else:
            f, df = np.sign(u) * us, s + np.sign(u) * us * (1 - s)
            below = np.exp(np.minimum(u + du, 0.0))
            ef = ues + 2 * U * us + np.where(below > 0, np.minimum(1.1, (1 + a + du) * below) * du, 0.0)
            edf = (es + ues) + us * (es + low) + 4 * U * (s + us * (1 - s)) + np.where(w > 0, np.minimum(0.5, (2 + a + du) * w) * du, 0.0)
    return f, df, ef, edf


def test_bounds_cover_the_reference():
    """The bounds' own f and f' are the reference's."""
    u = np.array(NEGATIVE + [-v for v in NEGATIVE] + [0.0, 1.0, -1.28])
    for kind in ("silu", "sigmoid"):
        f, df = O.act(u, kind)
        g, dg, ef, edf = act_bounds(u, kind)
        assert np.allclose(f, g, rtol=1e-12, atol=0) and np.allclose(df, dg, rtol=1e-9, atol=1e-300)
        assert np.isfinite(ef).all() and np.isfinite(edf).all()
        assert (ef <= 1e-4 * np.abs(f) + 1e-34).all()


# ---- convolution --------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("signs", ["negative", "both"])
@pytest.mark.parametrize("K", [1, 4])
@pytest.mark.parametrize("lengths", [None, [14, 6]])
def test_convolution(dtype, signs, K, lengths):
    """One row of each channel (in two sequences) is an extreme value; neighbouring rows meet it through the taps."""
    B, T = 2, 14
    E = extremes(dtype, signs)
    D = 5 * len(E)
    rng = np.random.default_rng(K)
    x = torch.from_numpy(rng.standard_normal((B, T, D))).to(dtype)
    for c in range(D):
        x[0, 5, c] = x[1, 3, c] = E[c % len(E)]
    w = torch.from_numpy(rng.uniform(0.05, 0.3, (D, K)) * rng.choice([-1.0, 1.0], (D, K))).float()
    w[:, K - 1] = 1.0
    dy = torch.from_numpy(rng.uniform(-0.2, 0.2, (B, T, D))).to(dtype)   # so that products with the lowest value stay finite
    ln = None if lengths is None else torch.tensor(lengths, dtype=torch.int32).cuda()
    y, _ = tfla.conv_forward(x.cuda(), w.cuda(), lengths=ln)
    dx, dw, _, _ = tfla.conv_backward(x.cuda(), w.cuda(), dy.cuda(), lengths=ln)
    torch.cuda.synchronize()

    X, W, G = x.double().numpy(), w.double().numpy(), dy.double().numpy()
    u, _ = O.conv(X, W, kind="none", lengths=lengths)
    mag, _ = O.conv(np.abs(X), np.abs(W), kind="none", lengths=lengths)
    du = np.zeros_like(u) if K == 1 else (K + 1) * U * mag   # a single product with weight 1 is exact
    f, df, ef, edf = act_bounds(u, "silu", du)
    want, _ = O.conv(X, W, lengths=lengths)
    h = HALF[dtype]
    within("y", y, want, h * np.abs(want) + ef + TINY)
    gx, gw, _, _ = O.conv_grads(X, W, G, lengths=lengths)
    # sums of K (dx) and B T (dw) products of du = dy f'
    term, off = np.abs(G * df), np.abs(G) * edf + TINY
    mx, mw, _, _ = O.conv_grads(np.abs(X), np.abs(W), term, kind="none", lengths=lengths)
    ex, ew, _, _ = O.conv_grads(np.abs(X), np.abs(W), off, kind="none", lengths=lengths)
    within("dx", dx, gx, h * np.abs(gx) + (K + 3) * U * mx + ex + TINY)
    within("dweight", dw, gw, (B * T + 16) * U * mw + ew + TINY)


# ---- scan ------------------------------------------------------------------------------------

def scan_case(dtype, B, T, D, N, seed=0):
    rng = np.random.default_rng(seed + T)
    d = dict(x=randn(rng, (B, T, D), dtype)[0], dt=randn(rng, (B, T, D), dtype, 1.0, -1.0)[0],
             a=-torch.exp(randn(rng, (D, N), F32, 0.3)[0]), bmat=randn(rng, (B, T, 1, N), dtype)[0],
             cmat=randn(rng, (B, T, 1, N), dtype)[0], skip=randn(rng, (D,), F32)[0], z=randn(rng, (B, T, D), dtype, 2.0)[0],
             dt_bias=randn(rng, (D,), F32, 0.5)[0], state=randn(rng, (B, D, N), F32)[0], dy=randn(rng, (B, T, D), dtype)[0],
             dend=randn(rng, (B, D, N), F32)[0])
    return d


def scan_check(dtype, d, floor):
    """Every output of both directions.  A product of decays is off by the sum of rho = |delta a| (e + 4 U) + 3 U over
    the steps, twice in the backward pass, e the relative error of delta = softplus(u): half a step of the rounded sum u
    through the slope, 8 U, and where u is below 17 the exponential's rounded argument, 2 |u| U.  Beyond |delta a| = 104
    a decay is 0 in fp32, and u below -104 gives a delta of 0: both count to `floor`.  A gate's sigmoid is within
    110 U of itself down to z = -104, and 0 below (`floor`); it enters a product at most twice."""
    B, T, D = d["x"].shape
    N = d["a"].shape[1]
    g = {k: v.cuda() for k, v in d.items()}
    kw = dict(skip=g["skip"], z=g["z"], dt_bias=g["dt_bias"], state=g["state"])
    args = (g["x"], g["dt"], g["a"], g["bmat"], g["cmat"])
    y, end = tfla.scan_forward(*args, want_state=True, **kw)
    o = tfla.scan_backward(*args, g["dy"], dstate_out=g["dend"], **kw)
    torch.cuda.synchronize()
    r = {k: v.double().numpy() for k, v in d.items()}
    rk = dict(x=r["x"], dt=r["dt"], a=r["a"], bm=r["bmat"], cm=r["cmat"], dout=r["dy"], skip=r["skip"], z=r["z"],
              dt_bias=r["dt_bias"], state=r["state"], dend=r["dend"])
    want, mag = O.scan_grads(**rk), O.scan_grads(magnitude=True, **rk)
    u = r["dt"] + r["dt_bias"]
    delta, slope = O._delta(r["dt"], r["dt_bias"], True)
    e = slope * U * (np.abs(r["dt"]) + np.abs(r["dt_bias"])) / delta + (8 + np.where(u < 17, 2 * np.minimum(np.abs(u), 104), 0)) * U
    rho = np.minimum(delta * np.abs(r["a"]).max(1), 104) * (e + 4 * U) + 3 * U
    rel = 2 * rho.sum(1).max() + 2 * e.max() + (100 + 220) * U
    h = HALF[dtype]
    for name, got, n, half in (("y", y, N, h), ("end", end, T, 0.0), ("dx", o.dx, N, h), ("ddt", o.ddt, 2 * N, h),
                               ("dz", o.dz, N, h), ("dbmat", o.dbmat, D, h), ("dcmat", o.dcmat, D, h),
                               ("da", o.da, B * T, 0.0), ("dskip", o.dskip, B * T, 0.0),
                               ("ddt_bias", o.ddt_bias, B * T * N, 0.0), ("dstate", o.dstate, T, 0.0)):
        within(name, got, want[name], half * np.abs(want[name]) + (rel + (n + 1) * U) * mag[name] + floor)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("signs", ["negative", "both"])
@pytest.mark.parametrize("T", [1, 3, 40, 200])
def test_scan_gates(dtype, signs, T):
    """Some rows' gates are extreme values.  T: the step kernel, one segment, several."""
    E = extremes(dtype, signs)
    d = scan_case(dtype, 2, T, 4 * len(E), 8)
    for c in range(d["z"].shape[2]):
        d["z"][:, T // 2, c] = d["z"][0, T - 1, c] = E[c % len(E)]
    # sigmoids below 2^-125 times gates of up to 105, and terms' magnitudes of at most 1e6
    scan_check(dtype, d, 1e-29)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T", [40, 700])
def test_scan_steps(dtype, T):
    """Steps from 0 to so large that every decay is 0, gated, both directions; T = 700 is cut into segments, some of
    which lie in one kind of step."""
    d = scan_case(dtype, 1, T, 64, 8)
    dt = d["dt"]
    for lo in range(0, T, 100):
        dt[:, lo + 5:lo + 10], dt[:, lo + 10:lo + 15], dt[:, lo + 15:lo + 20] = -200.0, 200.0, 5000.0
    if T > 500:
        dt[:, 420:490] = -200.0
        dt[:, 520:590] = 5000.0
    # decays below 2^-126 are 0: 1.2e-38 times states (5000 x b), steps (5000), gates, factors of order 10 and T terms
    scan_check(dtype, d, 1e-25)


# ---- norm -------------------------------------------------------------------------------------

def norm_check(dtype, x, w, b, z, dy, kind, sequence):
    """The bounds of mean, rstd and xh are those of test_gpu_norm.py."""
    B, T, G, C = x.shape
    cu = lambda t: None if t is None else t.cuda()  # noqa: E731
    kw = dict(act=ACT[kind], gate=cu(z), over=tfla.NORM_SEQUENCE if sequence else tfla.NORM_TOKEN)
    eps = 1e-5
    y, mean, rstd = tfla.norm_forward(x.cuda(), cu(w), cu(b), eps=eps, **kw)
    dx, dz, dw, db = tfla.norm_backward(x.cuda(), dy.cuda(), mean, rstd, cu(w), cu(b), **kw)
    torch.cuda.synchronize()
    x, w, b, dy = (t.double().numpy() for t in (x, w, b, dy))
    z = None if z is None else z.double().numpy()
    dims = (1, 3) if sequence else (3,)
    n = C * (T if sequence else 1)
    N = (n + 60) * U
    m = x.mean(dims, keepdims=True)
    var = ((x - m) ** 2).mean(dims, keepdims=True)
    r = 1.0 / np.sqrt(var + eps)
    xh = (x - m) * r
    em = N * np.abs(x).mean(dims, keepdims=True)
    er = 0.5 * (2 * N * var + 4 * np.sqrt(var) * em + em ** 2) / (var + eps) + 4 * U
    exh = r * (2 * U * (np.abs(x) + np.abs(m)) + em) + np.abs(xh) * er
    W = np.abs(w)
    u = xh * w + b
    eu = W * exh + 3 * U * (np.abs(xh) * W + np.abs(b))
    h = HALF[dtype]
    if z is not None:
        f, df, ef, edf = act_bounds(z, kind)
        wy, ey = u * f, np.abs(f) * eu + np.abs(u) * ef + 2 * U * np.abs(u * f)
        wdz = dy * u * df
        within("dgate", dz, wdz, h * np.abs(wdz) + np.abs(dy * df) * eu + np.abs(dy * u) * edf + 3 * U * np.abs(wdz) + TINY)
        du, edu = dy * f, np.abs(dy) * ef + 2 * U * np.abs(dy * f)
    else:
        f, df, ef, edf = act_bounds(u, kind, eu)
        wy, ey = f, ef
        du, edu = dy * df, np.abs(dy) * edf + 2 * U * np.abs(dy * df)
    within("y", y, wy, h * np.abs(wy) + ey + TINY)
    v, ev = du * w, W * edu + 2 * U * np.abs(du) * W
    mv, mvx = v.mean(dims, keepdims=True), (v * xh).mean(dims, keepdims=True)
    emv = ev.mean(dims, keepdims=True) + N * np.abs(v).mean(dims, keepdims=True)
    emvx = (ev * np.abs(xh) + np.abs(v) * exh).mean(dims, keepdims=True) + N * np.abs(v * xh).mean(dims, keepdims=True)
    wdx = r * (v - mv - xh * mvx)
    edx = r * (ev + emv + np.abs(xh) * emvx + exh * np.abs(mvx)) + (er + 5 * U) * r * (np.abs(v) + np.abs(mv) + np.abs(xh * mvx))
    within("dx", dx, wdx, h * np.abs(wdx) + edx + 1e-35)
    rows = (B * T + 60) * U
    within("dweight", dw, (du * xh).sum((0, 1)),
           (edu * np.abs(xh) + np.abs(du) * exh).sum((0, 1)) + rows * np.abs(du * xh).sum((0, 1)) + 1e-35)
    within("dbias", db, du.sum((0, 1)), edu.sum((0, 1)) + rows * np.abs(du).sum((0, 1)) + 1e-35)


def norm_inputs(dtype, G, C, seed):
    rng = np.random.default_rng(seed)
    B, T = 2, 9
    return (randn(rng, (B, T, G, C), dtype, 2.0, 0.5)[0], randn(rng, (G, C), F32, 0.3, 1.0)[0], randn(rng, (G, C), F32, 0.3)[0],
            randn(rng, (B, T, G, C), dtype, 2.0)[0], randn(rng, (B, T, G, C), dtype)[0])


# a row in a wave (vectors, single elements), in a workgroup, and walked from memory
WIDTHS = [(BF, 64), (BF, 7), (BF, 1000), (BF, 1031), (F32, 64), (F32, 7), (F32, 1000), (F32, 4100)]


@pytest.mark.parametrize("dtype,C", WIDTHS)
@pytest.mark.parametrize("kind", ["silu", "sigmoid"])
@pytest.mark.parametrize("signs", ["negative", "both"])
@pytest.mark.parametrize("sequence", [False, True])
def test_norm_gates(dtype, C, kind, signs, sequence):
    x, w, b, z, dy = norm_inputs(dtype, 3, C, C)
    E = torch.tensor(extremes(dtype, signs) + ([float("-inf")] if kind == "sigmoid" else [])).to(dtype)
    at = torch.arange(z.numel()) % (2 * len(E))   # every other value or so, at places that change from row to row
    flat = z.view(-1)
    flat[at < len(E)] = E[at[at < len(E)]]
    norm_check(dtype, x, w, b, z, dy, kind, sequence)


@pytest.mark.parametrize("dtype,C", WIDTHS)
@pytest.mark.parametrize("kind", ["silu", "sigmoid"])
@pytest.mark.parametrize("signs", ["negative", "both"])
@pytest.mark.parametrize("sequence", [False, True])
def test_norm_activations(dtype, C, kind, signs, sequence):
    x, w, b, _, dy = norm_inputs(dtype, 3, C, C + 1)
    E = torch.tensor(extremes(F32, signs))
    at = torch.arange(b.numel()) % (2 * len(E))
    b.view(-1)[at < len(E)] = E[at[at < len(E)]]
    norm_check(dtype, x, w, b, None, dy, kind, sequence)


def test_masked_gates_leave_no_gradient():
    """Rows of padding: dy 0 and gates of the lowest value give gradients of 0."""
    x, w, b, z, dy = (t.cuda() for t in norm_inputs(F32, 3, 64, 5))
    for over in (tfla.NORM_TOKEN, tfla.NORM_SEQUENCE):
        for act in (tfla.ACT_SILU, tfla.ACT_SIGMOID):
            zz, gg = z.clone(), dy.clone()
            zz[:, 6:], gg[:, 6:] = torch.finfo(F32).min, 0.0
            y, mean, rstd = tfla.norm_forward(x, w, b, act=act, gate=zz, over=over)
            dx, dz, dw, db = tfla.norm_backward(x, gg, mean, rstd, w, b, act=act, gate=zz, over=over)
            torch.cuda.synchronize()
            assert bool((y[:, 6:] == 0).all()) and bool((dz[:, 6:] == 0).all())
            assert over == tfla.NORM_SEQUENCE or bool((dx[:, 6:] == 0).all())
            assert all(bool(torch.isfinite(t).all()) for t in (dx, dw, db))
