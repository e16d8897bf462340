"""The 64-bit references of the operators around the recurrences: every
gradient against central differences of the forward formula, the carried
state against one long call, and padded rows without influence."""
import numpy as np
import pytest

from oracle import blocks as O

# central differences in 64 bits with step h: truncation h^2 f''' / 6 and rounding eps f / h,
# both below 1e-8 for values of order 1 at h = 1e-5
H, TOL = 1e-5, 2e-7


def check_grads(loss, args, grads):
    """d loss(args) / d args[k] against grads[k] for every key of grads, in random directions."""
    rng = np.random.default_rng(5)
    for k, g in grads.items():
        for _ in range(3):
            v = rng.standard_normal(args[k].shape)
            hi, lo = dict(args), dict(args)
            hi[k], lo[k] = args[k] + H * v, args[k] - H * v
            num = (loss(**hi) - loss(**lo)) / (2 * H)
            ana = float((g * v).sum())
            assert abs(num - ana) <= TOL * max(1.0, abs(ana)) * 10, (k, num, ana)


@pytest.mark.parametrize("K,kind,lengths", [(4, "silu", None), (1, "none", None), (3, "silu", [5, 0, 1]), (6, "none", [2, 5, 4])])
def test_conv_gradients(K, kind, lengths):
    rng = np.random.default_rng(K)
    B, T, D = 3, 5, 2
    a = dict(x=rng.standard_normal((B, T, D)), w=rng.standard_normal((D, K)), bias=rng.standard_normal(D),
             state=rng.standard_normal((B, K - 1, D)))
    dy, dend = rng.standard_normal((B, T, D)), rng.standard_normal((B, K - 1, D))

    def loss(x, w, bias, state):
        y, e = O.conv(x, w, bias, kind, state, lengths)
        return (y * dy).sum() + (e * dend).sum()

    dx, dw, db, ds = O.conv_grads(a["x"], a["w"], dy, a["bias"], kind, a["state"], lengths, dend)
    check_grads(loss, a, dict(x=dx, w=dw, bias=db, state=ds))


def test_conv_state_continues():
    rng = np.random.default_rng(1)
    x, w = rng.standard_normal((2, 9, 3)), rng.standard_normal((3, 4))
    y, end = O.conv(x, w)
    y1, s = O.conv(x[:, :2], w)
    y2, s = O.conv(x[:, 2:], w, state=s)
    assert np.array_equal(np.concatenate([y1, y2], 1), y) and np.array_equal(s, end)


@pytest.mark.parametrize("G,gated,softplus,lengths", [(1, True, True, None), (2, False, False, [0, 4]), (2, True, True, [1, 3])])
def test_scan_gradients(G, gated, softplus, lengths):
    rng = np.random.default_rng(7 + G)
    B, T, D, N = 2, 4, 4, 3
    a = dict(x=rng.standard_normal((B, T, D)), dt=rng.standard_normal((B, T, D)), a=-np.exp(rng.standard_normal((D, N))),
             bm=rng.standard_normal((B, T, G, N)), cm=rng.standard_normal((B, T, G, N)), skip=rng.standard_normal(D),
             dt_bias=rng.standard_normal(D), state=rng.standard_normal((B, D, N)))
    if gated:
        a["z"] = rng.standard_normal((B, T, D))
    dy, dend = rng.standard_normal((B, T, D)), rng.standard_normal((B, D, N))

    def loss(**k):
        y, e = O.scan(softplus=softplus, lengths=lengths, **k)
        return (y * dy).sum() + (e * dend).sum()

    g = O.scan_grads(dout=dy, softplus=softplus, lengths=lengths, dend=dend, **a)
    names = dict(x="dx", dt="ddt", a="da", bm="dbmat", cm="dcmat", skip="dskip", dt_bias="ddt_bias", state="dstate", z="dz")
    check_grads(loss, a, {k: g[names[k]] for k in a})


def test_scan_state_continues():
    rng = np.random.default_rng(2)
    B, T, D, N = 2, 7, 3, 4
    x, dt = rng.standard_normal((2, B, T, D))
    bm, cm = rng.standard_normal((2, B, T, 1, N))
    a = -np.exp(rng.standard_normal((D, N)))
    y, end = O.scan(x, dt, a, bm, cm)
    y1, s = O.scan(x[:, :3], dt[:, :3], a, bm[:, :3], cm[:, :3])
    y2, s = O.scan(x[:, 3:], dt[:, 3:], a, bm[:, 3:], cm[:, 3:], state=s)
    assert np.array_equal(np.concatenate([y1, y2], 1), y) and np.array_equal(s, end)


@pytest.mark.parametrize("sequence", [False, True])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("kind", ["none", "silu", "sigmoid"])
def test_norm_gradients(sequence, gated, kind):
    rng = np.random.default_rng(11)
    B, T, G, C = 2, 3, 2, 4
    a = dict(x=rng.standard_normal((B, T, G, C)) + 1, w=rng.standard_normal((G, C)), bias=rng.standard_normal((G, C)))
    if gated:
        a["gate"] = rng.standard_normal((B, T, G, C))
    dy = rng.standard_normal((B, T, G, C))

    def loss(**k):
        return (O.norm(kind=kind, sequence=sequence, **k)[0] * dy).sum()

    dx, dg, dw, db = O.norm_grads(dy=dy, kind=kind, sequence=sequence, **a)
    check_grads(loss, a, {k: v for k, v in dict(x=dx, gate=dg, w=dw, bias=db).items() if v is not None})
