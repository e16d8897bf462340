"""The 64-bit references of rotary positions, the gated linear recurrence of
channels and the residual sum with a norm: every gradient against central
differences of the forward formula, carried states against one long call,
padded rows without influence, and frequencies against their definitions."""
import math

import numpy as np
import pytest
import torch

from mlstm_sequence_amd import tfla
from oracle import edges as O
from test_blocks_oracle import check_grads


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("lengths", [None, [0, 3]])
def test_rotary_gradient_and_angle(interleaved, lengths):
    rng = np.random.default_rng(1)
    B, T, H, C, R = 2, 3, 2, 7, 6
    x, dy = rng.standard_normal((2, B, T, H, C))
    pos, freqs = rng.integers(-5, 1000, (B, T)), rng.random(R // 2)
    kw = dict(pos=pos, freqs=freqs, interleaved=interleaved, scale=1.3, lengths=lengths)
    check_grads(lambda x: (O.rotary(x, **kw) * dy).sum(), dict(x=x), dict(x=O.rotary(dy, inverse=True, **kw)))
    # lengths of pairs are kept up to the scale, and angles add up
    y = O.rotary(x, pos, freqs, interleaved)
    assert np.allclose(np.square(y).sum(-1), np.square(x).sum(-1), rtol=1e-13)
    twice = O.rotary(y, pos, freqs, interleaved)
    assert np.allclose(twice, O.rotary(x, 2 * pos, freqs, interleaved), atol=1e-11)
    # one pair by hand
    a, b = (x[0, 1, 0, 2], x[0, 1, 0, 3]) if interleaved else (x[0, 1, 0, 1], x[0, 1, 0, 4])
    th = float(pos[0, 1] * freqs[1])
    got = (y[0, 1, 0, 2], y[0, 1, 0, 3]) if interleaved else (y[0, 1, 0, 1], y[0, 1, 0, 4])
    assert np.allclose(got, (a * math.cos(th) - b * math.sin(th), b * math.cos(th) + a * math.sin(th)), atol=1e-12)


@pytest.mark.parametrize("kind", ["coupled", "sigmoid", "decay"])
@pytest.mark.parametrize("lengths", [None, [4, 0, 2]])
def test_diag_gradients(kind, lengths):
    rng = np.random.default_rng(3)
    B, T, D = 3, 5, 2
    a = dict(x=rng.standard_normal((B, T, D)), fg=rng.standard_normal((B, T, D)), state=rng.standard_normal((B, D)))
    if kind != "coupled":
        a["ig"] = rng.standard_normal((B, T, D))
    if kind == "decay":
        a["decay"] = rng.random(D) + 0.1
    dy, dend = rng.standard_normal((B, T, D)), rng.standard_normal((B, D))

    def loss(**k):
        y, e, _ = O.diag(kind=kind, lengths=lengths, **k)
        return (y * dy).sum() + (e * dend).sum()

    g = O.diag_grads(dy=dy, kind=kind, lengths=lengths, dend=dend, **a)
    names = dict(x="dx", fg="dfgate", ig="digate", decay="ddecay", state="dstate")
    check_grads(loss, a, {k: g[names[k]] for k in a})


def test_diag_by_hand_and_continued():
    x, fg = np.array([[[1.0], [2.0]]]), np.array([[[0.0], [math.log(3.0)]]])
    y, end, before = O.diag(x, fg)                       # f = 1/2, 3/4
    assert np.allclose(y[0, :, 0], [0.5, 0.75 * 0.5 + 0.25 * 2.0]) and before[0, 1, 0] == y[0, 0, 0]
    rng = np.random.default_rng(0)
    x, fg, ig = rng.standard_normal((3, 2, 9, 3))
    y, end, _ = O.diag(x, fg, ig, None, "sigmoid")
    y1, s, _ = O.diag(x[:, :4], fg[:, :4], ig[:, :4], None, "sigmoid")
    y2, s, _ = O.diag(x[:, 4:], fg[:, 4:], ig[:, 4:], None, "sigmoid", state=s)
    assert np.array_equal(np.concatenate([y1, y2], 1), y) and np.array_equal(s, end)


def test_diag_padded_rows_have_no_influence():
    rng = np.random.default_rng(4)
    x, fg, dy = rng.standard_normal((3, 2, 6, 3))
    short = O.diag_grads(x, fg, dy, lengths=[6, 2])
    for v in (x, fg, dy):
        v[1, 2:] = np.nan
    with np.errstate(invalid="ignore"):
        again = O.diag_grads(x, fg, dy, lengths=[6, 2])
    for k in ("dx", "dfgate", "dstate"):
        assert np.array_equal(short[k], again[k])


@pytest.mark.parametrize("rms", [False, True])
def test_addnorm_gradients(rms):
    rng = np.random.default_rng(6)
    B, T, C = 2, 3, 5
    a = dict(x=rng.standard_normal((B, T, C)), residual=rng.standard_normal((B, T, C)), weight=rng.standard_normal(C),
             bias=rng.standard_normal(C))
    dy, dt = rng.standard_normal((2, B, T, C))

    def loss(**k):
        y, t = O.addnorm(rms=rms, **k)
        return (y * dy).sum() + (t * dt).sum()

    g, dw, db = O.addnorm_grads(a["x"] + a["residual"], dy, a["weight"], rms=rms, dtotal=dt)
    check_grads(loss, a, dict(x=g, residual=g, weight=dw, bias=db))
    y, t = O.addnorm(**a)
    xh = (y - a["bias"]) / a["weight"]
    assert np.allclose(xh.mean(-1), 0, atol=1e-12) and np.array_equal(t, a["x"] + a["residual"])


def test_frequencies():
    f, s = tfla.rotary_frequencies(8, device="cpu")
    assert f.dtype == torch.float64 and s == 1.0
    assert np.allclose(f.numpy(), [1.0, 0.1, 0.01, 0.001], rtol=1e-14)
    assert np.allclose(tfla.rotary_frequencies(8, scaling="linear", factor=4.0, device="cpu")[0].numpy(), f.numpy() / 4)
    n, _ = tfla.rotary_frequencies(8, scaling="ntk", factor=4.0, device="cpu")
    assert np.allclose([n[0], n[3]], [1.0, 0.001 / 4], rtol=1e-14)         # the fastest stays, the slowest is divided
    y, s = tfla.rotary_frequencies(8, scaling="yarn", factor=4.0, original_length=4096, device="cpu")
    turns = 4096 * f.numpy() / (2 * math.pi)                                 # 652, 65, 6.5, 0.65
    keep = [1.0, 1.0, (turns[2] - 1) / 31, 0.0]
    assert np.allclose(y.numpy(), [k * v + (1 - k) * v / 4 for k, v in zip(keep, f.numpy())], rtol=1e-14)
    assert abs(s - (0.1 * math.log(4.0) + 1)) < 1e-15
    for dim in (0, 2):
        for kind in ("none", "linear", "ntk", "yarn"):
            assert tfla.rotary_frequencies(dim, scaling=kind, factor=2.0, original_length=10, device="cpu")[0].shape == (dim // 2,)
    for bad in (dict(dim=7), dict(dim=-2), dict(dim=8, base=0.0), dict(dim=8, base=float("inf")), dict(dim=8, scaling="other"),
                dict(dim=8, factor=0.5), dict(dim=8, factor=float("nan")), dict(dim=8, scaling="yarn"),
                dict(dim=8, scaling="yarn", original_length=100, slow=4.0, fast=4.0)):
        with pytest.raises(ValueError):
            tfla.rotary_frequencies(**bad, device="cpu")
