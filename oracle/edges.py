"""64-bit references of the operators at a block's edges and beside the
recurrences (numpy): rotary positions, gated linear recurrence of channels,
residual sum with a layer or RMS norm, each with its gradients written out
from the formulas.  Slow and plain; used by the tests only.

Arrays are float64 with channels last; ``lengths`` is None or one count of
valid rows per sequence: rows behind it are absent, and outputs and gradients
there are 0.
"""
from __future__ import annotations

import numpy as np

from .blocks import _lens, sigmoid


# ---- rotary positions --------------------------------------------------------------

def rotary(x, pos, freqs, interleaved=False, scale=1.0, lengths=None, inverse=False):
    """x [B,T,H,C], pos [B,T], freqs [R/2]: pairs as complex numbers times scale e^{i pos freq}."""
    B, T, _, C = x.shape
    R = 2 * len(freqs)
    y = x.copy()
    turn = scale * np.exp((-1j if inverse else 1j) * pos[:, :, None, None].astype(np.float64) * freqs)
    a, b = (x[..., 0:R:2], x[..., 1:R:2]) if interleaved else (x[..., :R // 2], x[..., R // 2:R])
    z = (a + 1j * b) * turn
    if interleaved:
        y[..., 0:R:2], y[..., 1:R:2] = z.real, z.imag
    else:
        y[..., :R // 2], y[..., R // 2:R] = z.real, z.imag
    for i, n in enumerate(_lens(lengths, B, T)):
        y[i, n:] = 0
    return y


# ---- gated linear recurrence of channels ---------------------------------------------

def diag_gates(fg, ig, decay, kind):
    """(f, i)"""
    if kind == "coupled":
        return sigmoid(fg), sigmoid(-fg)
    if kind == "sigmoid":
        return sigmoid(fg), sigmoid(ig)
    w = decay * sigmoid(fg)
    return np.exp(-w), np.sqrt(-np.expm1(-2 * w)) * sigmoid(ig)


def diag(x, fg, ig=None, decay=None, kind="coupled", state=None, lengths=None):
    """(y, state_out, states before every row)"""
    B, T, D = x.shape
    f, i = diag_gates(fg, ig, decay, kind)
    y, before, end = np.zeros_like(x), np.zeros_like(x), np.zeros((B, D))
    for b, n in enumerate(_lens(lengths, B, T)):
        h = np.zeros(D) if state is None else state[b]
        for t in range(n):
            before[b, t] = h
            h = f[b, t] * h + i[b, t] * x[b, t]
            y[b, t] = h
        before[b, n:] = h
        end[b] = h
    return y, end, before


def diag_grads(x, fg, dy, ig=None, decay=None, kind="coupled", state=None, lengths=None, dend=None):
    """dict of dx, dfgate, digate, ddecay, dstate"""
    B, T, D = x.shape
    f, i = diag_gates(fg, ig, decay, kind)
    _, _, before = diag(x, fg, ig, decay, kind, state, lengths)
    g = np.zeros_like(x)
    dstate = np.zeros((B, D))
    for b, n in enumerate(_lens(lengths, B, T)):
        a = np.zeros(D) if dend is None else dend[b]
        for t in range(n - 1, -1, -1):
            g[b, t] = dy[b, t] + a
            a = f[b, t] * g[b, t]
        dstate[b] = a
    live = np.zeros((B, T, 1), dtype=bool)
    for b, n in enumerate(_lens(lengths, B, T)):
        live[b, :n] = True
    xs = np.where(live, x, 0.0)
    df, di = g * before, g * xs
    r = sigmoid(fg)
    out = dict(dx=g * i, dstate=dstate, digate=None, ddecay=None)
    if kind == "coupled":
        out["dfgate"] = (df - di) * r * sigmoid(-fg)
    elif kind == "sigmoid":
        out["dfgate"], out["digate"] = df * r * sigmoid(-fg), di * i * sigmoid(-ig)
    else:
        w, s = decay * r, sigmoid(ig)
        m = np.sqrt(-np.expm1(-2 * w))
        with np.errstate(divide="ignore", invalid="ignore"):
            dm = np.where(m > 0, f * f / m, 0.0)
        dw = di * s * dm - df * f
        out.update(dfgate=dw * w * sigmoid(-fg), digate=di * i * sigmoid(-ig), ddecay=(dw * r).sum((0, 1)))
    for k in ("dx", "dfgate", "digate"):
        if out[k] is not None:
            out[k] = np.where(live, out[k], 0.0)
    return out


# ---- residual sum with a norm -----------------------------------------------------------

def addnorm(x, residual=None, weight=None, bias=None, eps=1e-5, rms=False):
    """(y, total)"""
    t = x if residual is None else x + residual
    d = t if rms else t - t.mean(-1, keepdims=True)
    th = d / np.sqrt((d * d).mean(-1, keepdims=True) + eps)
    return th * (1.0 if weight is None else weight) + (0.0 if bias is None else bias), t


def addnorm_grads(total, dy, weight=None, eps=1e-5, rms=False, dtotal=None):
    """(gradient of the sum, dweight, dbias)"""
    d = total if rms else total - total.mean(-1, keepdims=True)
    r = 1.0 / np.sqrt((d * d).mean(-1, keepdims=True) + eps)
    th, v = d * r, dy * (1.0 if weight is None else weight)
    dt = v - th * (v * th).mean(-1, keepdims=True)
    if not rms:
        dt = dt - v.mean(-1, keepdims=True)
    return r * dt + (0.0 if dtotal is None else dtotal), (dy * th).sum((0, 1)), dy.sum((0, 1))
