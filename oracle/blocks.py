"""64-bit references of the operators around the recurrences (numpy): causal
depthwise convolution, selective state space scan, group norm with an
activation or a gate, each with its gradients written out from the formulas.
Slow and plain; used by the tests only.

Arrays are float64 [B,T,...] with channels last; ``lengths`` is None or one
count of valid rows per sequence: rows behind it are absent, and outputs and
gradients there are 0.
"""
from __future__ import annotations

import numpy as np


def sigmoid(u):
    e = np.exp(-np.abs(u))
    return np.where(u >= 0, 1.0 / (1.0 + e), e / (1.0 + e))


def act(u, kind):
    """(f(u), f'(u)) of "none", "silu" or "sigmoid"."""
    if kind == "none":
        return u, np.ones_like(u)
    s = sigmoid(u)
    if kind == "sigmoid":
        return s, s * (1 - s)
    return u * s, s * (1 + u * (1 - s))


def _lens(lengths, B, T):
    return [T] * B if lengths is None else [min(max(int(n), 0), T) for n in lengths]


# ---- convolution -----------------------------------------------------------------

def conv(x, w, bias=None, kind="silu", state=None, lengths=None):
    """(y, state_out)"""
    B, T, D = x.shape
    K = w.shape[1]
    y, end = np.zeros_like(x), np.zeros((B, K - 1, D))
    for b, n in enumerate(_lens(lengths, B, T)):
        X = np.concatenate([np.zeros((K - 1, D)) if state is None else state[b], x[b, :n]])
        for t in range(n):
            u = np.einsum("kd,dk->d", X[t:t + K], w) + (0 if bias is None else bias)
            y[b, t] = act(u, kind)[0]
        end[b] = X[n:]
    return y, end


def conv_grads(x, w, dy, bias=None, kind="silu", state=None, lengths=None, dend=None):
    """(dx, dw, dbias, dstate)"""
    B, T, D = x.shape
    K = w.shape[1]
    dx, dw, db, ds = np.zeros_like(x), np.zeros_like(w), np.zeros(D), np.zeros((B, K - 1, D))
    for b, n in enumerate(_lens(lengths, B, T)):
        X = np.concatenate([np.zeros((K - 1, D)) if state is None else state[b], x[b, :n]])
        dX = np.zeros_like(X)
        for t in range(n):
            u = np.einsum("kd,dk->d", X[t:t + K], w) + (0 if bias is None else bias)
            du = dy[b, t] * act(u, kind)[1]
            dX[t:t + K] += du * w.T
            dw += (du * X[t:t + K]).T
            db += du
        if dend is not None:
            dX[n:] += dend[b]
        ds[b], dx[b, :n] = dX[:K - 1], dX[K - 1:]
    return dx, dw, db, ds


# ---- selective scan ------------------------------------------------------------------

def _delta(dt, dt_bias, softplus):
    u = dt + (0 if dt_bias is None else dt_bias)
    return (np.logaddexp(u, 0), sigmoid(u)) if softplus else (u, np.ones_like(u))


def scan(x, dt, a, bm, cm, skip=None, z=None, dt_bias=None, softplus=True, state=None, lengths=None):
    """(y, state_out); a [D,N], bm, cm [B,T,G,N]"""
    B, T, D = x.shape
    per = D // bm.shape[2]
    y = np.zeros_like(x)
    end = np.zeros((B,) + a.shape)
    for b, n in enumerate(_lens(lengths, B, T)):
        h = np.zeros(a.shape) if state is None else state[b].copy()
        d, _ = _delta(dt[b, :n], dt_bias, softplus)
        for t in range(n):
            Bt, Ct = np.repeat(bm[b, t], per, 0), np.repeat(cm[b, t], per, 0)
            h = np.exp(d[t][:, None] * a) * h + (d[t] * x[b, t])[:, None] * Bt
            o = (h * Ct).sum(1) + (0 if skip is None else skip * x[b, t])
            y[b, t] = o if z is None else o * act(z[b, t], "silu")[0]
        end[b] = h
    return y, end


def scan_grads(x, dt, a, bm, cm, dout, skip=None, z=None, dt_bias=None, softplus=True, state=None, lengths=None,
               dend=None, magnitude=False):
    """dict of y, end, dx, ddt, da, dbmat, dcmat, dskip, dz, ddt_bias, dstate;
    with ``magnitude`` the sums of the terms' absolute values instead (for
    error bounds)."""
    B, T, D = x.shape
    mag = np.abs if magnitude else (lambda v: v)
    x, bm, cm, dout = mag(x), mag(bm), mag(cm), mag(dout)
    skip, state, dend = (None if v is None else mag(v) for v in (skip, state, dend))
    G = bm.shape[2]
    per = D // G
    o = dict(dx=np.zeros_like(x), ddt=np.zeros_like(x), da=np.zeros_like(a), dbmat=np.zeros_like(bm),
             dcmat=np.zeros_like(cm), dskip=np.zeros(D), dz=np.zeros_like(x), ddt_bias=np.zeros(D),
             dstate=np.zeros((B,) + a.shape), y=np.zeros_like(x), end=np.zeros((B,) + a.shape))
    for b, n in enumerate(_lens(lengths, B, T)):
        d, slope = _delta(dt[b, :n], dt_bias, softplus)
        dm = mag(d)
        hs = [np.zeros(a.shape) if state is None else state[b]]
        for t in range(n):
            Bt = np.repeat(bm[b, t], per, 0)
            hs.append(np.exp(d[t][:, None] * a) * hs[-1] + (dm[t] * x[b, t])[:, None] * Bt)
        o["end"][b] = hs[-1]
        g = np.zeros(a.shape) if dend is None else dend[b].copy()
        for t in reversed(range(n)):
            Bt, Ct = np.repeat(bm[b, t], per, 0), np.repeat(cm[b, t], per, 0)
            dy = dout[b, t]
            y = (hs[t + 1] * Ct).sum(1) + (0 if skip is None else skip * x[b, t])
            if z is not None:
                f, df = act(z[b, t], "silu")
                if magnitude:   # SiLU' = s + s z (1 - s) is itself a sum, which cancels near z = -1.28
                    sg = sigmoid(z[b, t])
                    f, df = np.abs(f), sg + sg * np.abs(z[b, t]) * (1 - sg)
                o["dz"][b, t] = dy * y * df
                dy, y = dy * f, y * f
            o["y"][b, t] = y
            g = g + dy[:, None] * Ct
            decay = np.exp(d[t][:, None] * a)
            o["dcmat"][b, t] = (dy[:, None] * hs[t + 1]).reshape(G, per, -1).sum(1)
            o["dbmat"][b, t] = ((dm[t] * x[b, t])[:, None] * g).reshape(G, per, -1).sum(1)
            gb = (g * Bt).sum(1)
            dlog = g * decay * hs[t]
            o["da"] += dlog * dm[t][:, None]
            dd = ((dlog * mag(a)).sum(1) + gb * x[b, t]) * slope[t]
            o["ddt"][b, t] = dd
            o["ddt_bias"] += dd
            o["dx"][b, t] = gb * dm[t] + (0 if skip is None else skip * dy)
            o["dskip"] += dy * x[b, t]
            g = g * decay
        o["dstate"][b] = g
    return o


# ---- group norm ------------------------------------------------------------------------

def norm(x, w=None, bias=None, eps=1e-5, kind="silu", gate=None, sequence=False):
    """(y, mean, rstd); x [B,T,G,C], w, bias [G,C]; statistics over C, or over T and C (sequence)"""
    dims = (1, 3) if sequence else (3,)
    m = x.mean(dims, keepdims=True)
    r = 1.0 / np.sqrt(((x - m) ** 2).mean(dims, keepdims=True) + eps)
    u = (x - m) * r * (1.0 if w is None else w) + (0.0 if bias is None else bias)
    y = act(u, kind)[0] if gate is None else u * act(gate, kind)[0]
    sq = (lambda s: s[:, 0, :, 0]) if sequence else (lambda s: s[..., 0])
    return y, sq(m), sq(r)


def norm_grads(x, dy, w=None, bias=None, eps=1e-5, kind="silu", gate=None, sequence=False):
    """(dx, dgate, dw, dbias)"""
    dims = (1, 3) if sequence else (3,)
    m = x.mean(dims, keepdims=True)
    r = 1.0 / np.sqrt(((x - m) ** 2).mean(dims, keepdims=True) + eps)
    xh = (x - m) * r
    u = xh * (1.0 if w is None else w) + (0.0 if bias is None else bias)
    if gate is None:
        du, dgate = dy * act(u, kind)[1], None
    else:
        f, df = act(gate, kind)
        du, dgate = dy * f, dy * u * df
    v = du * (1.0 if w is None else w)
    dx = r * (v - v.mean(dims, keepdims=True) - xh * (v * xh).mean(dims, keepdims=True))
    return dx, dgate, (du * xh).sum((0, 1)), du.sum((0, 1))
