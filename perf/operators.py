"""The operators around the gated linear recurrences, as they are measured:
the causal depthwise convolution, the selective state space scan and the
group norm with an activation, each in a plain form (elementary torch
operations in 32 bits) and, where `own` is true, as this library's calls.

Every tensor has its channels last.  A case names its operator (`op`), its
direction (`dir`: "fwd", "bwd", or "train" for both), the element type and the
sizes.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ---- cases -------------------------------------------------------------------

def listed():
    return [
        # one token for each of 32 running sequences through the convolution in front of the
        # recurrence, its last inputs carried
        conv("conv_step", "fwd", "bf16", 32, 1, 4096, 4, state=True),
        # a padded batch of prompts of different lengths; the input is one half of a projection's
        # output, and the last inputs are kept for the tokens that follow
        conv("conv_prompt_ragged", "fwd", "bf16", 6, 1531, 2048, 4, split=True, ragged=True, state=True),
        # a training step's backward pass at full width
        conv("conv_train", "bwd", "bf16", 4, 4096, 4096, 4),
        # a small fp32 model with odd sizes, three taps and no activation, as tests and studies run it
        conv("conv_odd_fp32", "bwd", "fp32", 3, 515, 1001, 3, act="none", bias=False),
        # one token for each of 64 sequences through the scan, its state carried
        scan("scan_step", "fwd", "bf16", 64, 1, 4096, 16, state=True),
        # one long prompt: few rows in parallel, a long axis
        scan("scan_prompt_long", "fwd", "bf16", 1, 8192, 4096, 16, split=True, state=True),
        # a training step's backward pass
        scan("scan_train", "bwd", "bf16", 4, 2048, 4096, 16, split=True),
        # a small fp32 model: odd lengths in a padded batch, two groups of B and C, no gate
        scan("scan_odd_fp32", "bwd", "fp32", 3, 619, 1000, 8, groups=2, gated=False, ragged=True, state=True),
        # the heads of one token for each of 32 sequences, normalised and gated
        norm("norm_step", "fwd", "bf16", 32, 1, 8, 512, gated=True),
        # the heads of the mLSTM's output (head-major, B=4 H=8 T=8192 d_hv=512) normalised per
        # token, gated and laid out for the output projection
        norm("norm_heads", "fwd", "bf16", 4, 8192, 8, 512, head_major=True, gated=True),
        # the backward pass of the same stage at 32 heads of 128 (B=8 T=4096)
        norm("norm_heads_train", "bwd", "bf16", 8, 4096, 32, 128, head_major=True, gated=True),
        # a channels-last feature map (64 x 64 places, 512 channels in 32 groups): statistics over
        # the places of a group, SiLU behind it, forward and backward
        norm("norm_map_train", "train", "fp32", 6, 4096, 32, 16, over="sequence"),
    ]


def conv(name, dir, dtype, B, T, D, K, act="silu", bias=True, split=False, ragged=False, state=False):
    return dict(name=name, op="conv", dir=dir, dtype=dtype, B=B, T=T, D=D, K=K, act=act, bias=bias, split=split,
                ragged=ragged, state=state)


def scan(name, dir, dtype, B, T, D, N, groups=1, gated=True, split=False, ragged=False, state=False):
    return dict(name=name, op="scan", dir=dir, dtype=dtype, B=B, T=T, D=D, N=N, groups=groups, gated=gated,
                split=split, ragged=ragged, state=state)


def norm(name, dir, dtype, B, T, G, C, act="silu", over="token", head_major=False, gated=False):
    return dict(name=name, op="norm", dir=dir, dtype=dtype, B=B, T=T, G=G, C=C, act=act, over=over,
                head_major=head_major, gated=gated)


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["conv", "scan", "norm"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    B = _log(rng, 1, 64)
    T = 1 if rng.random() < 0.2 else _log(rng, 2, 8192)
    if op == "conv":
        D = _log(rng, 256, 4096) if rng.random() < 0.5 else 64 * _log(rng, 4, 64)
        T = max(1, min(T, 30000000 // (B * D)))
        return conv(None, rng.choice(["fwd", "bwd"]), dtype, B, T, D, rng.choice([2, 3, 4, 4]),
                    act=rng.choice(["silu", "none"]), bias=rng.random() < 0.7, split=rng.random() < 0.5,
                    ragged=rng.random() < 0.4, state=rng.random() < 0.5) | {"name": ""}
    if op == "scan":
        groups = rng.choice([1, 1, 2])
        D = groups * (_log(rng, 100, 2048) if rng.random() < 0.5 else 64 * _log(rng, 2, 32))
        N = rng.choice([8, 16, 16, 32])
        T = max(1, min(T, 250000000 // (B * D * N)))
        return scan(None, rng.choice(["fwd", "bwd"]), dtype, B, T, D, N, groups=groups, gated=rng.random() < 0.7,
                    split=rng.random() < 0.5, ragged=rng.random() < 0.4, state=rng.random() < 0.5) | {"name": ""}
    over = rng.choice(["token", "token", "sequence"])
    G = rng.choice([4, 8, 16, 32])
    C = _log(rng, 8, 64) if over == "sequence" else rng.choice([64, 96, 128, 200, 256, 512])
    dir, gated = rng.choice(["fwd", "bwd", "train"]), rng.random() < 0.5
    each = (2 if dtype == "bf16" else 4) * ((dir != "bwd") * (2 + gated) + (dir != "fwd") * (3 + 2 * gated))
    T = max(1, min(T, 600000000 // (B * G * C * each)))
    return norm(None, dir, dtype, B, T, G, C, act=rng.choice(["silu", "sigmoid", "none"]), over=over,
                head_major=over == "token" and rng.random() < 0.5, gated=gated) | {"name": ""}


def work(case):
    """Bytes of each input read once and each output written once, and the arithmetic of the definition."""
    e = 2 if case["dtype"] == "bf16" else 4
    n = case["B"] * case["T"]
    fwd, bwd = case["dir"] != "bwd", case["dir"] != "fwd"
    if case["op"] == "conv":
        D, K = case["D"], case["K"]
        par = D * (K + case["bias"]) * 4
        st = case["B"] * (K - 1) * D * e if case["state"] else 0
        act = 6 if case["act"] != "none" else 0
        b = fwd * (2 * n * D * e + par + 2 * st) + bwd * (3 * n * D * e + 2 * par + 3 * st)
        return {"bytes": b, "flops": n * D * (fwd * (2 * K + act) + bwd * (6 * K + 2 * act))}
    if case["op"] == "scan":
        D, N, z = case["D"], case["N"], bool(case["gated"])
        par = (D * N + 2 * D) * 4
        st = case["B"] * D * N * 4 if case["state"] else 0
        bc = 2 * n * case["groups"] * N * e
        b = fwd * ((3 + z) * n * D * e + bc + par + 2 * st) + bwd * ((5 + 2 * z) * n * D * e + 2 * bc + 2 * par + 3 * st)
        return {"bytes": b, "flops": n * D * (N * (fwd * 7 + bwd * 22) + 12)}
    W = case["G"] * case["C"]
    z = bool(case["gated"])
    stat = 2 * 4 * (n if case["over"] == "token" else case["B"]) * case["G"]
    b = fwd * ((2 + z) * n * W * e + 2 * W * 4 + stat) + bwd * ((3 + 2 * z) * n * W * e + 4 * W * 4 + stat)
    return {"bytes": b, "flops": n * W * (fwd * 12 + bwd * 24)}


# ---- inputs --------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def _rows(g, B, T, D, dtype, split):
    """[B,T,D]; with `split` one half of a projection's output of twice the width."""
    return _randn(g, (B, T, 2 * D), dtype)[..., :D] if split else _randn(g, (B, T, D), dtype)


def _lengths(g, B, T, ragged):
    if not ragged:
        return None
    n = torch.randint(T // 3, T + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
    n[0] = T
    return n


def prepare(case, seed):
    g = _gen(seed)
    dtype = DT[case["dtype"]]
    B, T = case["B"], case["T"]
    s = {"case": case}
    if case["op"] == "conv":
        D, K = case["D"], case["K"]
        s["x"] = _rows(g, B, T, D, dtype, case["split"])
        s["weight"] = _randn(g, (D, K), torch.float32, K ** -0.5)
        s["bias"] = _randn(g, (D,), torch.float32, 0.1) if case["bias"] else None
        s["state"] = _randn(g, (B, K - 1, D), dtype) if case["state"] else None
        s["lengths"] = _lengths(g, B, T, case["ragged"])
        if case["dir"] == "bwd":
            s["dy"] = _randn(g, (B, T, D), dtype)
            s["dstate_out"] = _randn(g, (B, K - 1, D), dtype) if case["state"] else None
    elif case["op"] == "scan":
        D, N, G = case["D"], case["N"], case["groups"]
        if case["split"]:   # x and the gate are the halves of one projection, B and C parts of another
            xz = _randn(g, (B, T, 2 * D), dtype)
            s["x"], z = xz[..., :D], xz[..., D:]
            r = 4 * (-(-D // 64))
            dbc = _randn(g, (B, T, r + 2 * G * N), dtype)
            bmat, cmat = dbc[..., r:r + G * N], dbc[..., r + G * N:]
            s["bmat"], s["cmat"] = bmat.unflatten(-1, (G, N)), cmat.unflatten(-1, (G, N))
        else:
            s["x"] = _randn(g, (B, T, D), dtype)
            z = _randn(g, (B, T, D), dtype)
            s["bmat"], s["cmat"] = _randn(g, (B, T, G, N), dtype), _randn(g, (B, T, G, N), dtype)
        s["z"] = z if case["gated"] else None
        s["dt"] = _randn(g, (B, T, D), dtype, 0.5)
        # steps between 0.001 and 0.1, as such layers are initialised
        step = torch.exp(torch.rand(D, generator=g, device="cuda") * math.log(100.0) + math.log(1e-3))
        s["dt_bias"] = step + torch.log(-torch.expm1(-step))
        s["a"] = -torch.arange(1, N + 1, device="cuda", dtype=torch.float32) * \
            torch.exp(0.1 * torch.randn((D, N), generator=g, device="cuda"))
        s["skip"] = torch.ones(D, device="cuda") + _randn(g, (D,), torch.float32, 0.1)
        s["state"] = _randn(g, (B, D, N), torch.float32) if case["state"] else None
        s["lengths"] = _lengths(g, B, T, case["ragged"])
        if case["dir"] == "bwd":
            s["dy"] = _randn(g, (B, T, D), dtype)
            s["dstate_out"] = _randn(g, (B, D, N), torch.float32) if case["state"] else None
    else:
        G, C = case["G"], case["C"]
        if case["head_major"]:
            s["x"] = (_randn(g, (B, G, T, C), dtype, 2.0) + 0.5).transpose(1, 2)
        else:
            s["x"] = _randn(g, (B, T, G, C), dtype, 2.0) + 0.5
        s["weight"] = 1.0 + _randn(g, (G, C), torch.float32, 0.2)
        s["bias"] = _randn(g, (G, C), torch.float32, 0.2)
        s["gate"] = _randn(g, (B, T, G, C), dtype) if case["gated"] else None
        if case["dir"] != "fwd":
            s["dy"] = _randn(g, (B, T, G, C), dtype)
        if case["dir"] == "bwd":   # the forward pass's statistics are kept for the backward pass
            dims = (3,) if case["over"] == "token" else (1, 3)
            x64 = s["x"].double()
            var, mean = torch.var_mean(x64, dim=dims, correction=0)
            s["mean"], s["rstd"] = mean.float().contiguous(), torch.rsqrt(var + 1e-5).float().contiguous()
    return s


# ---- one pass --------------------------------------------------------------------

def run(s):
    case = s["case"]
    if own:
        from mlstm_sequence_amd import tfla
        return {"conv": _own_conv, "scan": _own_scan, "norm": _own_norm}[case["op"]](s, case, tfla)
    return {"conv": _plain_conv, "scan": _plain_scan, "norm": _plain_norm}[case["op"]](s, case)


def _named(**outs):
    return {k: v for k, v in outs.items() if v is not None}


def _own_conv(s, case, tfla):
    act = tfla.ACT_SILU if case["act"] == "silu" else tfla.ACT_NONE
    if case["dir"] == "fwd":
        y, last = tfla.conv_forward(s["x"], s["weight"], s["bias"], act=act, state=s["state"], lengths=s["lengths"],
                                    want_state=case["state"])
        return _named(y=y, state=last)
    dx, dw, db, ds = tfla.conv_backward(s["x"], s["weight"], s["dy"], s["bias"], act=act, state=s["state"],
                                        lengths=s["lengths"], dstate_out=s["dstate_out"])
    return _named(dx=dx, dweight=dw, dbias=db, dstate=ds)


def _own_scan(s, case, tfla):
    kw = dict(skip=s["skip"], z=s["z"], dt_bias=s["dt_bias"], softplus=True, state=s["state"], lengths=s["lengths"])
    if case["dir"] == "fwd":
        y, last = tfla.scan_forward(s["x"], s["dt"], s["a"], s["bmat"], s["cmat"], want_state=case["state"], **kw)
        return _named(y=y, state=last)
    g = tfla.scan_backward(s["x"], s["dt"], s["a"], s["bmat"], s["cmat"], s["dy"], dstate_out=s["dstate_out"], **kw)
    return _named(dx=g.dx, ddt=g.ddt, da=g.da, db=g.dbmat, dc=g.dcmat, dskip=g.dskip, dz=g.dz, ddt_bias=g.ddt_bias,
                  dstate=g.dstate)


def _own_norm(s, case, tfla):
    act = {"silu": tfla.ACT_SILU, "sigmoid": tfla.ACT_SIGMOID, "none": tfla.ACT_NONE}[case["act"]]
    kw = dict(act=act, gate=s["gate"], over=tfla.NORM_TOKEN if case["over"] == "token" else tfla.NORM_SEQUENCE)
    out = {}
    mean, rstd = s.get("mean"), s.get("rstd")
    if case["dir"] != "bwd":
        y, mean, rstd = tfla.norm_forward(s["x"], s["weight"], s["bias"], eps=1e-5, **kw)
        out.update(y=y, mean=mean, rstd=rstd)
    if case["dir"] != "fwd":
        dx, dgate, dw, db = tfla.norm_backward(s["x"], s["dy"], mean, rstd, s["weight"], s["bias"], **kw)
        out.update(_named(dx=dx, dgate=dgate, dweight=dw, dbias=db))
    return out


# ---- plain forms (32 bits, rounded once at the end) ---------------------------------

def _act(u, kind):
    """act(u) and its derivative."""
    if kind == "none":
        return u, torch.ones_like(u)
    sg = 1.0 / (1.0 + torch.exp(-u))
    return (sg, sg * (1.0 - sg)) if kind == "sigmoid" else (u * sg, sg * (1.0 + u * (1.0 - sg)))


def _valid(x, lengths):
    """[B,T,1]: whether a row lies before its sequence's end (None: every row does)."""
    if lengths is None:
        return None
    return (torch.arange(x.shape[1], device=x.device)[None, :] < lengths[:, None])[..., None]


def _keep(x, valid):
    return x if valid is None else torch.where(valid, x, 0.0)


def _plain_conv(s, case):
    x, w, K = s["x"], s["weight"], case["K"]
    B, T, D = x.shape
    valid = _valid(x, s["lengths"])
    head = x.new_zeros((B, K - 1, D)) if s["state"] is None else s["state"]
    ext = torch.cat([head, x], 1)                      # row p of the extended sequence is step p - (K - 1)
    last = s["lengths"].long() if valid is not None else torch.full((B,), T, device=x.device)
    tail = last[:, None] + torch.arange(K - 1, device=x.device)[None, :]
    ef = ext.float()
    u = sum(ef[:, j:j + T] * w[:, j] for j in range(K))
    if s["bias"] is not None:
        u = u + s["bias"]
    f, df = _act(u, case["act"])
    if case["dir"] == "fwd":
        end = ext[torch.arange(B, device=x.device)[:, None], tail] if case["state"] else None
        return _named(y=_keep(f, valid).to(x.dtype), state=end)
    du = _keep(s["dy"].float() * df, valid)
    dext = torch.zeros_like(ef)
    for j in range(K):
        dext[:, j:j + T] += du * w[:, j]
    if valid is not None:
        ef = torch.cat([ef[:, :K - 1], _keep(ef[:, K - 1:], valid)], 1)
    dw = torch.stack([(du * ef[:, j:j + T]).sum((0, 1)) for j in range(K)], 1)
    if s["dstate_out"] is not None:
        dext[torch.arange(B, device=x.device)[:, None], tail] += s["dstate_out"].float()
    return _named(dx=_keep(dext[:, K - 1:], valid).to(x.dtype), dweight=dw,
                  dbias=du.sum((0, 1)) if s["bias"] is not None else None,
                  dstate=dext[:, :K - 1].to(x.dtype) if s["state"] is not None else None)


def _recurrence(a, b, first):
    """h_t = a_t h_{t-1} + b_t along dimension 1, all h_t: blocks of about sqrt(T) steps side by
    side, then the blocks' starts one after another."""
    B, T = a.shape[:2]
    c = 1 << ((T - 1).bit_length() + 1) // 2
    n = -(-T // c)
    if n * c > T:
        pad = (B, n * c - T) + tuple(a.shape[2:])
        a, b = torch.cat([a, a.new_ones(pad)], 1), torch.cat([b, b.new_zeros(pad)], 1)
    a, h = a.unflatten(1, (n, c)), b.unflatten(1, (n, c)).clone()
    for j in range(1, c):
        h[:, :, j].addcmul_(a[:, :, j], h[:, :, j - 1])
    if n > 1 or first is not None:
        p = torch.cumprod(a, 2)
        at = first if first is not None else torch.zeros_like(h[:, 0, 0])
        for k in range(n):
            h[:, k].addcmul_(p[:, k], at[:, None])
            at = h[:, k, -1]
    return h.flatten(1, 2)[:, :T]


def _plain_scan(s, case):
    valid = _valid(s["x"], s["lengths"])
    x, a, G = _keep(s["x"].float(), valid), s["a"], case["groups"]
    B, T, D = x.shape
    u = s["dt"].float() + s["dt_bias"]
    delta = _keep(torch.clamp(u, min=0.0) + torch.log1p(torch.exp(-torch.abs(u))), valid)
    bm, cm = _keep(s["bmat"].float().flatten(2), valid), _keep(s["cmat"].float().flatten(2), valid)
    bm = bm.unflatten(-1, (G, 1, -1))                                # [B,T,G,1,N] against [B,T,G,D/G,N]
    cm = cm.unflatten(-1, (G, 1, -1))
    by_group = lambda t: t.unflatten(2, (G, D // G))                 # noqa: E731
    decay = torch.exp(delta[..., None] * a)
    h = _recurrence(decay, (by_group(delta * x)[..., None] * bm).flatten(2, 3), s["state"])
    hg = by_group(h)
    y = (hg * cm).sum(-1).flatten(2) + s["skip"] * x
    f, df = _act(s["z"].float(), "silu") if s["z"] is not None else (None, None)
    if case["dir"] == "fwd":
        end = h[:, -1].contiguous() if case["state"] else None
        return _named(y=_keep(y if f is None else y * f, valid).to(s["x"].dtype), state=end)
    dout = _keep(s["dy"].float(), valid)
    dz = None if f is None else _keep(dout * y * df, valid)
    dy = dout if f is None else _keep(dout * f, valid)
    # the gradient of h_t: g_t = C_t dy_t + a_{t+1} g_{t+1}, run from the end
    after = torch.cat([decay[:, 1:], torch.ones_like(decay[:, :1])], 1)
    dh = (by_group(dy)[..., None] * cm).flatten(2, 3)
    g = _recurrence(after.flip(1), dh.flip(1), s["dstate_out"]).flip(1)
    del after, dh
    first = s["state"] if s["state"] is not None else torch.zeros_like(h[:, 0])
    dlog = g * decay * torch.cat([first[:, None], h[:, :-1]], 1)     # the gradient of delta A
    gb = (by_group(g) * bm).sum(-1).flatten(2)
    ddelta = (dlog * a).sum(-1) + gb * x
    ddt = _keep(ddelta / (1.0 + torch.exp(-u)), valid)
    e = s["x"].dtype
    return _named(dx=_keep(gb * delta + s["skip"] * dy, valid).to(e), ddt=ddt.to(e),
                  da=(dlog * delta[..., None]).sum((0, 1)),
                  db=(by_group(g) * by_group(delta * x)[..., None]).sum(3).to(e),
                  dc=(hg * by_group(dy)[..., None]).sum(3).to(e),
                  dskip=(dy * x).sum((0, 1)), dz=None if dz is None else dz.to(e), ddt_bias=ddt.sum((0, 1)),
                  dstate=(decay[:, 0] * g[:, 0]) if s["state"] is not None else None)


def _plain_norm(s, case):
    x, w, b = s["x"].float(), s["weight"], s["bias"]
    dims = (3,) if case["over"] == "token" else (1, 3)
    out = {}
    mean, rstd = s.get("mean"), s.get("rstd")
    if case["dir"] != "bwd":
        m = x.mean(dims, keepdim=True)
        r = 1.0 / torch.sqrt((x - m).square().mean(dims, keepdim=True) + 1e-5)
        mean, rstd = m.squeeze(3), r.squeeze(3)
        if case["over"] != "token":
            mean, rstd = mean.squeeze(1), rstd.squeeze(1)
    at = (Ellipsis, None) if case["over"] == "token" else (slice(None), None, slice(None), None)
    xh = (x - mean[at]) * rstd[at]
    u = xh * w + b
    f, df = _act(u if s["gate"] is None else s["gate"].float(), case["act"])
    if case["dir"] != "bwd":
        out.update(y=(f if s["gate"] is None else u * f).to(s["x"].dtype), mean=mean, rstd=rstd)
    if case["dir"] != "fwd":
        dy = s["dy"].float()
        du = dy * (df if s["gate"] is None else f)
        v = du * w
        dx = rstd[at] * (v - v.mean(dims, keepdim=True) - xh * (v * xh).mean(dims, keepdim=True))
        out.update(_named(dx=dx.to(s["x"].dtype), dgate=None if s["gate"] is None else (dy * u * df).to(s["x"].dtype),
                          dweight=(du * xh).sum((0, 1)), dbias=du.sum((0, 1))))
    return out


# ---- the definitions in 64 bits -------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"conv": _exact_conv, "scan": _exact_scan, "norm": _exact_norm}[case["op"]](s, case)


def _f64(t):
    return None if t is None else t.double()


def _exact_conv(s, case):
    """Sequence by sequence: the window of every step times the weights."""
    B, T, D = s["x"].shape
    K = case["K"]
    w = _f64(s["weight"])
    y, dx = torch.zeros((2, B, T, D), dtype=torch.float64, device="cuda").unbind(0)
    end, dstate = torch.zeros((2, B, K - 1, D), dtype=torch.float64, device="cuda").unbind(0)
    dw, db = torch.zeros_like(w), torch.zeros_like(w[:, 0])
    for i in range(B):
        n = T if s["lengths"] is None else int(s["lengths"][i])
        seq = torch.zeros((K - 1 + n, D), dtype=torch.float64, device="cuda")
        if s["state"] is not None:
            seq[:K - 1] = s["state"][i]
        seq[K - 1:] = s["x"][i, :n]
        seq.requires_grad_(case["dir"] == "bwd")
        wi = w.clone().requires_grad_(case["dir"] == "bwd")
        bi = (_f64(s["bias"]) if case["bias"] else torch.zeros_like(db)).clone().requires_grad_(case["dir"] == "bwd")
        u = bi.expand(n, D)
        if n:
            u = u + (seq.unfold(0, K, 1) * wi).sum(-1)
        f = u * torch.sigmoid(u) if case["act"] == "silu" else u
        if case["dir"] == "fwd":
            y[i, :n], end[i] = f, seq[n:]
            continue
        loss = (f * s["dy"][i, :n]).sum()
        if s["dstate_out"] is not None:
            loss = loss + (seq[n:] * s["dstate_out"][i]).sum()
        if n or s["dstate_out"] is not None:
            gs, gw, gb = torch.autograd.grad(loss, (seq, wi, bi), allow_unused=True)
            dstate[i], dx[i, :n] = gs[:K - 1], gs[K - 1:]
            if gw is not None:
                dw += gw
            if gb is not None:
                db += gb
    if case["dir"] == "fwd":
        return _named(y=y, state=end if case["state"] else None)
    return _named(dx=dx, dweight=dw, dbias=db if case["bias"] else None,
                  dstate=dstate if s["state"] is not None else None)


def _exact_scan(s, case):
    """Step by step, as the recurrence is written."""
    B, T, D = s["x"].shape
    per = D // case["groups"]
    x, a, skip, z = _f64(s["x"]), _f64(s["a"]), _f64(s["skip"]), _f64(s["z"])
    u = _f64(s["dt"]) + _f64(s["dt_bias"])
    delta = torch.logaddexp(u, torch.zeros_like(u))
    n = torch.full((B,), T, device="cuda") if s["lengths"] is None else s["lengths"].long()
    h = torch.zeros((B, D, case["N"]), dtype=torch.float64, device="cuda") if s["state"] is None else _f64(s["state"])
    first = h
    row = lambda m, t: _f64(m[:, t]).repeat_interleave(per, dim=1)   # noqa: E731  [B,D,N]
    y = torch.zeros_like(x)
    hs = []
    for t in range(T):
        live = (t < n)[:, None]
        step = torch.exp(delta[:, t, :, None] * a) * h + (delta[:, t] * x[:, t])[..., None] * row(s["bmat"], t)
        h = torch.where(live[..., None], step, h)
        y[:, t] = torch.where(live, (h * row(s["cmat"], t)).sum(-1) + skip * x[:, t], 0.0)
        if case["dir"] == "bwd":
            hs.append(h)
    sg = None if z is None else torch.sigmoid(z)
    if case["dir"] == "fwd":
        return _named(y=y if z is None else y * z * sg, state=h if case["state"] else None)
    dout = _f64(s["dy"])
    mask = (torch.arange(T, device="cuda")[None, :] < n[:, None])[..., None]
    dy = torch.where(mask, dout if z is None else dout * z * sg, 0.0)
    dz = None if z is None else torch.where(mask, dout * y * sg * (1.0 + z * (1.0 - sg)), 0.0)
    g = torch.zeros_like(h) if s["dstate_out"] is None else _f64(s["dstate_out"])
    dx, ddt = torch.zeros_like(x), torch.zeros_like(x)
    da = torch.zeros_like(a)
    db, dc = torch.zeros((2,) + tuple(s["bmat"].shape), dtype=torch.float64, device="cuda").unbind(0)
    for t in reversed(range(T)):
        live = (t < n)[:, None, None]
        cur = torch.where(live, g + dy[:, t, :, None] * row(s["cmat"], t), g)
        decay = torch.exp(delta[:, t, :, None] * a)
        before = hs[t - 1] if t else first
        dlog = torch.where(live, cur * decay * before, 0.0)
        gb = torch.where(live, cur * row(s["bmat"], t), 0.0).sum(-1)
        dx[:, t] = gb * delta[:, t] + skip * dy[:, t]
        ddt[:, t] = ((dlog * a).sum(-1) + gb * x[:, t]) * torch.sigmoid(u[:, t])
        da += (dlog * delta[:, t, :, None]).sum(0)
        at = (delta[:, t] * x[:, t])[..., None]
        db[:, t] = torch.where(live, cur * at, 0.0).unflatten(1, (case["groups"], per)).sum(2)
        dc[:, t] = (dy[:, t, :, None] * hs[t]).unflatten(1, (case["groups"], per)).sum(2)
        g = torch.where(live, cur * decay, g)
    return _named(dx=dx, ddt=ddt, da=da, db=db, dc=dc, dskip=(dy * x).sum((0, 1)), dz=dz, ddt_bias=ddt.sum((0, 1)),
                  dstate=g if s["state"] is not None else None)


def _exact_norm(s, case):
    """Normalise, scale, activate; the gradients by differentiating just that in 64 bits."""
    x, w, b, z = (t.clone().requires_grad_() if t is not None else None
                  for t in map(_f64, (s["x"], s["weight"], s["bias"], s["gate"])))
    dims = (3,) if case["over"] == "token" else (1, 3)
    var, mean = torch.var_mean(x, dim=dims, correction=0, keepdim=True)
    rstd = torch.rsqrt(var + 1e-5)
    fn = {"silu": torch.nn.functional.silu, "sigmoid": torch.sigmoid, "none": lambda t: t}[case["act"]]
    u = (x - mean) * rstd * w + b
    y = fn(u) if z is None else u * fn(z)
    out = {}
    if case["dir"] != "bwd":
        shape = tuple(s["x"].shape[:3]) if case["over"] == "token" else (case["B"], case["G"])
        out.update(y=y.detach(), mean=mean.detach().reshape(shape), rstd=rstd.detach().reshape(shape))
    if case["dir"] != "fwd":
        leaves = [t for t in (x, w, b, z) if t is not None]
        gs = torch.autograd.grad((y * s["dy"]).sum(), leaves)
        out.update(_named(dx=gs[0], dweight=gs[1], dbias=gs[2], dgate=gs[3] if z is not None else None))
    return out
