"""The operators at a block's edges and beside the recurrences, as they are
measured: rotary positions of queries and keys, the gated linear recurrence
with one state a channel, and the residual sum with a layer or RMS norm, each
in a plain form (elementary torch operations in 32 bits, angles in 64) and,
where `own` is true, as this library's calls.

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
        # the query and key heads of one token for each of 32 running sequences, each at its own
        # position, the heads being parts of one projection's output
        rotary("rotary_step", "fwd", "bf16", 32, 1, 32, 8, 128, at="start", split=True),
        # a training batch's queries and keys (B=8 H=32 T=4096 d=128), rotated on their way into the
        # recurrence's head-major layout
        rotary("rotary_heads", "fwd", "bf16", 8, 4096, 32, 32, 128, head_major=True),
        # the backward pass of a long document: neighbouring pairs, half of each head, frequencies
        # stretched for 16 times the trained length
        rotary("rotary_long_bwd", "bwd", "bf16", 1, 65536, 16, 4, 128, part=2, layout="interleaved", scaling="yarn"),
        # a small fp32 model with a quarter of 80 channels rotated, a padded batch, documents packed
        # behind each other (positions given)
        rotary("rotary_odd_fp32", "fwd", "fp32", 3, 517, 5, 5, 80, part=4, at="given", ragged=True),
        # one token for each of 64 sequences, the states carried
        diag("diag_step", "fwd", "bf16", "coupled", 64, 1, 4096, state=True),
        # one long prompt: a long axis over few channels, its end state kept for the tokens that follow
        diag("diag_prompt_long", "fwd", "bf16", "decay", 1, 8192, 4096, state=True),
        # a training step at full width, forward and backward, with the decays' gradient
        diag("diag_train", "train", "bf16", "decay", 4, 4096, 4096),
        # a small fp32 model: odd sizes, two gates, a padded batch that continues from a state
        diag("diag_odd_fp32", "train", "fp32", "sigmoid", 3, 619, 1001, state=True, ragged=True),
        # the residual stream of 32 tokens before a layer's projections
        addnorm("addnorm_step", "fwd", "bf16", 32, 1, 4096, kind="rms"),
        # a training batch's residual stream, kept in fp32 beside bf16 activations
        addnorm("addnorm_stream_fp32", "fwd", "bf16", 4, 4096, 4096, stream="fp32"),
        # a training step's backward pass, the gradient of the stream behind it added
        addnorm("addnorm_train", "bwd", "bf16", 8, 4096, 4096, kind="rms", bias=False),
        # a small fp32 model of odd width, with a bias
        addnorm("addnorm_odd_fp32", "bwd", "fp32", 3, 211, 1001),
    ]


def rotary(name, dir, dtype, B, T, H, Hk, C, part=1, layout="halves", scaling="none", at="none", split=False,
           head_major=False, ragged=False):
    return dict(name=name, op="rotary", dir=dir, dtype=dtype, B=B, T=T, H=H, Hk=Hk, C=C, part=part, layout=layout,
                scaling=scaling, at=at, split=split, head_major=head_major, ragged=ragged)


def diag(name, dir, dtype, kind, B, T, D, state=False, ragged=False):
    return dict(name=name, op="diag", dir=dir, dtype=dtype, kind=kind, B=B, T=T, D=D, state=state, ragged=ragged)


def addnorm(name, dir, dtype, B, T, C, kind="layer", stream="same", bias=True):
    return dict(name=name, op="addnorm", dir=dir, dtype=dtype, B=B, T=T, C=C, kind=kind, stream=stream, bias=bias)


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotary", "diag", "addnorm"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    B = _log(rng, 1, 64)
    T = 1 if rng.random() < 0.2 else _log(rng, 2, 65536)
    if op == "rotary":
        C = rng.choice([64, 80, 96, 128, 128, 256])
        H = _log(rng, 1, 32)
        Hk = rng.choice([h for h in range(1, H + 1) if H % h == 0])
        T = max(1, min(T, 200000000 // (B * (H + Hk) * C)))
        at = rng.choice(["none", "start", "given"])
        return rotary("", rng.choice(["fwd", "bwd"]), dtype, B, T, H, Hk, C, part=rng.choice([1, 1, 2, 4]),
                      layout=rng.choice(["halves", "interleaved"]), scaling=rng.choice(["none", "linear", "ntk", "yarn"]),
                      at=at, split=rng.random() < 0.5, head_major=rng.random() < 0.5, ragged=rng.random() < 0.3)
    if op == "diag":
        D = _log(rng, 100, 4096) if rng.random() < 0.5 else 64 * _log(rng, 2, 64)
        T = max(1, min(T, 30000000 // (B * D)))
        return diag("", rng.choice(["fwd", "train"]), dtype, rng.choice(["coupled", "sigmoid", "decay"]), B, T, D,
                    state=rng.random() < 0.5, ragged=rng.random() < 0.4)
    C = _log(rng, 64, 8192) if rng.random() < 0.4 else 64 * _log(rng, 2, 128)
    T = max(1, min(T, 60000000 // (B * C)))
    return addnorm("", rng.choice(["fwd", "bwd"]), dtype, B, T, C, kind=rng.choice(["layer", "rms"]),
                   stream=rng.choice(["same", "same", "fp32"]), bias=rng.random() < 0.5)


def _streams(case):
    """Element types of activations and residual stream."""
    return DT[case["dtype"]], DT["fp32"] if case["stream"] == "fp32" else DT[case["dtype"]]


def work(case):
    """Bytes of each input read once and each output written once, and the arithmetic of the definition."""
    e = 2 if case["dtype"] == "bf16" else 4
    B, T = case["B"], case["T"]
    n = B * T
    if case["op"] == "rotary":
        W = n * (case["H"] + case["Hk"]) * case["C"]
        at = {"none": 0, "start": 4 * B, "given": 4 * n}[case["at"]]
        return {"bytes": 2 * W * e + at + 4 * (case["C"] // case["part"]), "flops": 3 * W // case["part"]}
    if case["op"] == "diag":
        D, gates = case["D"], 1 if case["kind"] == "coupled" else 2
        par = 4 * D if case["kind"] == "decay" else 0
        st = 4 * B * D if case["state"] else 0
        train = case["dir"] == "train"
        b = (2 + gates) * n * D * e + par + 2 * st + train * ((3 + 2 * gates) * n * D * e + 2 * par + 2 * st)
        return {"bytes": b, "flops": n * D * (8 + 6 * gates + train * (12 + 14 * gates))}
    C = case["C"]
    s = 4 if case["stream"] == "fp32" else e
    par = 4 * C * (1 + case["bias"])
    if case["dir"] == "fwd":   # x and the stream in, the stream and y out
        return {"bytes": 2 * n * C * (e + s) + par, "flops": 8 * n * C}
    # the stream, its gradient and dy in; one gradient out, two where the types differ
    return {"bytes": n * C * (2 * s + e + (e if s == e else e + s)) + 2 * par - 4 * C * case["bias"], "flops": 16 * n * C}


# ---- inputs --------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def _lengths(g, B, T, ragged):
    if not ragged:
        return None
    n = torch.randint(T // 3, T + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
    n[0] = T
    return n


def _frequencies(R, scaling):
    """The R/2 frequencies in 64 bits and the factor of the rotated values: base 10000, stretched by 16 from a
    trained length of 4096 where asked."""
    j = torch.arange(R // 2, dtype=torch.float64, device="cuda")
    f, s, length = 10000.0 ** (-2 * j / R), 16.0, 4096.0
    if scaling == "linear":
        return f / s, 1.0
    if scaling == "ntk":
        return (10000.0 * s ** (R / max(R - 2, 1))) ** (-2 * j / R), 1.0
    if scaling == "yarn":
        keep = ((length * f / (2 * math.pi) - 1.0) / 31.0).clamp(0.0, 1.0)
        return (1.0 - keep) * f / s + keep * f, 0.1 * math.log(s) + 1.0
    return f, 1.0


def prepare(case, seed):
    g = _gen(seed)
    dtype = DT[case["dtype"]]
    B, T = case["B"], case["T"]
    s = {"case": case}
    if case["op"] == "rotary":
        H, Hk, C = case["H"], case["Hk"], case["C"]
        if case["split"]:   # queries, keys and values of one projection
            qkv = _randn(g, (B, T, H + 2 * Hk, C), dtype)
            s["q"], s["k"] = qkv[:, :, :H], qkv[:, :, H:H + Hk]
        else:
            s["q"], s["k"] = _randn(g, (B, T, H, C), dtype), _randn(g, (B, T, Hk, C), dtype)
        R = C // case["part"]
        s["freqs"], s["scale"] = _frequencies(R, case["scaling"])
        s["start"] = s["positions"] = None
        if case["at"] == "start":
            s["start"] = torch.randint(0, 100000, (B,), generator=g, device="cuda", dtype=torch.int32)
        elif case["at"] == "given":   # documents of up to 400 rows behind each other
            first = torch.rand((B, T), generator=g, device="cuda") < 1.0 / 200
            t = torch.arange(T, device="cuda", dtype=torch.int32).expand(B, T)
            s["positions"] = (t - torch.where(first, t, 0).cummax(1).values).contiguous()
        s["lengths"] = _lengths(g, B, T, case["ragged"])
    elif case["op"] == "diag":
        D, kind = case["D"], case["kind"]
        s["x"] = _randn(g, (B, T, D), dtype)
        # forget gates near 1, as such layers are initialised
        shift = {"coupled": 2.0, "sigmoid": 4.5, "decay": 0.0}[kind]
        s["fgate"] = (torch.randn((B, T, D), generator=g, device="cuda") + shift).to(dtype)
        s["igate"] = None if kind == "coupled" else _randn(g, (B, T, D), dtype)
        # decays of 0.9 to 0.999 to the power of 8 gates
        s["decay"] = None if kind != "decay" else \
            -8.0 * torch.log(0.9 + 0.099 * torch.rand(D, generator=g, device="cuda"))
        s["state"] = _randn(g, (B, D), torch.float32) if case["state"] else None
        s["lengths"] = _lengths(g, B, T, case["ragged"])
        if case["dir"] == "train":
            s["dy"] = _randn(g, (B, T, D), dtype)
            s["dstate_out"] = _randn(g, (B, D), torch.float32) if case["state"] else None
    else:
        C = case["C"]
        act, stream = _streams(case)
        s["weight"] = 1.0 + _randn(g, (C,), torch.float32, 0.2)
        s["bias"] = _randn(g, (C,), torch.float32, 0.2) if case["bias"] else None
        s["dy" if case["dir"] == "bwd" else "x"] = _randn(g, (B, T, C), act)
        s["total" if case["dir"] == "bwd" else "residual"] = _randn(g, (B, T, C), stream, 3.0)
        if case["dir"] == "bwd":
            s["dtotal"] = _randn(g, (B, T, C), stream)
    return s


# ---- one pass --------------------------------------------------------------------

def run(s):
    case = s["case"]
    if own:
        from mlstm_sequence_amd import tfla
        return {"rotary": _own_rotary, "diag": _own_diag, "addnorm": _own_addnorm}[case["op"]](s, case, tfla)
    return {"rotary": _plain_rotary, "diag": _plain_diag, "addnorm": _plain_addnorm}[case["op"]](s, case)


def _named(**outs):
    return {k: v for k, v in outs.items() if v is not None}


def _own_rotary(s, case, tfla):
    call = tfla.rotary_forward if case["dir"] == "fwd" else tfla.rotary_backward
    layout = tfla.ROTARY_HALVES if case["layout"] == "halves" else tfla.ROTARY_INTERLEAVED
    q, k = call(s["q"], s["k"], s["freqs"], layout=layout, scale=s["scale"], positions=s["positions"], start=s["start"],
                lengths=s["lengths"], head_major=case["head_major"])
    return {"q": q, "k": k}


def _own_diag(s, case, tfla):
    kind = {"coupled": tfla.DIAG_COUPLED, "sigmoid": tfla.DIAG_SIGMOID, "decay": tfla.DIAG_DECAY}[case["kind"]]
    train = case["dir"] == "train"
    y, end, starts = tfla.diag_forward(s["x"], s["fgate"], s["igate"], s["decay"], kind=kind, state=s["state"],
                                       lengths=s["lengths"], want_state=case["state"], want_starts=train)
    out = _named(y=y, state=end)
    if train:
        g = tfla.diag_backward(s["x"], s["fgate"], s["dy"], starts, s["igate"], s["decay"], kind=kind,
                               lengths=s["lengths"], dstate_out=s["dstate_out"], want_dstate=case["state"])
        out.update(_named(dx=g.dx, dfgate=g.dfgate, digate=g.digate, ddecay=g.ddecay, dstate=g.dstate))
    return out


def _own_addnorm(s, case, tfla):
    kw = dict(eps=1e-5, rms=case["kind"] == "rms")
    if case["dir"] == "fwd":
        y, total = tfla.addnorm_forward(s["x"], s["residual"], s["weight"], s["bias"], **kw)
        return {"y": y, "total": total}
    dx, dres, dw, db = tfla.addnorm_backward(s["total"], s["dy"], s["weight"], bias=s["bias"] is not None,
                                             dtotal=s["dtotal"], **kw)
    return _named(dx=dx, dresidual=dres if case["stream"] == "fp32" else None, dweight=dw, dbias=db)


# ---- plain forms (32 bits, rounded once at the end) ---------------------------------

def _valid(x, lengths):
    """[B,T,1]: whether a row lies before its sequence's end (None: every row does)."""
    if lengths is None:
        return None
    return (torch.arange(x.shape[1], device=x.device)[None, :] < lengths[:, None])[..., None]


def _keep(x, valid):
    return x if valid is None else torch.where(valid, x, 0.0)


def _plain_rotary(s, case):
    B, T = case["B"], case["T"]
    if s["positions"] is not None:
        pos = s["positions"].double()
    else:
        pos = torch.arange(T, device="cuda", dtype=torch.float64)[None, :]
        if s["start"] is not None:
            pos = pos + s["start"][:, None].double()
    angle = pos[..., None] * s["freqs"]                              # in 64 bits: far positions times 1 are thousands of turns
    cos, sin = (s["scale"] * f(angle) for f in (torch.cos, torch.sin))
    cos, sin = cos.float()[:, :, None], (sin if case["dir"] == "fwd" else -sin).float()[:, :, None]
    valid = _valid(s["q"], s["lengths"])
    R = case["C"] // case["part"]

    def turned(x):
        f = x[..., :R].float()
        if case["layout"] == "halves":
            a, b = f[..., :R // 2], f[..., R // 2:]
            f = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        else:
            a, b = f[..., 0::2], f[..., 1::2]
            f = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        f = f.to(x.dtype)
        if R < case["C"]:
            f = torch.cat([f, x[..., R:]], -1)
        if valid is not None:
            f = torch.where(valid[..., None], f, 0.0)
        return f.transpose(1, 2).contiguous().transpose(1, 2) if case["head_major"] else f

    return {"q": turned(s["q"]), "k": turned(s["k"])}


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


def _sigmoid(u):
    return 1.0 / (1.0 + torch.exp(-u))


def _plain_diag(s, case):
    valid, kind = _valid(s["x"], s["lengths"]), case["kind"]
    x = _keep(s["x"].float(), valid)
    r = _sigmoid(s["fgate"].float())
    if kind == "coupled":
        f, i = r, _sigmoid(-s["fgate"].float())
    else:
        si = _sigmoid(s["igate"].float())
        if kind == "sigmoid":
            f, i = r, si
        else:
            u = s["decay"] * r
            f, m = torch.exp(-u), torch.sqrt(-torch.expm1(-2.0 * u))
            i = m * si
    if valid is not None:
        f = torch.where(valid, f, 1.0)
    h = _recurrence(f, i * x, s["state"])
    e = s["x"].dtype
    out = _named(y=_keep(h, valid).to(e), state=h[:, -1].contiguous() if case["state"] else None)
    if case["dir"] == "fwd":
        return out
    # the gradient of h_t: g_t = dy_t + f_{t+1} g_{t+1}, run from the end
    after = torch.cat([f[:, 1:], torch.ones_like(f[:, :1])], 1)
    g = _recurrence(after.flip(1), _keep(s["dy"].float(), valid).flip(1), s["dstate_out"]).flip(1)
    first = s["state"] if s["state"] is not None else torch.zeros_like(h[:, 0])
    before = torch.cat([first[:, None], h[:, :-1]], 1)
    dx, df = i * g, g * before
    digate = ddecay = None
    if kind == "coupled":
        dfgate = (df - g * x) * f * i
    elif kind == "sigmoid":
        dfgate, digate = df * r * (1.0 - r), g * x * si * (1.0 - si)
    else:
        # dm/du = f^2 / m, df/du = -f
        du = _keep(g * x * si * f * f / m - df * f, valid)
        dfgate, digate, ddecay = du * u * (1.0 - r), g * x * i * (1.0 - si), (du * r).sum((0, 1))
    out.update(_named(dx=_keep(dx, valid).to(e), dfgate=_keep(dfgate, valid).to(e),
                      digate=None if digate is None else _keep(digate, valid).to(e), ddecay=ddecay,
                      dstate=(f[:, 0] * g[:, 0]) if s["state"] is not None else None))
    return out


def _plain_addnorm(s, case):
    rms, eps, w = case["kind"] == "rms", 1e-5, s["weight"]
    t = (s["x"].float() + s["residual"].float()) if case["dir"] == "fwd" else s["total"].float()
    d = t if rms else t - t.mean(-1, keepdim=True)
    rstd = 1.0 / torch.sqrt(d.square().mean(-1, keepdim=True) + eps)
    xh = d * rstd
    act, stream = _streams(case)
    if case["dir"] == "fwd":
        y = xh * w
        if s["bias"] is not None:
            y = y + s["bias"]
        return {"y": y.to(act), "total": t.to(stream)}
    dy = s["dy"].float()
    v = dy * w
    dt = v - xh * (v * xh).mean(-1, keepdim=True)
    if not rms:
        dt = dt - v.mean(-1, keepdim=True)
    dt = rstd * dt + s["dtotal"].float()
    return _named(dx=dt.to(act), dresidual=dt.to(stream) if case["stream"] == "fp32" else None,
                  dweight=(dy * xh).sum((0, 1)), dbias=dy.sum((0, 1)) if s["bias"] is not None else None)


# ---- the definitions in 64 bits -------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"rotary": _exact_rotary, "diag": _exact_diag, "addnorm": _exact_addnorm}[case["op"]](s, case)


def _exact_rotary(s, case):
    """Each pair as a complex number times scale e^{i angle}; backward, times the conjugate."""
    B, T, R = case["B"], case["T"], case["C"] // case["part"]
    t = torch.arange(T, dtype=torch.int64, device="cuda").expand(B, T)
    if s["start"] is not None:
        t = t + s["start"].long()[:, None]
    if s["positions"] is not None:
        t = s["positions"].long()
    turn = torch.polar(torch.full((B, T, 1, R // 2), float(s["scale"]), dtype=torch.float64, device="cuda"),
                       (t[:, :, None, None].double() * s["freqs"]) * (1.0 if case["dir"] == "fwd" else -1.0))
    out = {}
    for name in ("q", "k"):
        y = s[name].double().clone()
        z = y[..., :R]
        z = z.unflatten(-1, (2, R // 2)).transpose(-1, -2) if case["layout"] == "halves" else z.unflatten(-1, (R // 2, 2))
        z = torch.view_as_real(torch.view_as_complex(z.contiguous()) * turn)
        y[..., :R] = (z.transpose(-1, -2) if case["layout"] == "halves" else z).flatten(-2)
        if s["lengths"] is not None:
            for b in range(B):
                y[b, int(s["lengths"][b]):] = 0.0
        out[name] = y
    return out


def _exact_diag(s, case):
    """Step by step, as the recurrence is written; the gates' gradients by differentiating f h + i x."""
    B, T, D = s["x"].shape
    train = case["dir"] == "train"
    leaf = lambda t: None if t is None else t.double().requires_grad_(train)   # noqa: E731
    x, fg, ig, decay = map(leaf, (s["x"], s["fgate"], s["igate"], s["decay"]))
    if case["kind"] == "decay":
        logf = -decay * torch.sigmoid(fg)
        f, i = logf.exp(), torch.sqrt(-torch.expm1(2.0 * logf)) * torch.sigmoid(ig)
    else:
        f, i = torch.sigmoid(fg), torch.sigmoid(-fg) if ig is None else torch.sigmoid(ig)
    add = i * x
    n = torch.full((B,), T, device="cuda") if s["lengths"] is None else s["lengths"].long()
    h = torch.zeros((B, D), dtype=torch.float64, device="cuda") if s["state"] is None else s["state"].double()
    before, y = torch.zeros_like(x), torch.zeros_like(x)
    with torch.no_grad():
        for t in range(T):
            live = (t < n)[:, None]
            before[:, t] = h
            h = torch.where(live, f[:, t] * h + add[:, t], h)
            y[:, t] = torch.where(live, h, 0.0)
    out = _named(y=y.detach(), state=h if case["state"] else None)
    if not train:
        return out
    g = torch.zeros_like(h) if s["dstate_out"] is None else s["dstate_out"].double()
    gs = torch.zeros_like(before)
    with torch.no_grad():
        for t in reversed(range(T)):
            live = (t < n)[:, None]
            at = g + s["dy"][:, t].double()
            gs[:, t] = torch.where(live, at, 0.0)
            g = torch.where(live, at * f[:, t], g)
    leaves = [(k, v) for k, v in (("dx", x), ("dfgate", fg), ("digate", ig), ("ddecay", decay)) if v is not None]
    grads = torch.autograd.grad([f, add], [v for _, v in leaves], [gs * before, gs])
    out.update({k: v for (k, _), v in zip(leaves, grads)})
    if case["state"]:
        out["dstate"] = g
    return out


def _exact_addnorm(s, case):
    """The sum, normalised and scaled; the gradients by differentiating just that in 64 bits."""
    fwd = case["dir"] == "fwd"
    t = s["x"].double() + s["residual"].double() if fwd else s["total"].double().requires_grad_()
    w = s["weight"].double().requires_grad_(not fwd)
    b = torch.zeros_like(w) if s["bias"] is None else s["bias"].double()
    b = b.detach().requires_grad_(not fwd)
    if case["kind"] == "rms":
        xh = t * torch.rsqrt(t.pow(2).mean(-1, keepdim=True) + 1e-5)
    else:
        var, mean = torch.var_mean(t, dim=-1, correction=0, keepdim=True)
        xh = (t - mean) * torch.rsqrt(var + 1e-5)
    y = xh * w + b
    if fwd:
        return {"y": y, "total": t}
    dt, dw, db = torch.autograd.grad((y * s["dy"]).sum(), (t, w, b))
    dt = dt + s["dtotal"].double()
    return _named(dx=dt, dresidual=dt if case["stream"] == "fp32" else None, dweight=dw,
                  dbias=db if s["bias"] is not None else None)
