"""Selective state space scan against the 64-bit reference.

Every output is a sum of products of inputs, decays and gate values.  A decay
a = exp(delta A) evaluated in fp32 is off by rho = |delta A| (e + 4 U) + 3 U
relative, e the relative error of delta: half a step of the rounded sum
dt + dt_bias through softplus, and (8 + 2 |u|) U for softplus itself (the
exponential's argument is rounded).  A product holds at most the decays of a
whole sequence, twice in the backward pass; beside them at most 8 factors of
up to 12 U each; a sum of n terms adds (n + 1) U.  So an output is within
(2 sum_t rho_t + (n + 100) U) times the sum of its terms' magnitudes, which
the reference computes, and half a step of its type.  SiLU's slope
s (1 + z (1 - s)) counts as its two terms: 1 + z (1 - s) passes through 0 near
z = -1.28, where fp32 leaves about 2 U s, whatever is left of the sum."""
import numpy as np
import pytest
import torch

from blocks_helpers import HALF, U, as_view, randn, within
from mlstm_sequence_amd import tfla
from oracle import blocks as O

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
NAN = float("nan")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    tfla.lib()


def cuda(t):
    return None if t is None else t.cuda()


def make(dtype, B, T, D, N, G=1, gated=True, bias=True, skip=True, state=True, softplus=True, lengths=None, seed=0):
    rng = np.random.default_rng(seed + 13 * T + D + N)
    d = dict(x=randn(rng, (B, T, D), dtype), dt=randn(rng, (B, T, D), dtype, 1.0, -1.0) if softplus else None,
             a=randn(rng, (D, N), F32, 0.3, 0.0), bmat=randn(rng, (B, T, G, N), dtype), cmat=randn(rng, (B, T, G, N), dtype),
             skip=randn(rng, (D,), F32) if skip else None, z=randn(rng, (B, T, D), dtype, 2.0) if gated else None,
             dt_bias=randn(rng, (D,), F32, 0.5) if bias else None,
             state=randn(rng, (B, D, N), F32) if state else None, dy=randn(rng, (B, T, D), dtype),
             dend=randn(rng, (B, D, N), F32) if state else None)
    d["a"] = (-torch.exp(d["a"][0]), None)
    d["a"] = (d["a"][0], d["a"][0].double().numpy())
    if not softplus:   # steps as they are: positive
        t = torch.from_numpy(np.abs(rng.standard_normal((B, T, D))) * 0.5).to(dtype)
        d["dt"] = (t, t.double().numpy())
        if bias:
            t = torch.from_numpy(np.abs(rng.standard_normal(D)) * 0.1).float()
            d["dt_bias"] = (t, t.double().numpy())
    dev = {k: None if v is None else v[0] for k, v in d.items()}
    ref = {k: None if v is None else v[1] for k, v in d.items()}
    if lengths is not None:
        for k in ("x", "dt", "z", "dy", "bmat", "cmat"):
            if dev[k] is not None:
                for b, n in enumerate(lengths):
                    dev[k][b, max(0, n):] = NAN
    dev["lengths"] = None if lengths is None else torch.tensor(lengths, dtype=torch.int32)
    return dev, ref


def bounds(ref, softplus, lengths, T):
    """Relative factor of the magnitudes (see above), without the sums' length."""
    dt, b = ref["dt"], 0.0 if ref["dt_bias"] is None else ref["dt_bias"]
    u = dt + b
    ab = np.abs(dt) + np.abs(b)
    delta, slope = O._delta(dt, ref["dt_bias"], softplus)
    e = slope * U * ab / np.abs(delta) + ((8 + 2 * np.abs(u)) * U if softplus else 0.0)
    big = np.abs(ref["a"]).max(1)                                        # of the channel's states
    rho = np.abs(delta) * big * (e + 4 * U) + 3 * U
    if lengths is not None:
        rho = rho * (np.arange(T)[None, :] < np.asarray(lengths)[:, None])[..., None]
        e = np.where(rho > 0, e, 0)
    return 2 * rho.sum(1).max() + 2 * e.max() + 100 * U


def check(dtype, B, T, D, N, G=1, gated=True, bias=True, skip=True, state=True, softplus=True, lengths=None, view="plain"):
    print("scan", dtype, B, T, D, N, G, gated, bias, skip, state, softplus, lengths, view, flush=True)
    dev, ref = make(dtype, B, T, D, N, G, gated, bias, skip, state, softplus, lengths)
    x, dt, z, dy = (as_view(dev[k], view) for k in ("x", "dt", "z", "dy"))
    bmat, cmat = (as_view(dev[k].flatten(2), view).unflatten(-1, (G, N)) for k in ("bmat", "cmat"))
    a, sk, db, st, de, ln = (cuda(dev[k]) for k in ("a", "skip", "dt_bias", "state", "dend", "lengths"))
    kw = dict(skip=sk, z=z, dt_bias=db, softplus=softplus, state=st, lengths=ln)
    y = as_view(torch.full((B, T, D), NAN, dtype=dtype), view)
    _, end = tfla.scan_forward(x, dt, a, bmat, cmat, want_state=True, y=y, **kw)
    outs = {k: as_view(torch.full((B, T, D), NAN, dtype=dtype), view) for k in ("dx", "ddt", "dz") if k != "dz" or gated}
    g = tfla.scan_backward(x, dt, a, bmat, cmat, dy, dstate_out=de, **kw, **outs)
    torch.cuda.synchronize()

    rk = dict(x=ref["x"], dt=ref["dt"], a=ref["a"], bm=ref["bmat"], cm=ref["cmat"], dout=ref["dy"], skip=ref["skip"],
              z=ref["z"], dt_bias=ref["dt_bias"], softplus=softplus, state=ref["state"], lengths=lengths, dend=ref["dend"])
    want, mag = O.scan_grads(**rk), O.scan_grads(magnitude=True, **rk)
    rel = bounds(ref, softplus, lengths, T)
    h = HALF[dtype]
    for name, got, n, half in (("y", y, N, h), ("end", end, T, 0.0), ("dx", g.dx, N, h), ("ddt", g.ddt, 2 * N, h),
                               ("dz", g.dz, N, h), ("dbmat", g.dbmat, D, h), ("dcmat", g.dcmat, D, h), ("da", g.da, B * T, 0.0),
                               ("dskip", g.dskip, B * T, 0.0), ("ddt_bias", g.ddt_bias, B * T * N, 0.0),
                               ("dstate", g.dstate, T, 0.0)):
        if got is None:
            assert {"dz": not gated, "dskip": not skip, "ddt_bias": not bias, "dstate": not state}[name]
            continue
        within(name, got, want[name], half * np.abs(want[name]) + (rel + (n + 1) * U) * mag[name] + 1e-37)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T", [1, 2, 7, 8, 9, 15, 16, 17, 33, 130])
def test_lengths_of_one_call(dtype, T):
    check(dtype, 2, T, 70, 16, gated=T % 2 == 0)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("N", [1, 2, 4, 5, 8, 11, 12, 16, 20, 31, 32, 36, 61, 64])
def test_state_sizes(dtype, N):
    check(dtype, 2, 37, 40, N, G=2)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D,G", [(1, 1), (3, 3), (63, 1), (64, 1), (65, 1), (130, 2), (192, 3), (300, 1)])
def test_widths_and_groups(dtype, D, G):
    check(dtype, 2, 21, D, 8, G=G)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("view", ["half", "odd", "wide", "time"])
def test_views(dtype, view):
    check(dtype, 3, 20, 66, 16, view=view)


@pytest.mark.parametrize("off", ["gated", "bias", "skip", "state", "softplus"])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_without(dtype, off):
    check(dtype, 2, 40, 64, 16, **{off: False})


@pytest.mark.parametrize("dtype", [BF, F32])
def test_padded_batch(dtype):
    check(dtype, 6, 90, 66, 16, lengths=[90, 0, 1, 16, 17, 89])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_long_axis_few_rows(dtype):
    """A single sequence of few channels, long enough to be split over workgroups."""
    check(dtype, 1, 1111, 64, 8, lengths=[1100])


def test_two_long_sequences_padded():
    check(F32, 2, 700, 20, 4, lengths=[700, 300], state=False)


def test_lengths_out_of_range_are_clamped():
    dev, _ = make(BF, 3, 20, 64, 16)
    x, dt, a, b, c, s = (dev[k].cuda() for k in ("x", "dt", "a", "bmat", "cmat", "state"))
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    got = tfla.scan_forward(x, dt, a, b, c, state=s, want_state=True, lengths=i32([-5, 20, 1 << 30]))
    want = tfla.scan_forward(x, dt, a, b, c, state=s, want_state=True, lengths=i32([0, 20, 20]))
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert torch.equal(got[1][0], s[0])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_prompt_then_single_tokens(dtype):
    """A prompt, then one token at a time with the state updated in place,
    against the reference of the whole sequence."""
    T, N = 24, 16
    dev, ref = make(dtype, 3, T, 72, N, state=False)
    x, dt, a, b, c, sk, z, db = (cuda(dev[k]) for k in ("x", "dt", "a", "bmat", "cmat", "skip", "z", "dt_bias"))
    part = lambda lo, hi: dict(x=x[:, lo:hi], dt=dt[:, lo:hi], a=a, bmat=b[:, lo:hi], cmat=c[:, lo:hi], skip=sk,  # noqa: E731
                               z=z[:, lo:hi], dt_bias=db)
    y, st = tfla.scan_forward(want_state=True, **part(0, 9))
    ys = [y]
    for t in range(9, T):
        y, same = tfla.scan_forward(state=st, state_out=st, **part(t, t + 1))
        assert same is st
        ys.append(y)
    torch.cuda.synchronize()
    rk = dict(x=ref["x"], dt=ref["dt"], a=ref["a"], bm=ref["bmat"], cm=ref["cmat"], dout=ref["dy"], skip=ref["skip"],
              z=ref["z"], dt_bias=ref["dt_bias"])
    want, mag = O.scan_grads(**rk), O.scan_grads(magnitude=True, **rk)
    rel = bounds(ref, True, None, T) + (N + 1) * U
    within("y", torch.cat(ys, 1), want["y"], HALF[dtype] * np.abs(want["y"]) + rel * mag["y"])
    within("end", st, want["end"], rel * mag["end"])


def test_extreme_steps():
    """Steps from 0 to so large that every decay is 0: nothing overflows."""
    B, T, D, N = 1, 40, 64, 8
    dev, ref = make(F32, B, T, D, N, bias=False, gated=False)
    dt = dev["dt"]
    dt[:, 5:10], dt[:, 10:15], dt[:, 15:20] = -200.0, 200.0, 5000.0
    got, end = tfla.scan_forward(dev["x"].cuda(), dt.cuda(), dev["a"].cuda(), dev["bmat"].cuda(), dev["cmat"].cuda(),
                                 state=dev["state"].cuda(), want_state=True)
    torch.cuda.synchronize()
    want, wend = O.scan(ref["x"], dt.double().numpy(), ref["a"], ref["bmat"], ref["cmat"], state=ref["state"])
    mag = O.scan_grads(ref["x"], dt.double().numpy(), ref["a"], ref["bmat"], ref["cmat"], ref["dy"], state=ref["state"],
                       magnitude=True)
    # delta A up to 5000 max|a|: where that is above 104 the decay is 0 on both sides of fp32's range; below,
    # rho <= 104 * 12 U + 3 U for each of at most T steps, and delta itself within 12 U
    rel = (T * (104 * 12 + 3) + 100 + T) * U
    within("y", got, want, rel * mag["y"] + 1e-30)
    within("end", end, wend, rel * mag["end"] + 1e-30)


def test_refusals_on_tensors():
    dev, _ = make(BF, 2, 10, 64, 16)
    x, dt, a, b, c, s, z, dy = (dev[k].cuda() for k in ("x", "dt", "a", "bmat", "cmat", "state", "z", "dy"))
    good = dict(x=x, dt=dt, a=a, bmat=b, cmat=c, state=s, z=z)
    for bad in (dict(dt=dt.float()), dict(a=a.bfloat16()), dict(a=a[:, :8]), dict(bmat=b[..., :8]), dict(cmat=c.transpose(1, 3)),
                dict(state=s.bfloat16()), dict(z=z[:, :5]), dict(y=x), dict(state_out=s[:, :, ::2]), dict(x=x[0]),
                dict(bmat=b[:, :, 0]), dict(lengths=torch.tensor([1, 2])), dict(z=z.cpu())):
        kw = dict(good)
        kw.update(bad)
        with pytest.raises((TypeError, ValueError, tfla.TflaError)):
            tfla.scan_forward(**kw)
    with pytest.raises((ValueError, tfla.TflaError)):
        tfla.scan_backward(x, dt, a, b, c, dy, dx=dy)


def grads_equal(p, q):
    return all((u is None and v is None) or torch.equal(u, v) for u, v in zip(p, q))


def test_stream_workspace_and_repeat():
    dev, _ = make(BF, 1, 600, 64, 16)
    x, dt, a, b, c, s, z, dy = (dev[k].cuda() for k in ("x", "dt", "a", "bmat", "cmat", "state", "z", "dy"))
    args = (x, dt, a, b, c)
    f0, g0 = tfla.scan_forward(*args, z=z, state=s, want_state=True), tfla.scan_backward(*args, dy, z=z, state=s)
    L = tfla.lib()
    flags = 0x100 | 0x1000
    ws = torch.empty(max(256, L.tfla_scan_workspace_bytes(1, 600, 64, 16, 1, flags),
                         L.tfla_scan_bwd_workspace_bytes(1, 600, 64, 16, 1, flags)), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = []
    with torch.cuda.stream(side):
        got.append((tfla.scan_forward(*args, z=z, state=s, want_state=True), tfla.scan_backward(*args, dy, z=z, state=s)))
    for kw in (dict(workspace=ws), dict(stream=side)):
        got.append((tfla.scan_forward(*args, z=z, state=s, want_state=True, **kw),
                    tfla.scan_backward(*args, dy, z=z, state=s, **kw)))
        torch.cuda.synchronize()
    for f, g in got:
        assert grads_equal(f, f0) and grads_equal(g, g0)


def test_captured_and_replayed():
    dev, _ = make(BF, 1, 600, 64, 16)
    x, dt, a, b, c, s, z, dy = (dev[k].cuda() for k in ("x", "dt", "a", "bmat", "cmat", "state", "z", "dy"))
    args = (x, dt, a, b, c)
    tfla.scan_forward(*args, z=z)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        f = tfla.scan_forward(*args, z=z, state=s, want_state=True)
        g = tfla.scan_backward(*args, dy, z=z, state=s)
    for _ in range(3):
        x.copy_(torch.randn_like(x))
        s.copy_(torch.randn_like(s))
        graph.replay()
        torch.cuda.synchronize()
        wf = tfla.scan_forward(*args, z=z, state=s, want_state=True)
        wg = tfla.scan_backward(*args, dy, z=z, state=s)
        torch.cuda.synchronize()
        assert grads_equal(f, wf) and grads_equal(g, wg)


def test_offsets_beyond_32_bits():
    """Batches 2^32 elements apart in one buffer."""
    T, D, N = 70, 64, 16
    far = (1 << 32) + 64
    dev, _ = make(BF, 2, T, D, N, state=False)
    x, dt, a, b, c, dy = (dev[k].cuda() for k in ("x", "dt", "a", "bmat", "cmat", "dy"))
    view, out = (torch.as_strided(torch.empty(far + T * D, dtype=BF, device="cuda"), (2, T, D), (far, D, 1)) for _ in range(2))
    view.copy_(x)
    want = tfla.scan_forward(x, dt, a, b, c)[0]
    assert torch.equal(tfla.scan_forward(view, dt, a, b, c, y=out)[0], want)
    assert torch.equal(tfla.scan_forward(view[:, :1], dt[:, :1], a, b[:, :1], c[:, :1], y=out[:, :1])[0], want[:, :1])
    g = tfla.scan_backward(x, dt, a, b, c, dy)
    assert grads_equal(tfla.scan_backward(view, dt, a, b, c, dy, dx=out), g)
    torch.cuda.synchronize()


@pytest.mark.parametrize("T", [1, 3, 4, 5])
def test_many_short_sequences(T):
    check(BF, 300, T, 40, 12, lengths=[min(T, i % 6) for i in range(300)])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_every_segment_of_a_padded_batch(dtype):
    """Sequences that end in the first, a middle and the last of many segments, one of them empty."""
    check(dtype, 4, 1030, 33, 16, lengths=[1030, 0, 65, 500])


def test_a_very_long_sequence():
    check(F32, 1, 20000, 5, 3)
