"""Causal depthwise convolution against the 64-bit reference."""
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


def make(dtype, B, T, D, K, bias=True, state=True, lengths=None, seed=0):
    rng = np.random.default_rng(seed + 13 * T + D)
    d = dict(x=randn(rng, (B, T, D), dtype), w=randn(rng, (D, K), F32, 0.5), bias=randn(rng, (D,), F32) if bias else None,
             state=randn(rng, (B, K - 1, D), dtype) if state and K > 1 else None, dy=randn(rng, (B, T, D), dtype),
             dend=randn(rng, (B, K - 1, D), dtype) if state and K > 1 else None)
    dev = {k: None if v is None else v[0] for k, v in d.items()}
    ref = {k: None if v is None else v[1] for k, v in d.items()}
    if lengths is not None:   # what lies behind a sequence must not matter
        for k in ("x", "dy"):
            for b, n in enumerate(lengths):
                dev[k][b, max(0, n):] = NAN
    dev["lengths"] = None if lengths is None else torch.tensor(lengths, dtype=torch.int32)
    return dev, ref


def check(dtype, B, T, D, K, act="silu", view="plain", bias=True, state=True, lengths=None):
    print("conv", dtype, B, T, D, K, act, view, bias, state, lengths, flush=True)
    dev, ref = make(dtype, B, T, D, K, bias, state, lengths)
    kind = tfla.ACT_SILU if act == "silu" else tfla.ACT_NONE
    x, dy = as_view(dev["x"], view), as_view(dev["dy"], view)
    w, b, s, ln, de = (cuda(dev[k]) for k in ("w", "bias", "state", "lengths", "dend"))
    y = as_view(torch.full((B, T, D), NAN, dtype=dtype), view)
    got, end = tfla.conv_forward(x, w, b, act=kind, state=s, lengths=ln, want_state=True, y=y)
    assert got is y
    dx = as_view(torch.full((B, T, D), NAN, dtype=dtype), view)
    g = tfla.conv_backward(x, w, dy, b, act=kind, state=s, lengths=ln, dstate_out=de, dx=dx)
    torch.cuda.synchronize()

    r = {k: ref[k] for k in ("x", "w", "bias", "state", "dy", "dend")}
    want, wend = O.conv(r["x"], r["w"], r["bias"], act, r["state"], lengths)
    ab = {k: None if v is None else np.abs(v) for k, v in r.items()}
    # u: K products and the bias; |SiLU'| <= 1.1, and the sigmoid itself within 6 U relative
    mag, _ = O.conv(ab["x"], ab["w"], ab["bias"], "none", ab["state"], lengths)
    du = (K + 2) * U * mag
    h = HALF[dtype]
    within("y", y, want, h * np.abs(want) + 1.1 * du + 8 * U * np.abs(want) + 1e-38)
    within("state_out", end, wend, 0.0)
    # du = dy act'(u): |act''| <= 0.5, act' within 12 U; the rest are sums of K (dx) or B T (dw) products.
    # B T + 16 of them at most in any order.
    gx, gw, gb, gs = O.conv_grads(r["x"], r["w"], r["dy"], r["bias"], act, r["state"], lengths, r["dend"])
    one = np.ones_like(want) if act == "none" else 1.1
    slack = (0.5 * du + 12 * U) if act == "silu" else 0.0   # of act'(u), absolute
    full = ab["dy"] * one
    lin = dict(kind="none", lengths=lengths)
    mx, mw, mb, ms = O.conv_grads(ab["x"], ab["w"], full, ab["bias"], state=ab["state"], dend=ab["dend"], **lin)
    ex, ew, eb, es = O.conv_grads(ab["x"], ab["w"], ab["dy"] * slack, ab["bias"], state=ab["state"], **lin)
    within("dx", dx, gx, h * np.abs(gx) + (K + 2) * U * mx + ex + 1e-38)
    n = (B * T + 16) * U
    within("dweight", g[1], gw, n * mw + ew + U * np.abs(gw))
    if bias:
        within("dbias", g[2], gb, n * mb + eb + U * np.abs(gb))
    else:
        assert g[2] is None
    if s is not None:
        within("dstate", g[3], gs, h * np.abs(gs) + (K + 2) * U * ms + es + 1e-38)
    else:
        assert g[3] is None


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("K", [1, 2, 3, 4, 5, 8])
def test_taps(dtype, K):
    check(dtype, 2, 70, 24, K)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T", [1, 2, 3, 4, 7, 8, 9, 63, 64, 65, 257])
def test_lengths_of_one_call(dtype, T):
    check(dtype, 2, T, 16, 4, act="silu" if T % 2 else "none")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D", [1, 5, 8, 12, 64, 264, 1001])
@pytest.mark.parametrize("view", ["plain", "half", "odd", "wide", "time"])
def test_widths_and_views(dtype, D, view):
    check(dtype, 3, 19, D, 4, view=view, bias=D % 2 == 0, state=view != "half")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("K", [4, 8])
def test_padded_batch(dtype, K):
    check(dtype, 6, 130, 40, K, lengths=[130, 0, 1, 2, 77, 129])


def test_lengths_out_of_range_are_clamped():
    dev, ref = make(BF, 3, 20, 8, 4)
    x, w, s = dev["x"].cuda(), dev["w"].cuda(), dev["state"].cuda()
    got = tfla.conv_forward(x, w, state=s, want_state=True, lengths=torch.tensor([-5, 20, 1 << 30], dtype=torch.int32).cuda())
    want = tfla.conv_forward(x, w, state=s, want_state=True, lengths=torch.tensor([0, 20, 20], dtype=torch.int32).cuda())
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_prompt_then_single_tokens_equal_one_call(dtype):
    """The state carries exact inputs, so the rows agree bit for bit."""
    dev, _ = make(dtype, 3, 21, 72, 4, state=False)
    x, w, b = dev["x"].cuda(), dev["w"].cuda(), dev["bias"].cuda()
    y, end = tfla.conv_forward(x, w, b, want_state=True)
    parts = []
    p, st = tfla.conv_forward(x[:, :2], w, b, want_state=True)
    parts.append(p)
    for t in range(2, 21):
        p, again = tfla.conv_forward(x[:, t:t + 1], w, b, state=st, state_out=st)   # updated in place
        assert again is st
        parts.append(p)
    torch.cuda.synchronize()
    assert torch.equal(torch.cat(parts, 1), y) and torch.equal(st, end)


def test_halves_of_one_buffer_as_outputs():
    """dx written into one half of a projection's gradient leaves the other half alone."""
    dev, _ = make(BF, 2, 50, 32, 4)
    x, w, dy = dev["x"].cuda(), dev["w"].cuda(), dev["dy"].cuda()
    both = torch.full((2, 50, 64), 7.0, dtype=BF, device="cuda")
    tfla.conv_backward(x, w, dy, dx=both[..., 32:])
    want = tfla.conv_backward(x, w, dy)[0]
    torch.cuda.synchronize()
    assert torch.equal(both[..., 32:], want) and bool((both[..., :32] == 7.0).all())


def test_refusals_on_tensors():
    dev, _ = make(BF, 2, 10, 16, 4)
    x, w, b, s, dy = (dev[k].cuda() for k in ("x", "w", "bias", "state", "dy"))
    for bad in (dict(weight=w.bfloat16()), dict(weight=w[:8]), dict(bias=b[:4]), dict(state=s.float()), dict(state=s[:1]),
                dict(x=x.transpose(1, 2)), dict(lengths=torch.tensor([1, 2]).cuda()), dict(weight=w.t().contiguous().t()),
                dict(y=x), dict(y=x.new_zeros(2, 10, 8)), dict(weight=w.cpu())):
        kw = dict(x=x, weight=w, bias=b, state=s)
        kw.update(bad)
        with pytest.raises((TypeError, ValueError, tfla.TflaError)):
            tfla.conv_forward(**kw)
    with pytest.raises(ValueError):
        tfla.conv_backward(x, w, dy[:, :5])
    with pytest.raises(tfla.TflaError):
        tfla.conv_backward(x, w, dy, dx=dy)
    with pytest.raises(ValueError):
        tfla.conv_backward(x, w, dy, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))


def test_stream_workspace_and_repeat():
    """Another stream, the caller's workspace and the library's own allocation give the same bits."""
    dev, _ = make(BF, 2, 333, 136, 4)
    x, w, b, s, dy = (dev[k].cuda() for k in ("x", "w", "bias", "state", "dy"))
    want = tfla.conv_backward(x, w, dy, b, state=s)
    ws = torch.empty(tfla.lib().tfla_conv_bwd_workspace_bytes(2, 333, 136, 4, 0x100), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        a = tfla.conv_backward(x, w, dy, b, state=s)
    c = tfla.conv_backward(x, w, dy, b, state=s, workspace=ws)
    e = tfla.conv_backward(x, w, dy, b, state=s, stream=side)   # allocated by the library on that stream
    torch.cuda.synchronize()
    for got in (a, c, e):
        assert all(torch.equal(p, q) for p, q in zip(got, want))


def test_captured_and_replayed():
    dev, _ = make(BF, 2, 40, 64, 4)
    x, w, b, s, dy = (dev[k].cuda() for k in ("x", "w", "bias", "state", "dy"))
    tfla.conv_forward(x, w, b, state=s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, end = tfla.conv_forward(x, w, b, state=s, want_state=True)
        g = tfla.conv_backward(x, w, dy, b, state=s)
    for i in range(3):
        x.copy_(torch.randn_like(x))
        dy.copy_(torch.randn_like(dy))
        graph.replay()
        torch.cuda.synchronize()
        wy, wend = tfla.conv_forward(x, w, b, state=s, want_state=True)
        wg = tfla.conv_backward(x, w, dy, b, state=s)
        torch.cuda.synchronize()
        assert torch.equal(y, wy) and torch.equal(end, wend)
        assert all(torch.equal(p, q) for p, q in zip(g, wg))


def test_offsets_beyond_32_bits():
    """Batches 2^32 elements apart in one buffer."""
    T, D, K = 9, 128, 4
    far = (1 << 32) + 128
    view, out = (torch.as_strided(torch.empty(far + T * D, dtype=BF, device="cuda"), (2, T, D), (far, D, 1)) for _ in range(2))
    x, w = torch.randn(2, T, D, device="cuda").to(BF), torch.randn(D, K, device="cuda")
    view.copy_(x)
    assert torch.equal(tfla.conv_forward(view, w, y=out)[0], tfla.conv_forward(x, w)[0])
    got, want = tfla.conv_backward(view, w, view, dx=out), tfla.conv_backward(x, w, x)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    torch.cuda.synchronize()


def test_many_short_sequences():
    """More sequences than a run of rows is long, one and two rows each."""
    for T in (1, 2):
        check(BF, 700, T, 72, 4, lengths=[T * (i % 3 > 0) for i in range(700)])


def test_a_very_long_sequence():
    check(F32, 1, 30000, 3, 4)
