"""Where a call on a given stream takes the memory of its outputs and its
workspace from: that stream's, not the current one's."""
import ctypes

import pytest
import torch

from mlstm_sequence_amd import blocks, tfla

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    tfla.lib()


def calls():
    """name -> a call with keyword arguments that returns its outputs"""
    r = lambda *s: torch.randn(*s, device="cuda")  # noqa: E731
    B, T, D, N, K = 2, 700, 64, 16, 4
    x, dt, z, dy = (r(B, T, D).to(BF) for _ in range(4))
    bm, cm = r(B, T, 1, N).to(BF), r(B, T, 1, N).to(BF)
    w, b, cs = r(D, K), r(D), r(B, K - 1, D).to(BF)
    a, sk, db, ss = -torch.exp(r(D, N) * 0.3), r(D), r(D), r(B, D, N)
    h, g, dh, nw, nb = r(B, T, 4, 16).to(BF), r(B, T, 4, 16).to(BF), r(B, T, 4, 16).to(BF), r(4, 16), r(4, 16)
    kw = dict(skip=sk, z=z, dt_bias=db, state=ss)
    out = {"conv_forward": lambda **k: tfla.conv_forward(x, w, b, state=cs, want_state=True, **k),
           "conv_backward": lambda **k: tfla.conv_backward(x, w, dy, b, state=cs, **k),
           "scan_forward": lambda **k: tfla.scan_forward(x, dt, a, bm, cm, want_state=True, **kw, **k),
           "scan_backward": lambda **k: tfla.scan_backward(x, dt, a, bm, cm, dy, **kw, **k)}
    for name, over in (("token", tfla.NORM_TOKEN), ("sequence", tfla.NORM_SEQUENCE)):
        nk = dict(act=tfla.ACT_SILU, gate=g, over=over)
        _, m, s = tfla.norm_forward(h, nw, nb, **nk)
        out["norm_forward " + name] = lambda nk=nk, **k: tfla.norm_forward(h, nw, nb, **nk, **k)
        out["norm_backward " + name] = lambda nk=nk, m=m, s=s, **k: tfla.norm_backward(h, dh, m, s, nw, nb, **nk, **k)
    q, k_, v, dv = r(2, 2, 300, 64).to(BF), r(2, 2, 300, 64).to(BF), r(2, 2, 300, 64).to(BF), r(2, 2, 300, 64).to(BF)
    ig, fg = r(2, 2, 300), r(2, 2, 300) + 3
    out["forward"] = lambda **k: (tfla.forward(q, k_, v, ig, fg, tfla.MLSTM_SIG, 64, **k),)
    out["backward"] = lambda **k: tfla.backward(q, k_, v, ig, fg, dv, tfla.MLSTM_SIG, 64, **k)
    return out


def home(t):
    """Handle of the stream whose memory the tensor lies in."""
    p = t.untyped_storage().data_ptr()
    return next(s["stream"] for s in torch.cuda.memory_snapshot() if s["address"] <= p < s["address"] + s["total_size"])


NAMES = ["conv_forward", "conv_backward", "scan_forward", "scan_backward", "norm_forward token", "norm_backward token",
         "norm_forward sequence", "norm_backward sequence", "forward", "backward"]


@pytest.mark.parametrize("how", ["stream", "handle"])
@pytest.mark.parametrize("name", NAMES)
def test_outputs_lie_in_the_given_streams_memory(name, how):
    call = calls()[name]
    side = torch.cuda.Stream()
    want = call()
    torch.cuda.synchronize()
    got = call(stream=side if how == "stream" else side.cuda_stream)
    torch.cuda.synchronize()
    assert torch.cuda.current_stream() == torch.cuda.default_stream()
    for g, w in zip(got, want):
        assert home(g) == side.cuda_stream and home(w) == torch.cuda.default_stream().cuda_stream
        assert torch.equal(g, w)


@pytest.mark.parametrize("name", NAMES)
def test_the_null_stream_by_its_handle(name):
    """Handle 0 is the default stream, also while another one is current."""
    call = calls()[name]
    want = call()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = call(stream=0)
        here = call(stream=side)
    torch.cuda.synchronize()
    for g, h, w in zip(got, here, want):
        assert home(g) == 0 and home(h) == side.cuda_stream
        assert torch.equal(g, w) and torch.equal(h, w)


def test_workspaces_of_the_library_itself():
    """A NULL workspace is allocated in the stream's order by the library."""
    B, T, D, N = 2, 700, 64, 16
    x, dt, dy = (torch.randn(B, T, D, device="cuda") for _ in range(3))
    bm, cm, a = torch.randn(B, T, 1, N, device="cuda"), torch.randn(B, T, 1, N, device="cuda"), -torch.rand(D, N, device="cuda")
    wy, wend = tfla.scan_forward(x, dt, a, bm, cm, want_state=True)
    wg = tfla.scan_backward(x, dt, a, bm, cm, dy)
    y, end, dx, ddt, db, dc, da = (torch.empty_like(t) for t in (wy, wend, wg.dx, wg.ddt, wg.dbmat, wg.dcmat, wg.da))
    rows = lambda t: blocks.Rows(t.data_ptr(), t.stride(0), t.stride(1))  # noqa: E731
    args = blocks.ScanArgs(B=B, T=T, D=D, N=N, G=1, flags=blocks.SCAN_SOFTPLUS, x=rows(x), dt=rows(dt), bmat=rows(bm),
                           cmat=rows(cm), a=a.data_ptr(), y=rows(y), state_out=end.data_ptr(), dy=rows(dy), dx=rows(dx),
                           ddt=rows(ddt), dbmat=rows(db), dcmat=rows(dc), da=da.data_ptr())
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    L = tfla.lib()
    for _ in range(2):
        tfla._check(L.tfla_scan_fwd(ctypes.byref(args), None, 0, side.cuda_stream), "tfla_scan_fwd")
        tfla._check(L.tfla_scan_bwd(ctypes.byref(args), None, 0, side.cuda_stream), "tfla_scan_bwd")
        torch.cuda.synchronize()
        for g, w in ((y, wy), (end, wend), (dx, wg.dx), (ddt, wg.ddt), (db, wg.dbmat), (dc, wg.dcmat), (da, wg.da)):
            assert torch.equal(g, w)
            g.zero_()
        torch.cuda.synchronize()


@pytest.mark.parametrize("name", NAMES[:8])
def test_a_given_stream_inside_a_capture(name):
    """A call on a side stream that a capture has forked to and joins again."""
    call = calls()[name]
    want = call()
    torch.cuda.synchronize()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        got = call(stream=side)
        torch.cuda.current_stream().wait_stream(side)
    for _ in range(3):
        for g in got:
            g.zero_()
        graph.replay()
        torch.cuda.synchronize()
        again = call()
        torch.cuda.synchronize()
        assert all(torch.equal(g, w) and torch.equal(a, w) for g, a, w in zip(got, again, want))
