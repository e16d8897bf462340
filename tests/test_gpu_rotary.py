"""Rotary positions against the 64-bit reference.

An output a cos - b sin has its angle's product in fp64 (|angle| 2^-53, and as
much again in the reference), the reduced angle rounded to fp32 and its sine
and cosine within 6 U of them, the scale, two products and a sum: within
(12 U + |angle| 2^-51) scale (|a| + |b|), and half a step of its type."""
import numpy as np
import pytest
import torch

from blocks_helpers import HALF, U, randn, within
from mlstm_sequence_amd import tfla
from oracle import edges as O

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
NAN = float("nan")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    tfla.lib()


def as_heads(t, layout):
    """The CPU tensor [B,T,H,C] on the GPU: "plain"; "heads" head-major
    memory; "odd" heads one element longer; "by2", "by4", "by8" heads longer
    by that many elements, from that element on; "part" the middle of rows
    three times as wide."""
    t = t.cuda()
    B, T, H, C = t.shape
    if layout == "plain":
        return t
    if layout == "heads":
        return t.transpose(1, 2).contiguous().transpose(1, 2)
    if layout == "part":
        full = torch.full((B, T, 3 * H, C), NAN, dtype=t.dtype, device="cuda")
        full[:, :, H:2 * H] = t
        return full[:, :, H:2 * H]
    pad = {"odd": 1, "by2": 2, "by4": 4, "by8": 8}[layout]
    full = torch.full((B, T, H, C + pad), NAN, dtype=t.dtype, device="cuda")
    full[..., pad:] = t
    return full[..., pad:]


def check(dtype, B, T, H, Hk, C, R, interleaved=False, at="none", scale=1.0, lengths=None, layout="plain", out="plain",
          base=10000.0, seed=0, far=100000):
    print("rotary", dtype, B, T, H, Hk, C, R, interleaved, at, scale, lengths, layout, out, flush=True)
    rng = np.random.default_rng(seed + T + C + H)
    (tq, q), (tk, k) = randn(rng, (B, T, H, C), dtype), randn(rng, (B, T, max(Hk, 1), C), dtype)
    freqs, _ = tfla.rotary_frequencies(R, base)
    kw = dict(layout=tfla.ROTARY_INTERLEAVED if interleaved else tfla.ROTARY_HALVES, scale=scale)
    pos = np.broadcast_to(np.arange(T), (B, T))
    if at == "start":
        first = rng.integers(-far, far, B)
        kw["start"] = torch.tensor(first, dtype=torch.int32).cuda()
        pos = pos + first[:, None]
    elif at in ("given", "shared"):
        pos = np.broadcast_to(rng.integers(-far, far, (B if at == "given" else 1, T)), (B, T))
        p = torch.tensor(np.ascontiguousarray(pos), dtype=torch.int32).cuda()
        kw["positions"] = p if at == "given" else p[0]
    if lengths is not None:
        kw["lengths"] = torch.tensor(lengths, dtype=torch.int32).cuda()
        for b, n in enumerate(lengths):
            tq[b, max(0, n):] = NAN
            tk[b, max(0, n):] = NAN
    new = lambda t: as_heads(torch.full(t.shape, NAN, dtype=dtype), out)  # noqa: E731
    gq, gk = as_heads(tq, layout), as_heads(tk, layout) if Hk else None
    f = freqs.cpu().numpy()
    for inverse, call in ((False, tfla.rotary_forward), (True, tfla.rotary_backward)):
        oq, ok = call(gq, gk, freqs, q_out=new(tq), k_out=new(tk) if Hk else None, **kw)
        torch.cuda.synchronize()
        s = float(np.float32(scale))
        for name, got, x in (("q", oq, q), ("k", ok, k)):
            if name == "k" and not Hk:
                assert got is None
                continue
            want = O.rotary(x, pos, f, interleaved, s, lengths, inverse)
            mag = np.abs(x).copy()
            a, b = (mag[..., 0:R:2], mag[..., 1:R:2]) if interleaved else (mag[..., :R // 2], mag[..., R // 2:R])
            both = s * (a + b) * (12 * U + np.abs(pos[:, :, None, None] * f) * 2.0 ** -51)
            tol = np.zeros_like(mag)
            if interleaved:
                tol[..., 0:R:2], tol[..., 1:R:2] = both, both
            else:
                tol[..., :R // 2], tol[..., R // 2:R] = both, both
            tol[..., :R] += HALF[dtype] * np.abs(want[..., :R]) + 1e-37
            within(name, got, want, tol)                              # channels behind R: exact


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("C,R", [(64, 64), (128, 128), (128, 64), (80, 20), (96, 24), (7, 6), (64, 2), (5, 0), (256, 256), (1024, 1024)])
def test_head_sizes(dtype, interleaved, C, R):
    check(dtype, 2, 9, 3, 2, C, R, interleaved, at="start")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 130, 1000])
def test_lengths_of_one_call(dtype, T):
    check(dtype, 2, T, 4, 1, 64, 32)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("layout", ["heads", "odd", "by2", "by4", "by8", "part"])
@pytest.mark.parametrize("out", ["plain", "heads", "odd"])
def test_views(dtype, layout, out):
    for interleaved in (False, True):
        check(dtype, 2, 11, 3, 2, 64, 48, interleaved, layout=layout, out=out)


@pytest.mark.parametrize("H,Hk", [(1, 0), (32, 8), (3, 3), (40, 0), (128, 128)])
def test_heads(H, Hk):
    check(BF, 2, 5, H, Hk, 128, 128)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("at", ["start", "given", "shared"])
@pytest.mark.parametrize("far", [10, 10 ** 6, 2 ** 31 - 2000])
def test_positions(dtype, at, far):
    check(dtype, 3, 40, 2, 2, 32, 32, at=at, far=far, scale=1.277)


def test_start_beyond_32_bits():
    """start + t is formed in 64 bits."""
    T = 50
    x = torch.randn(1, T, 1, 16, device="cuda")
    freqs, _ = tfla.rotary_frequencies(16)
    got, _ = tfla.rotary_forward(x, None, freqs, start=torch.tensor([2 ** 31 - 10], dtype=torch.int32, device="cuda"))
    pos = np.arange(T)[None] + 2 ** 31 - 10
    x64 = x.double().cpu().numpy()
    mag = np.abs(x64[..., :8]) + np.abs(x64[..., 8:])
    tol = np.concatenate([mag, mag], -1) * (12 * U + 2.0 ** 31 * 2.0 ** -51) + 2 * U * 4
    within("far", got, O.rotary(x64, pos, freqs.cpu().numpy()), tol)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_padded_batches(dtype):
    check(dtype, 4, 33, 4, 2, 64, 64, lengths=[33, 0, 7, 40])
    check(dtype, 3, 33, 4, 2, 64, 32, interleaved=True, lengths=[-3, 1, 32], at="given", out="heads")


def test_in_place_and_head_major():
    freqs, _ = tfla.rotary_frequencies(64)
    for R in (64, 32):
        for kind in (tfla.ROTARY_HALVES, tfla.ROTARY_INTERLEAVED):
            qkv = torch.randn(2, 70, 12, 64, device="cuda").to(BF)
            q, k = qkv[:, :, :4], qkv[:, :, 4:8]
            f = freqs[:R // 2]
            wq, wk = tfla.rotary_forward(q, k, f, layout=kind, head_major=True)
            assert wq.shape == (2, 70, 4, 64) and wq.transpose(1, 2).is_contiguous()
            v = qkv[:, :, 8:].clone()
            gq, gk = tfla.rotary_forward(q, k, f, layout=kind, q_out=q, k_out=k)
            torch.cuda.synchronize()
            assert gq is q and torch.equal(q, wq) and torch.equal(k, wk) and torch.equal(qkv[:, :, 8:], v)


def test_special_values_stay_in_their_pair():
    """Infinities and NaN reach their own pair alone; a broadcast head gives every head's turn."""
    freqs, _ = tfla.rotary_frequencies(8)
    x = torch.randn(1, 6, 2, 10, device="cuda")
    x[0, 3, 1, 1], x[0, 4, 0, 2] = NAN, float("inf")
    y, _ = tfla.rotary_forward(x, None, freqs)
    bad = ~torch.isfinite(y)
    want = torch.zeros_like(bad)
    want[0, 3, 1, [1, 5]] = True
    want[0, 4, 0, [2, 6]] = True
    torch.cuda.synchronize()
    assert torch.equal(bad, want)
    one = torch.randn(2, 6, 1, 8, device="cuda")
    wide, _ = tfla.rotary_forward(one.expand(2, 6, 5, 8), None, freqs)
    want, _ = tfla.rotary_forward(one, None, freqs)
    torch.cuda.synchronize()
    assert torch.equal(wide, want.expand(2, 6, 5, 8))


def test_relative_positions():
    """Scores of rotated queries and keys depend on the distance alone."""
    freqs, s = tfla.rotary_frequencies(64, scaling="yarn", factor=8.0, original_length=4096)
    q, k = torch.randn(1, 1, 1, 64, device="cuda"), torch.randn(1, 1, 1, 64, device="cuda")

    def score(a, b):
        at = lambda n: torch.tensor([n], dtype=torch.int32, device="cuda")  # noqa: E731
        return float((tfla.rotary_forward(q, None, freqs, start=at(a))[0].double()
                      * tfla.rotary_forward(k, None, freqs, start=at(b))[0].double()).sum())

    big = float((q.abs() * k.abs()).sum()) * 2
    assert abs(score(5, 2) - score(1000005, 1000002)) <= 60 * U * big


def test_refusals_on_tensors():
    q, k = torch.randn(2, 10, 4, 32, device="cuda"), torch.randn(2, 10, 2, 32, device="cuda")
    f, _ = tfla.rotary_frequencies(32)
    i32 = dict(dtype=torch.int32, device="cuda")
    for bad in (dict(freqs=f.float()), dict(freqs=f.cpu()), dict(freqs=f[None]), dict(freqs=torch.cat([f, f])), dict(freqs=f[::2]),
                dict(k=k.to(BF)), dict(k=k[:1]), dict(k=k[0]), dict(k=k[..., :16]), dict(q=q.transpose(2, 3)),
                dict(start=torch.zeros(3, **i32)), dict(start=torch.zeros(2, device="cuda")), dict(positions=torch.zeros(9, **i32)),
                dict(positions=torch.zeros(2, 20, **i32)[:, ::2]), dict(positions=torch.zeros(2, 10, dtype=torch.int64, device="cuda")),
                dict(start=torch.zeros(2, **i32), positions=torch.zeros(2, 10, **i32)), dict(lengths=torch.zeros(2, 1, **i32)),
                dict(layout=1), dict(q_out=k), dict(q_out=q[:, :, :1].expand_as(q)), dict(k=None, k_out=k)):
        kw = dict(q=q, k=k, freqs=f)
        kw.update(bad)
        with pytest.raises((TypeError, ValueError, tfla.TflaError)):
            tfla.rotary_forward(**kw)


def test_captured_and_replayed():
    """The positions are read when the graph runs: a token's step counts them up."""
    q, k = torch.randn(3, 1, 4, 64, device="cuda").to(BF), torch.randn(3, 1, 2, 64, device="cuda").to(BF)
    f, _ = tfla.rotary_frequencies(64)
    start = torch.tensor([5, 0, 77], dtype=torch.int32, device="cuda")
    tfla.rotary_forward(q, k, f, start=start)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = tfla.rotary_forward(q, k, f, start=start, head_major=True)
    for _ in range(3):
        start.add_(1)
        graph.replay()
        want = tfla.rotary_forward(q, k, f, start=start)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_offsets_beyond_32_bits():
    far = (1 << 32) + 64
    full = [torch.empty(far + 5 * 64, dtype=BF, device="cuda") for _ in range(2)]
    view, out = (torch.as_strided(t, (2, 5, 2, 32), (far, 64, 32, 1)) for t in full)
    x = torch.randn(2, 5, 2, 32, device="cuda").to(BF)
    view.copy_(x)
    f, _ = tfla.rotary_frequencies(32)
    got, _ = tfla.rotary_forward(view, None, f, q_out=out)
    want, _ = tfla.rotary_forward(x, None, f)
    torch.cuda.synchronize()
    assert torch.equal(got, want)


def test_very_many_sequences():
    """More workgroups than one dimension of a grid holds."""
    B = (1 << 21) + 3
    x = torch.randn(B, 1, 1, 4, device="cuda")
    freqs, _ = tfla.rotary_frequencies(4)
    start = torch.arange(B, dtype=torch.int32, device="cuda")
    y, _ = tfla.rotary_forward(x, None, freqs, start=start)
    ang = start.double()[:, None] * freqs
    a, b = x[:, 0, 0, :2].double(), x[:, 0, 0, 2:].double()
    want = torch.cat([a * ang.cos() - b * ang.sin(), b * ang.cos() + a * ang.sin()], -1)
    tol = (12 * U + 2.0 ** 22 * 2.0 ** -51) * (a.abs() + b.abs()).repeat(1, 2) + U * want.abs()
    torch.cuda.synchronize()
    assert bool(((y[:, 0, 0] - want).abs() <= tol).all())
