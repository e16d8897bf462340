"""The operators around the recurrences as a model uses them together: the
convolution in front, the scan (or the mLSTM) behind it, the gated norm at the
end; trained, and served as prompts followed by single tokens."""
import numpy as np
import pytest
import torch

import oracle
import workloads as W
from gpu_helpers import TOL, h_f64, rel_err
from mlstm_sequence_amd import tfla
from oracle import blocks as O

pytestmark = pytest.mark.gpu
F32, BF = torch.float32, torch.bfloat16

# fp32 data: each of the three operators stays within about 100 half-steps of fp32 of its terms' magnitudes (their
# own tests), terms cancel to a tenth here, and three operators follow each other, once forward and once backward:
# 2 * 3 * 100 * 10 * 2^-24, relative to the largest value.
CHAIN = 6000 * 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    tfla.lib()


class Block:
    """One block: a projection's output [B,T,2D] holds the convolution's input and the gate."""

    def __init__(self, D, N, H, K=4, seed=0, dtype=F32):
        g = torch.Generator().manual_seed(seed)
        self.D, self.N, self.H = D, N, H
        self.w, self.b = torch.randn(D, K, generator=g) * 0.4, torch.randn(D, generator=g) * 0.1
        self.a = -torch.exp(torch.randn(D, N, generator=g) * 0.3)
        self.skip, self.dt_bias = torch.randn(D, generator=g), torch.randn(D, generator=g) * 0.3 - 1
        self.nw, self.nb = 1 + 0.2 * torch.randn(H, D // H, generator=g), 0.1 * torch.randn(H, D // H, generator=g)
        for k in ("w", "b", "a", "skip", "dt_bias", "nw", "nb"):
            setattr(self, k, getattr(self, k).cuda())

    def forward(self, xz, dt, bm, cm, conv_state=None, scan_state=None, lengths=None):
        B, T, D, H = xz.shape[0], xz.shape[1], self.D, self.H
        x, z = xz[..., :D], xz[..., D:]
        u, cs = tfla.conv_forward(x, self.w, self.b, state=conv_state, lengths=lengths, want_state=True)
        s, ss = tfla.scan_forward(u, dt, self.a, bm, cm, skip=self.skip, dt_bias=self.dt_bias, state=scan_state,
                                  lengths=lengths, want_state=True)
        y, m, r = tfla.norm_forward(s.view(B, T, H, D // H), self.nw, self.nb, act=tfla.ACT_SILU,
                                    gate=z.unflatten(-1, (H, D // H)))
        self.saved = (x, z, u, s, m, r, dt, bm, cm, lengths)
        return y.flatten(2), cs, ss

    def backward(self, dy):
        x, z, u, s, m, r, dt, bm, cm, lengths = self.saved
        B, T, D, H = x.shape[0], x.shape[1], self.D, self.H
        dxz = torch.full((B, T, 2 * D), float("nan"), dtype=x.dtype, device="cuda")
        heads = (H, D // H)
        ds, _, dnw, dnb = tfla.norm_backward(s.unflatten(-1, heads), dy.unflatten(-1, heads), m, r, self.nw, self.nb,
                                             act=tfla.ACT_SILU, gate=z.unflatten(-1, heads),
                                             dgate=dxz[..., D:].unflatten(-1, heads))
        g = tfla.scan_backward(u, dt, self.a, bm, cm, ds.flatten(2), skip=self.skip, dt_bias=self.dt_bias, lengths=lengths)
        _, dw, db, _ = tfla.conv_backward(x, self.w, g.dx, self.b, lengths=lengths, dx=dxz[..., :D])
        return dict(xz=dxz, dt=g.ddt, bm=g.dbmat, cm=g.dcmat, a=g.da, skip=g.dskip, dt_bias=g.ddt_bias, w=dw, b=db,
                    nw=dnw, nb=dnb)


def reference(blk, xz, dt, bm, cm, lengths):
    """The block in 64 bits on the CPU, by torch operations that differentiate themselves."""
    p = {k: getattr(blk, k).double().cpu().requires_grad_() for k in ("w", "b", "a", "skip", "dt_bias", "nw", "nb")}
    p.update(xz=xz.double().cpu().requires_grad_(), dt=dt.double().cpu().requires_grad_(),
             bm=bm.double().cpu().requires_grad_(), cm=cm.double().cpu().requires_grad_())
    B, T, D, H = xz.shape[0], xz.shape[1], blk.D, blk.H
    K = p["w"].shape[1]
    live = torch.arange(T)[None, :] < torch.tensor(lengths)[:, None]
    x, z = p["xz"][..., :D], p["xz"][..., D:]
    x = torch.where(live[..., None], x, 0.0)
    pad = torch.cat([torch.zeros(B, K - 1, D, dtype=torch.float64), x], 1)
    u = torch.nn.functional.silu(sum(pad[:, j:j + T] * p["w"][:, j] for j in range(K)) + p["b"])
    delta = torch.nn.functional.softplus(p["dt"] + p["dt_bias"])
    h = torch.zeros(B, D, blk.N, dtype=torch.float64)
    rows, ends = [], []
    per = D // bm.shape[2]
    for t in range(T):
        Bt, Ct = (p[k][:, t].repeat_interleave(per, 1) for k in ("bm", "cm"))
        n = torch.exp(delta[:, t, :, None] * p["a"]) * h + (delta[:, t] * u[:, t])[..., None] * Bt
        h = torch.where(live[:, t, None, None], n, h)
        o = (h * Ct).sum(-1) + p["skip"] * u[:, t]
        rows.append(torch.where(live[:, t, None], o, 0.0))
    s = torch.stack(rows, 1).unflatten(-1, (H, D // H))
    m = s.mean(-1, keepdim=True)
    r = torch.rsqrt(((s - m) ** 2).mean(-1, keepdim=True) + 1e-5)
    y = ((s - m) * r * p["nw"] + p["nb"]) * torch.nn.functional.silu(z.unflatten(-1, (H, D // H)))
    return y.flatten(2), h, p


def close(name, got, want, rel=CHAIN):
    got, want = got.detach().cpu().double().numpy(), want.detach().numpy()
    err = np.abs(got - want).max() / max(np.abs(want).max(), 1e-30)
    print(f"{name}: {err:.2e}", flush=True)
    assert err <= rel, (name, err)


def inputs(B, T, D, N, G, seed=1):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g).cuda()  # noqa: E731
    return r(B, T, 2 * D), r(B, T, D), r(B, T, G, N), r(B, T, G, N)


def test_training_step_of_a_block():
    B, T, D, N, G, H = 3, 45, 64, 8, 2, 4
    blk, lengths = Block(D, N, H), [45, 17, 40]
    xz, dt, bm, cm = inputs(B, T, D, N, G)
    ln = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    y, _, _ = blk.forward(xz, dt, bm, cm, lengths=ln)
    dy = torch.randn(B, T, D, generator=torch.Generator().manual_seed(9))
    live = (torch.arange(T)[None, :] < torch.tensor(lengths)[:, None])[..., None]
    dy = torch.where(live, dy, 0.0)   # padded rows carry no loss
    got = blk.backward(dy.cuda())
    torch.cuda.synchronize()
    want, _, p = reference(blk, xz, dt, bm, cm, lengths)
    close("y", y.cpu() * live, want * live)
    (want * dy.double()).sum().backward()
    for k, v in got.items():
        close(k, v, p[k].grad)


def test_prompts_then_single_tokens():
    """A padded batch of prompts, then one token at a time with the states
    updated in place, against each sequence in one go."""
    B, T, D, N, G, H, more = 4, 33, 128, 16, 1, 2, 6
    blk, lengths = Block(D, N, H, seed=4), [33, 1, 20, 5]
    xz, dt, bm, cm = inputs(B, T + more, D, N, G, seed=5)
    # sequence b's rows: its prompt, then the tokens that follow (rows T ..)
    ln = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    y, cs, ss = blk.forward(xz[:, :T], dt[:, :T], bm[:, :T], cm[:, :T], lengths=ln)
    tokens = []
    for t in range(T, T + more):
        u, _ = tfla.conv_forward(xz[:, t:t + 1, :D], blk.w, blk.b, state=cs, state_out=cs)
        s, _ = tfla.scan_forward(u, dt[:, t:t + 1], blk.a, bm[:, t:t + 1], cm[:, t:t + 1], skip=blk.skip,
                                 dt_bias=blk.dt_bias, state=ss, state_out=ss)
        o, _, _ = tfla.norm_forward(s.view(B, 1, H, D // H), blk.nw, blk.nb, act=tfla.ACT_SILU,
                                    gate=xz[:, t:t + 1, D:].unflatten(-1, (H, D // H)))
        tokens.append(o.flatten(2))
    tokens = torch.cat(tokens, 1)
    torch.cuda.synchronize()
    for b, n in enumerate(lengths):
        rows = list(range(n)) + list(range(T, T + more))
        one = [v[b:b + 1, rows].contiguous() for v in (xz, dt, bm, cm)]
        want, end, _ = reference(blk, *one, [len(rows)])
        close(f"prompt {b}", y[b:b + 1, :n], want[:, :n])
        close(f"tokens {b}", tokens[b:b + 1], want[:, n:])
        close(f"state {b}", ss[b:b + 1], end)


def test_convolution_mlstm_and_gated_norm():
    """q and k from the convolution's output, the mLSTM, and its head-major
    output normalised, gated and laid out for a projection, in bf16; each
    stage against the reference of what it was given."""
    B, H, T, d, dhv = 2, 4, 200, 64, 128
    g = torch.Generator().manual_seed(2)
    x = torch.randn(B, T, H * d, generator=g).to(BF)
    w, b = torch.randn(H * d, 4, generator=g) * 0.4, torch.randn(H * d, generator=g) * 0.1
    v = torch.randn(B, H, T, dhv, generator=g).to(BF)
    ig, fg = torch.randn(B, H, T, generator=g), torch.randn(B, H, T, generator=g) + 3
    gate = torch.randn(B, T, H, dhv, generator=g).to(BF)
    u, _ = tfla.conv_forward(x.cuda(), w.cuda(), b.cuda())
    qk = u.view(B, T, H, d).transpose(1, 2).contiguous()
    h = tfla.forward(qk, qk, v.cuda(), ig.cuda(), fg.cuda(), tfla.MLSTM_SIG, 64)
    y, _, _ = tfla.norm_forward(h.transpose(1, 2), act=tfla.ACT_SIGMOID, gate=gate.cuda())
    torch.cuda.synchronize()
    assert rel_err(h_f64(u), O.conv(x.double().numpy(), w.double().numpy(), b.double().numpy())[0]) <= TOL[BF]
    q64 = qk.double().cpu().numpy()
    ref = oracle.recurrent_fwd(q64, q64, v.double().numpy(), ig.double().numpy(), fg.double().numpy(), W.MLSTM_SIG)
    assert rel_err(h_f64(h), ref) <= TOL[BF]
    want = O.norm(h.transpose(1, 2).double().cpu().numpy(), kind="sigmoid", gate=gate.double().numpy())[0]
    assert rel_err(h_f64(y), want) <= TOL[BF]


def test_two_captured_graphs_and_two_streams():
    """Two graphs of the same block, replayed in turn with eager work between,
    and two streams at once: every call has workspace of its own."""
    B, T, D, N, G, H = 1, 400, 64, 16, 1, 2
    blk = Block(D, N, H, seed=7)
    sets = [inputs(B, T, D, N, G, seed=20 + i) for i in range(2)]
    dy = torch.randn(B, T, D, device="cuda")

    def step(i):
        y, cs, ss = blk.forward(*sets[i])
        return [y, cs, ss] + list(blk.backward(dy).values())

    want = [step(i) for i in range(2)]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for i in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[i]):
            outs.append(step(i))
    for _ in range(3):
        for i in range(2):
            graphs[i].replay()
        eager = step(0)
        torch.cuda.synchronize()
        for i in range(2):
            assert all(torch.equal(p, q) for p, q in zip(outs[i], want[i]))
        assert all(torch.equal(p, q) for p, q in zip(eager, want[0]))
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [None, None]
    for _ in range(5):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                got[i] = step(i)
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(p, q) for p, q in zip(got[i], want[i]))
