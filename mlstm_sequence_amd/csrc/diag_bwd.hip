// diag_bwd.hip -- gated linear recurrence of channels, backward (diag_impl.hpp).
//
// The walk of the forward pass from the end: with a_t = f_t g_t, what row t
// hands to row t - 1, a tile's rows are a map of the state, h -> F h + H, and
// one of the adjoint, a -> F a + A, with the same F.  A lane forms both maps of
// its rows, halves and waves join theirs as in the forward pass, and each lane
// then runs its rows forward from the state before them (the chunk's start,
// which the forward pass left) and backward from the adjoint behind them.
// Inputs and dy are read once, the gradients written once: bound by memory.
// The gates stay in registers between the two.
//
// A long axis over few channels is cut into segments, whose adjoint maps are
// formed first from fgate and dy alone.
#include "diag_impl.hpp"
#include "sums.hpp"

namespace tfla {
namespace {

using namespace diag;

constexpr int kPer = 16, kTile = kWaves * kPer;
static_assert(kTile == kChunk, "a tile starts where the forward pass left a state");

// The adjoint behind segment `seg`: dstate_out through the maps of the segments from the last on.
template <int V>
__device__ __forceinline__ void adjoint_behind(const DiagProblem& p, const Segments& sg, const Place& q, int cc,
                                               const f32x2* ends, float* a)
{
#pragma unroll
    for (int k = 0; k < V; ++k) a[k] = p.dstate_out ? p.dstate_out[q.b * p.D + cc + k] : 0.0f;
    constexpr int LINKS = 8;                           // in batches, whose loads are under way together
    const f32x2* e = ends + q.b * sg.nseg * p.D + cc;
    for (int j0 = sg.nseg - 1; j0 > q.seg; j0 -= LINKS) {
        f32x2 m[LINKS][V];
#pragma unroll
        for (int j = 0; j < LINKS; ++j)
#pragma unroll
            for (int k = 0; k < V; ++k) m[j][k] = e[(int64_t)max(j0 - j, q.seg + 1) * p.D + k];
#pragma unroll
        for (int j = 0; j < LINKS; ++j)
            if (j0 - j > q.seg)
#pragma unroll
                for (int k = 0; k < V; ++k) a[k] = m[j][k][0] * a[k] + m[j][k][1];
    }
}

template <typename T, int KIND, int V, bool BUF>
__global__ __launch_bounds__(64 * kWaves, 2) void diag_bwd_kernel(DiagProblem p, Segments sg, const f32x2* __restrict__ ends,
                                                                   float* __restrict__ part)
{
    constexpr int R = kPer / V;
    __shared__ f32x2 totf[2][kWaves][64];              // F, H
    __shared__ float tota[2][kWaves][64];              // A
    Place q;
    if (!place(p, sg, &q)) return;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    int half;
    const Lane l = lane_of<V, kPer>(p, q, &half);
    const int s0 = q.seg * sg.len, all = min(sg.len, p.T - s0);
    const int n = min(max(clamp_len(p.lengths, (int)q.b, p.T) - s0, 0), all);
    const int cc = min(l.c, l.last);
    const int64_t nc = (p.T + kChunk - 1) / kChunk;
    Walk<T, V, BUF> wx, wu, wv, wg, ox, ou, ov;
    wx.open(p.x, q.b, s0, l);
    wu.open(p.fgate, q.b, s0, l);
    wg.open(p.dy, q.b, s0, l);
    ox.open(p.dx, q.b, s0, l);
    ou.open(p.dfgate, q.b, s0, l);
    if (KIND != kCoupled) {
        wv.open(p.igate, q.b, s0, l);
        ov.open(p.digate, q.b, s0, l);
    }
    float decay[V], a0[V], dd[V];
#pragma unroll
    for (int k = 0; k < V; ++k) {
        decay[k] = KIND == kDecay ? p.decay[cc + k] : 0.0f;
        dd[k] = 0.0f;
    }
    adjoint_behind<V>(p, sg, q, cc, ends, a0);
    typename Walk<T, V, BUF>::raw rx[R], ru[R], rv[R], rg[R];
    float rh[V];
    auto fetch = [&](int t0) {                         // t0 may be < 0: nothing that is used
        const int rows = t0 < 0 ? 0 : min(n - t0, kTile), at = max(t0, 0);
        wu.template load<R>(ru, at, rows, n, l);
        if (KIND != kCoupled) wv.template load<R>(rv, at, rows, n, l);
        wx.template load<R>(rx, at, rows, n, l);
        wg.template load<R>(rg, at, rows, n, l);
#pragma unroll
        for (int k = 0; k < V; ++k) rh[k] = p.starts[(q.b * nc + (s0 + at) / kChunk) * p.D + cc + k];
    };
    ox.clear(n, all, q.cb * 64, p.D);
    ou.clear(n, all, q.cb * 64, p.D);
    if (KIND != kCoupled) ov.clear(n, all, q.cb * 64, p.D);
    const int last = (n - 1) / kTile * kTile;
    if (n > 0) fetch(last);
    int buf = 0;
    for (int t0 = last; n > 0 && t0 >= 0; t0 -= kTile, buf ^= 1) {
        const int rows = min(n - t0, kTile);
        Gate g[R][V];
        float x[R][V], dy[R][V], h[V];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            float u[V], v[V];
            decode<T, V>(ru[r], u);
            if (KIND != kCoupled) decode<T, V>(rv[r], v);
            decode<T, V>(rx[r], x[r]);
            decode<T, V>(rg[r], dy[r]);
#pragma unroll
            for (int k = 0; k < V; ++k) g[r][k] = gate_of<T, KIND>(u[k], KIND != kCoupled ? v[k] : 0.0f, decay[k]);
        }
#pragma unroll
        for (int k = 0; k < V; ++k) h[k] = rh[k];
        fetch(t0 - kTile);
        if (rows < kTile)                              // rows behind the end change nothing
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int k = 0; k < V; ++k)
                    if (l.row + r >= rows) {
                        g[r][k].f = 1.0f;
                        g[r][k].i = x[r][k] = dy[r][k] = 0.0f;
                        if (KIND == kDecay) g[r][k].r = 0.0f;   // nothing for ddecay
                    }
        float fl[V], hl[V], fa[V], aa[V];              // the state before the lane's rows, the adjoint behind them
#pragma unroll
        for (int k = 0; k < V; ++k) {
            float F = 1.0f, H = 0.0f, A = 0.0f;
#pragma unroll
            for (int r = 0; r < R; ++r) {
                H = g[r][k].f * H + g[r][k].i * x[r][k];
                F *= g[r][k].f;
            }
#pragma unroll
            for (int r = R - 1; r >= 0; --r) A = g[r][k].f * (dy[r][k] + A);
            fl[k] = fa[k] = 1.0f;
            hl[k] = aa[k] = 0.0f;
            if (V == 2) {
                float lf, uf, lh, uh, la, ua;
                halves(F, &lf, &uf);
                halves(H, &lh, &uh);
                halves(A, &la, &ua);
                if (half) {
                    fl[k] = lf;
                    hl[k] = lh;
                } else {
                    fa[k] = uf;
                    aa[k] = ua;
                }
                F = lf * uf;
                H = uf * lh + uh;
                A = lf * ua + la;
            }
            if (half == 0) {
                totf[buf][wave][lane * V + k] = f32x2{F, H};
                tota[buf][wave][lane * V + k] = A;
            }
        }
        __syncthreads();
        float a[V];
#pragma unroll
        for (int w = kWaves - 1; w >= 0; --w)
#pragma unroll
            for (int k = 0; k < V; ++k) {
                const int c = lane % (64 / V) * V + k;
                if (w == wave) a[k] = a0[k];
                a0[k] = totf[buf][w][c][0] * a0[k] + tota[buf][w][c];
            }
        for (int w = 0; w < wave; ++w)
#pragma unroll
            for (int k = 0; k < V; ++k) {
                const f32x2 m = totf[buf][w][lane % (64 / V) * V + k];
                h[k] = m[0] * h[k] + m[1];
            }
        float before[R][V];
#pragma unroll
        for (int k = 0; k < V; ++k) {
            if (V == 2) {
                h[k] = fl[k] * h[k] + hl[k];
                a[k] = fa[k] * a[k] + aa[k];
            }
#pragma unroll
            for (int r = 0; r < R; ++r) {
                before[r][k] = h[k];
                h[k] = g[r][k].f * h[k] + g[r][k].i * x[r][k];
            }
        }
#pragma unroll
        for (int r = R - 1; r >= 0; --r) {
            float dx[V], du[V], dv[V];
#pragma unroll
            for (int k = 0; k < V; ++k) {
                const float gr = dy[r][k] + a[k];
                const GateGrads o = grads_of<KIND>(g[r][k], x[r][k], before[r][k], gr, decay[k]);
                a[k] = g[r][k].f * gr;
                dx[k] = o.dx;
                du[k] = o.du;
                dv[k] = o.dv;
                dd[k] += o.dd;
            }
            ox.store(encode<T, V>(dx), r, t0, rows, l);
            ou.store(encode<T, V>(du), r, t0, rows, l);
            if (KIND != kCoupled) ov.store(encode<T, V>(dv), r, t0, rows, l);
        }
    }
    if (p.dstate && q.seg == 0 && wave == 0 && half == 0 && l.live)
#pragma unroll
        for (int k = 0; k < V; ++k) p.dstate[q.b * p.D + l.c + k] = a0[k];
    if (KIND != kDecay) return;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < V; ++k) {
        if (V == 2) {
            float lo, hi;
            halves(dd[k], &lo, &hi);
            dd[k] = lo + hi;
        }
        if (half == 0) tota[0][wave][lane * V + k] = dd[k];
    }
    __syncthreads();
    const int c = q.cb * 64 + lane;
    if (wave != 0 || c >= p.D) return;
    float s = 0.0f;
    for (int w = 0; w < kWaves; ++w) s += tota[0][w][lane];
    part[(q.b * sg.nseg + q.seg) * p.D + c] = s;
}

// The adjoint maps of all segments but the first.
template <typename T, int KIND, int V, bool BUF>
__global__ __launch_bounds__(64 * kWaves, 2) void diag_adjoint_kernel(DiagProblem p, Segments sg, f32x2* __restrict__ ends)
{
    constexpr int R = kPer / V;
    __shared__ f32x2 tot[2][kWaves][64];
    Place q;
    if (!place(p, sg, &q) || q.seg == 0) return;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    int half;
    const Lane l = lane_of<V, kPer>(p, q, &half);
    const int s0 = q.seg * sg.len, all = min(sg.len, p.T - s0);
    const int n = min(max(clamp_len(p.lengths, (int)q.b, p.T) - s0, 0), all);
    const int cc = min(l.c, l.last);
    Walk<T, V, BUF> wu, wg;
    wu.open(p.fgate, q.b, s0, l);
    wg.open(p.dy, q.b, s0, l);
    float decay[V], a0[V], f0[V];
#pragma unroll
    for (int k = 0; k < V; ++k) {
        decay[k] = KIND == kDecay ? p.decay[cc + k] : 0.0f;
        a0[k] = 0.0f;
        f0[k] = 1.0f;
    }
    typename Walk<T, V, BUF>::raw ru[R], rg[R];
    auto fetch = [&](int t0) {
        const int rows = t0 < 0 ? 0 : min(n - t0, kTile), at = max(t0, 0);
        wu.template load<R>(ru, at, rows, n, l);
        wg.template load<R>(rg, at, rows, n, l);
    };
    const int last = (n - 1) / kTile * kTile;
    if (n > 0) fetch(last);
    int buf = 0;
    for (int t0 = last; n > 0 && t0 >= 0; t0 -= kTile, buf ^= 1) {
        const int rows = min(n - t0, kTile);
        float f[R][V], dy[R][V];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            float u[V];
            decode<T, V>(ru[r], u);
            decode<T, V>(rg[r], dy[r]);
#pragma unroll
            for (int k = 0; k < V; ++k) f[r][k] = forget_of<T, KIND>(u[k], decay[k]);
        }
        fetch(t0 - kTile);
        if (rows < kTile)
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int k = 0; k < V; ++k)
                    if (l.row + r >= rows) {
                        f[r][k] = 1.0f;
                        dy[r][k] = 0.0f;
                    }
#pragma unroll
        for (int k = 0; k < V; ++k) {
            float F = 1.0f, A = 0.0f;
#pragma unroll
            for (int r = R - 1; r >= 0; --r) {
                A = f[r][k] * (dy[r][k] + A);
                F *= f[r][k];
            }
            if (V == 2) {
                float lf, uf, la, ua;
                halves(F, &lf, &uf);
                halves(A, &la, &ua);
                F = lf * uf;
                A = lf * ua + la;
            }
            if (half == 0) tot[buf][wave][lane * V + k] = f32x2{F, A};
        }
        __syncthreads();
#pragma unroll
        for (int w = kWaves - 1; w >= 0; --w)
#pragma unroll
            for (int k = 0; k < V; ++k) {
                const f32x2 m = tot[buf][w][lane % (64 / V) * V + k];
                a0[k] = m[0] * a0[k] + m[1];
                f0[k] *= m[0];
            }
    }
    if (wave == 0 && half == 0 && l.live)
#pragma unroll
        for (int k = 0; k < V; ++k) ends[(q.b * sg.nseg + q.seg) * p.D + l.c + k] = f32x2{f0[k], a0[k]};
}

__global__ __launch_bounds__(1024) void diag_params_kernel(DiagProblem p, const float* part, int64_t parts)
{
    __shared__ float red[16][64];
    const int64_t i = (int64_t)blockIdx.x * 64 + threadIdx.x;
    const float s = part_sum(part, parts, p.D, p.D, blockIdx.x, red);
    if (threadIdx.x < 64 && i < p.D) p.ddecay[i] = s;
}

template <typename T, int KIND, int V, bool BUF>
hipError_t bwd_v(const DiagProblem& p, hipStream_t stream)
{
    const Segments sg = segments_of(p, kTile);
    f32x2* ends = (f32x2*)p.ws;
    const int64_t parts = (int64_t)p.B * sg.nseg;
    float* part = parts == 1 ? p.ddecay : (float*)(p.ws + ends_bytes(p, sg));
    const dim3 grid = grid_of(parts * sg.ncb);
    hipError_t e;
    if (sg.nseg > 1) {
        diag_adjoint_kernel<T, KIND, V, BUF><<<grid, 64 * kWaves, 0, stream>>>(p, sg, ends);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    diag_bwd_kernel<T, KIND, V, BUF><<<grid, 64 * kWaves, 0, stream>>>(p, sg, ends, part);
    if ((e = hipGetLastError()) != hipSuccess || KIND != kDecay || parts == 1) return e;
    diag_params_kernel<<<(unsigned)((p.D + 63) / 64), 1024, 0, stream>>>(p, part, parts);
    return hipGetLastError();
}

template <typename T, int KIND>
hipError_t bwd_k(const DiagProblem& p, hipStream_t stream)
{
    bool buf = true, two = p.D % 2 == 0;
    for (const Rows* m : {&p.x, &p.fgate, &p.igate, &p.dy, (const Rows*)&p.dx, (const Rows*)&p.dfgate, (const Rows*)&p.digate}) {
        buf = buf && walks(*m, p, kTile);
        two = two && aligned(*m, p, 2 * sizeof(T));
    }
    if (!buf) return bwd_v<T, KIND, 1, false>(p, stream);
    return two ? bwd_v<T, KIND, 2, true>(p, stream) : bwd_v<T, KIND, 1, true>(p, stream);
}

template <typename T>
hipError_t bwd_t(const DiagProblem& p, hipStream_t stream)
{
    switch (p.kind) {
    case kCoupled: return bwd_k<T, kCoupled>(p, stream);
    case kSigmoid: return bwd_k<T, kSigmoid>(p, stream);
    default: return bwd_k<T, kDecay>(p, stream);
    }
}

}  // namespace

size_t diag_bwd_workspace(const DiagProblem& p)
{
    const Segments sg = segments_of(p, kTile);
    const int64_t parts = (int64_t)p.B * sg.nseg;
    return ends_bytes(p, sg) + (p.kind == kDecay && parts > 1 ? (size_t)parts * p.D * sizeof(float) : 0);
}

hipError_t launch_diag_bwd(const DiagProblem& p, hipStream_t stream)
{
    DiagProblem q = p;
    if (p.T == 1)                                      // the stride of a single row says nothing
        for (Rows* m : {&q.x, &q.fgate, &q.igate, &q.dy, &q.dx, &q.dfgate, &q.digate}) m->row = p.D;
    return p.bf16 ? bwd_t<bf16>(q, stream) : bwd_t<float>(q, stream);
}

}  // namespace tfla
