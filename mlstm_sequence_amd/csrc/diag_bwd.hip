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

#include <algorithm>

#include "sums.hpp"

namespace tfla {
namespace {

using namespace diag;

constexpr int kGroup = 4;   // rows whose gates a lane forms together

// The adjoint behind segment `seg`: dstate_out through the maps of the segments from the last on.
template <int V>
__device__ __forceinline__ void adjoint_behind(const DiagProblem& p, const Cut& sg, const Place& q, int cc,
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

template <typename T, int KIND, int CH, int V, bool BUF>
__global__ __launch_bounds__(64 * kWaves, 2) void diag_bwd_kernel(DiagProblem p, Cut sg, const f32x2* __restrict__ ends,
                                                                   float* __restrict__ part)
{
    typedef Shape<CH, V> S;
    constexpr int R = S::R, kTile = S::tile, LA = CH == 64 ? kStreamed : 0,
                  SA = CH == 64 && (KIND != kCoupled || sizeof(T) == 4) ? kStreamed : 0;
    __shared__ f32x2 totf[2][kWaves][CH];              // F, H
    __shared__ float tota[2][kWaves][CH];              // A
    Place q;
    if (!place(p, sg, &q)) return;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const Lane l = lane_of<CH, V>(p, q);
    const bool first = lane < S::lanes;                // of the lanes that share channels
    const int col = lane % S::lanes * V;
    const int s0 = q.seg * sg.len, all = min(sg.len, p.T - s0);
    const int n = __builtin_amdgcn_readfirstlane(min(max(clamp_len(p.lengths, (int)q.b, p.T) - s0, 0), all));
    const int cc = min(l.c, l.last);
    const int64_t nc = (p.T + kChunk - 1) / kChunk;
    Walk<T, V, BUF, LA> wx, wu, wv, wg;
    Walk<T, V, BUF, SA> ox, ou, ov;
    wx.open(p.x, q.b, s0, l);
    wu.open(p.fgate, q.b, s0, l);
    wg.open(p.dy, q.b, s0, l);
    ox.open(p.dx, q.b, s0, l);
    ou.open(p.dfgate, q.b, s0, l);
    if (KIND != kCoupled) {
        wv.open(p.igate, q.b, s0, l);
        ov.open(p.digate, q.b, s0, l);
    }
    Rate decay[V];
    float a0[V], dd[V];
#pragma unroll
    for (int k = 0; k < V; ++k) {
        decay[k] = Rate(KIND == kDecay ? p.decay[cc + k] : 0.0f);
        dd[k] = 0.0f;
    }
    adjoint_behind<V>(p, sg, q, cc, ends, a0);
    typename RawOf<sizeof(T) * V>::type rx[R], ru[R], rv[R], rg[R];
    float rh[V];
    ox.template clear<CH>(n, all, q.cb * CH, p.D);
    ou.template clear<CH>(n, all, q.cb * CH, p.D);
    if (KIND != kCoupled) ov.template clear<CH>(n, all, q.cb * CH, p.D);
    const int last = (n - 1) / kTile * kTile;
    auto start = [&](int t0) {                         // the state at a tile's start
#pragma unroll
        for (int k = 0; k < V; ++k) rh[k] = p.starts[(q.b * nc + (s0 + max(t0, 0)) / kChunk) * p.D + cc + k];
    };
    if (n > 0) {
        const auto tu = wu.tile(last, n - last, n), tv = wv.tile(last, n - last, n), tx = wx.tile(last, n - last, n),
                   tg = wg.tile(last, n - last, n);
        start(last);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            ru[r] = wu.load(tu, r, l);
            if (KIND != kCoupled) rv[r] = wv.load(tv, r, l);
            rx[r] = wx.load(tx, r, l);
            rg[r] = wg.load(tg, r, l);
        }
    }
    int buf = 0;
    for (int t0 = last; n > 0 && t0 >= 0; t0 -= kTile, buf ^= 1) {
        const int rows = min(n - t0, kTile), t1 = max(t0 - kTile, 0), rows1 = t0 ? kTile : 0;   // the next tile is whole, or none
        const auto tu = wu.tile(t1, rows1, n), tv = wv.tile(t1, rows1, n), tx = wx.tile(t1, rows1, n), tg = wg.tile(t1, rows1, n);
        Gate g[R][V];
        typename RawOf<sizeof(T) * V>::type ax[R], ag[R];    // x and dy as they were loaded
        float h[V];
#pragma unroll
        for (int k = 0; k < V; ++k) h[k] = rh[k];
        start(t1);
#pragma unroll
        for (int r0 = 0; r0 < R; r0 += kGroup) {
            float u[kGroup][V], v[kGroup][V];
#pragma unroll
            for (int i = 0; i < kGroup; ++i) {         // the next tile's rows into the registers of those taken
                const int r = r0 + i;
                decode<T, V>(ru[r], u[i]);
                ru[r] = wu.load(tu, r, l);
                if (KIND != kCoupled) {
                    decode<T, V>(rv[r], v[i]);
                    rv[r] = wv.load(tv, r, l);
                }
                ax[r] = rx[r];
                rx[r] = wx.load(tx, r, l);
                ag[r] = rg[r];
                rg[r] = wg.load(tg, r, l);
            }
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int i = 0; i < kGroup; ++i)
#pragma unroll
                for (int k = 0; k < V; ++k) g[r0 + i][k] = gate_of<T, KIND>(u[i][k], KIND != kCoupled ? v[i][k] : 0.0f, decay[k]);
        }
        if (rows < kTile) {                            // rows behind the end change nothing
            const int end = (int)hidden((unsigned)rows);   // a branch, not selections in every tile
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int k = 0; k < V; ++k)
                    if (l.row + r >= end) {
                        g[r][k].f = 1.0f;
                        g[r][k].i = 0.0f;
                        ax[r] = ag[r] = {};
                        if (KIND == kDecay) g[r][k].r = 0.0f;   // nothing for ddecay
                    }
        }
        float x[R][V], dy[R][V];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            decode<T, V>(ax[r], x[r]);
            decode<T, V>(ag[r], dy[r]);
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
            join_both<S::lanes>(lane, &F, &H, &A, &fl[k], &hl[k], &fa[k], &aa[k]);
            if (first) {
                totf[buf][wave][col + k] = f32x2{F, H};
                tota[buf][wave][col + k] = A;
            }
        }
        __syncthreads();
        float a[V];
#pragma unroll
        for (int w = kWaves - 1; w >= 0; --w)
#pragma unroll
            for (int k = 0; k < V; ++k) {
                if (w == wave) a[k] = a0[k];
                a0[k] = totf[buf][w][col + k][0] * a0[k] + tota[buf][w][col + k];
            }
        for (int w = 0; w < wave; ++w)
#pragma unroll
            for (int k = 0; k < V; ++k) {
                const f32x2 m = totf[buf][w][col + k];
                h[k] = m[0] * h[k] + m[1];
            }
        float before[R][V];
#pragma unroll
        for (int k = 0; k < V; ++k) {
            h[k] = fl[k] * h[k] + hl[k];
            a[k] = fa[k] * a[k] + aa[k];
#pragma unroll
            for (int r = 0; r < R; ++r) {
                before[r][k] = h[k];
                h[k] = g[r][k].f * h[k] + g[r][k].i * x[r][k];
            }
        }
        const auto tdx = ox.tile(t0, rows, n), tdu = ou.tile(t0, rows, n), tdv = ov.tile(t0, rows, n);
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
            ox.store(tdx, encode<T, V>(dx), r, l);
            ou.store(tdu, encode<T, V>(du), r, l);
            if (KIND != kCoupled) ov.store(tdv, encode<T, V>(dv), r, l);
        }
    }
    if (p.dstate && q.seg == 0 && wave == 0 && first && l.live)
#pragma unroll
        for (int k = 0; k < V; ++k) p.dstate[q.b * p.D + l.c + k] = a0[k];
    if (KIND != kDecay) return;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < V; ++k) {
        dd[k] = sum_groups<S::lanes>(lane, dd[k]);
        if (first) tota[0][wave][col + k] = dd[k];
    }
    __syncthreads();
    const int c = q.cb * CH + (int)threadIdx.x;
    if (threadIdx.x >= CH || c >= p.D) return;
    float s = 0.0f;
    for (int w = 0; w < kWaves; ++w) s += tota[0][w][threadIdx.x];
    part[(q.b * sg.nseg + q.seg) * p.D + c] = s;
}

// The adjoint maps of all segments but the first.
template <typename T, int KIND, int CH, int V, bool BUF>
__global__ __launch_bounds__(64 * kWaves, 2) void diag_adjoint_kernel(DiagProblem p, Cut sg, f32x2* __restrict__ ends)
{
    typedef Shape<CH, V> S;
    constexpr int R = S::R, kTile = S::tile;
    __shared__ f32x2 tot[2][kWaves][CH];
    Place q;
    if (!place(p, sg, &q) || q.seg == 0) return;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const Lane l = lane_of<CH, V>(p, q);
    const bool first = lane < S::lanes;                // of the lanes that share channels
    const int col = lane % S::lanes * V;
    const int s0 = q.seg * sg.len, all = min(sg.len, p.T - s0);
    const int n = __builtin_amdgcn_readfirstlane(min(max(clamp_len(p.lengths, (int)q.b, p.T) - s0, 0), all));
    const int cc = min(l.c, l.last);
    Walk<T, V, BUF, 0> wu, wg;
    wu.open(p.fgate, q.b, s0, l);
    wg.open(p.dy, q.b, s0, l);
    Rate decay[V];
    float a0[V], f0[V];
#pragma unroll
    for (int k = 0; k < V; ++k) {
        decay[k] = Rate(KIND == kDecay ? p.decay[cc + k] : 0.0f);
        a0[k] = 0.0f;
        f0[k] = 1.0f;
    }
    typename RawOf<sizeof(T) * V>::type ru[R], rg[R];
    const int last = (n - 1) / kTile * kTile;
    if (n > 0) {
        const auto tu = wu.tile(last, n - last, n), tg = wg.tile(last, n - last, n);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            ru[r] = wu.load(tu, r, l);
            rg[r] = wg.load(tg, r, l);
        }
    }
    int buf = 0;
    for (int t0 = last; n > 0 && t0 >= 0; t0 -= kTile, buf ^= 1) {
        const int rows = min(n - t0, kTile), t1 = max(t0 - kTile, 0), rows1 = t0 ? kTile : 0;
        const auto tu = wu.tile(t1, rows1, n), tg = wg.tile(t1, rows1, n);
        float f[R][V], dy[R][V];
#pragma unroll
        for (int r0 = 0; r0 < R; r0 += kGroup) {
            float u[kGroup][V];
#pragma unroll
            for (int i = 0; i < kGroup; ++i) {
                decode<T, V>(ru[r0 + i], u[i]);
                ru[r0 + i] = wu.load(tu, r0 + i, l);
                decode<T, V>(rg[r0 + i], dy[r0 + i]);
                rg[r0 + i] = wg.load(tg, r0 + i, l);
            }
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int i = 0; i < kGroup; ++i)
#pragma unroll
                for (int k = 0; k < V; ++k) f[r0 + i][k] = forget_of<T, KIND>(u[i][k], decay[k]);
        }
        if (rows < kTile) {
            const int end = (int)hidden((unsigned)rows);
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int k = 0; k < V; ++k)
                    if (l.row + r >= end) {
                        f[r][k] = 1.0f;
                        dy[r][k] = 0.0f;
                    }
        }
#pragma unroll
        for (int k = 0; k < V; ++k) {
            float F = 1.0f, A = 0.0f;
#pragma unroll
            for (int r = R - 1; r >= 0; --r) {
                A = f[r][k] * (dy[r][k] + A);
                F *= f[r][k];
            }
            join_behind<S::lanes>(lane, &F, &A);
            if (first) tot[buf][wave][col + k] = f32x2{F, A};
        }
        __syncthreads();
#pragma unroll
        for (int w = kWaves - 1; w >= 0; --w)
#pragma unroll
            for (int k = 0; k < V; ++k) {
                const f32x2 m = tot[buf][w][col + k];
                a0[k] = m[0] * a0[k] + m[1];
                f0[k] *= m[0];
            }
    }
    if (wave == 0 && first && l.live)
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

template <typename T, int KIND, int CH, int V, bool BUF>
hipError_t bwd_v(const DiagProblem& p, const Cut& cut, hipStream_t stream)
{
    f32x2* ends = (f32x2*)p.ws;
    const int64_t parts = (int64_t)p.B * cut.nseg;
    float* part = parts == 1 ? p.ddecay : (float*)(p.ws + ends_bytes(p, cut));
    hipError_t e;
    if constexpr (CH == 64) {
        if (cut.nseg > 1) {
            diag_adjoint_kernel<T, KIND, CH, V, BUF><<<grid_of(cut.blocks), 64 * kWaves, 0, stream>>>(p, cut, ends);
            if ((e = hipGetLastError()) != hipSuccess) return e;
        }
    }
    diag_bwd_kernel<T, KIND, CH, V, BUF><<<grid_of(cut.blocks), 64 * kWaves, 0, stream>>>(p, cut, ends, part);
    if ((e = hipGetLastError()) != hipSuccess || KIND != kDecay || parts == 1) return e;
    diag_params_kernel<<<(unsigned)((p.D + 63) / 64), 1024, 0, stream>>>(p, part, parts);
    return hipGetLastError();
}

template <typename T, int KIND, int V>
hipError_t bwd_c(const DiagProblem& p, hipStream_t stream)
{
    const Cut cut = cut_of(p, true, true);
    switch (cut.ch) {
    case 64: return bwd_v<T, KIND, 64, V, true>(p, cut, stream);
    case 32: return bwd_v<T, KIND, 32, V, true>(p, cut, stream);
    default: return bwd_v<T, KIND, 16, V, true>(p, cut, stream);
    }
}

template <typename T, int KIND>
hipError_t bwd_k(const DiagProblem& p, hipStream_t stream)
{
    bool buf = true, two = sizeof(T) == 2 && p.D % 2 == 0;
    for (const Rows* m : {&p.x, &p.fgate, &p.igate, &p.dy, (const Rows*)&p.dx, (const Rows*)&p.dfgate, (const Rows*)&p.digate}) {
        buf = buf && walks(*m, p);
        two = two && aligned(*m, p, 2 * sizeof(T));
    }
    if (!buf) return bwd_v<T, KIND, 64, 1, false>(p, cut_of(p, false, true), stream);
    return two ? bwd_c<T, KIND, 2>(p, stream) : bwd_c<T, KIND, 1>(p, stream);
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

// For whichever way the call's strides allow.
size_t diag_bwd_workspace(const DiagProblem& p)
{
    size_t most = 0;
    for (const bool buf : {true, false}) {
        const Cut cut = cut_of(p, buf, true);
        const int64_t parts = (int64_t)p.B * cut.nseg;
        most = std::max(most, ends_bytes(p, cut) + (p.kind == kDecay && parts > 1 ? (size_t)parts * p.D * sizeof(float) : 0));
    }
    return most;
}

hipError_t launch_diag_bwd(const DiagProblem& p, hipStream_t stream)
{
    DiagProblem q = p;
    if (p.T == 1)                                      // the stride of a single row says nothing
        for (Rows* m : {&q.x, &q.fgate, &q.igate, &q.dy, &q.dx, &q.dfgate, &q.digate}) m->row = p.D;
    return p.bf16 ? bwd_t<bf16>(q, stream) : bwd_t<float>(q, stream);
}

}  // namespace tfla
