// diag_bwd.hip -- gated linear recurrence of channels, backward (diag_impl.hpp).
//
// The walk of the forward pass from the end: with a_t = f_t g_t, what row t
// hands to row t - 1, a tile's rows are a map of the state, h -> F h + H, and
// one of the adjoint, a -> F a + A, with the same F.  A lane forms both maps of
// its rows, row groups and waves join theirs as in the forward pass, and each
// lane then runs its rows forward from the state before them (the chunk's
// start, which the forward pass left) and backward from the adjoint behind
// them, the gates kept in registers between the two; the next tile's loads are
// under way meanwhile.  Inputs and dy are read once, the gradients written
// once: bound by memory.  B=4 T=4096 D=4096 bf16, coupled gates 671 MB in 128 us,
// two gates or a decay 940 MB in 203 and 208 (5.2 to 4.5 TB/s, where a copy
// moves 5.0); fp32 270, 353, 361.
//
// A long axis over few channels is cut into segments, whose adjoint maps are
// formed first from fgate and dy alone: B=1 T=8192 D=4096 bf16 96, 114, 126 us.
#include "diag_impl.hpp"

#include <algorithm>

#include "sums.hpp"

namespace tfla {
namespace {

using namespace diag;

// The adjoint behind segment `seg`: dstate_out through the maps of the segments from the last on.
__device__ __forceinline__ float adjoint_behind(const DiagProblem& p, const Cut& cut, const Place& q, int cc, const f32x2* ends)
{
    float a = p.dstate_out ? p.dstate_out[q.b * p.D + cc] : 0.0f;
    constexpr int LINKS = 8;                           // in batches, whose loads are under way together
    const f32x2* e = ends + q.b * cut.nseg * p.D + cc;
    for (int j0 = cut.nseg - 1; j0 > q.seg; j0 -= LINKS) {
        f32x2 m[LINKS];
#pragma unroll
        for (int j = 0; j < LINKS; ++j) m[j] = e[(int64_t)max(j0 - j, q.seg + 1) * p.D];
#pragma unroll
        for (int j = 0; j < LINKS; ++j)
            if (j0 - j > q.seg) a = m[j][0] * a + m[j][1];
    }
    return a;
}

// NT: rows on lines, whose loads and stores go past the caches (B=4 T=4096 D=4096 bf16 with a decay, before the blocks
// of today: 219 us, neither so 226), but not the stores of bf16 gradients of coupled gates (133 us, 150 so).
template <typename T, int KIND, int CH, bool BUF, bool NT>
__global__ __launch_bounds__(64 * kWaves, 2) void diag_bwd_kernel(DiagProblem p, Cut cut, const f32x2* __restrict__ ends,
                                                                   float* __restrict__ part)
{
    typedef Shape<CH> S;
    typedef Walk<T, BUF, NT ? kStreamed : 0> In;
    typedef Walk<T, BUF, NT && (KIND != kCoupled || sizeof(T) == 4) ? kStreamed : 0> Out;
    constexpr int kTile = S::tile;
    __shared__ f32x2 totf[2][kWaves][CH];              // F, H
    __shared__ float tota[2][kWaves][CH];              // A
    Place q;
    if (!place(p, cut, &q)) return;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const Lane l = lane_of<CH>(p, q);
    const int col = lane % CH, cc = min(l.c, p.D - 1);
    const bool first = lane < CH;                      // of the lanes that share a channel
    const int s0 = q.seg * cut.len, all = min(cut.len, p.T - s0);
    const int n = __builtin_amdgcn_readfirstlane(min(max(clamp_len(p.lengths, (int)q.b, p.T) - s0, 0), all));
    const int64_t nc = (p.T + kChunk - 1) / kChunk;
    In wx, wu, wv, wg;
    Out ox, ou, ov;
    wx.open(p.x, q.b, s0, l, p.D);
    wu.open(p.fgate, q.b, s0, l, p.D);
    wg.open(p.dy, q.b, s0, l, p.D);
    ox.open(p.dx, q.b, s0, l, p.D);
    ou.open(p.dfgate, q.b, s0, l, p.D);
    if (KIND != kCoupled) {
        wv.open(p.igate, q.b, s0, l, p.D);
        ov.open(p.digate, q.b, s0, l, p.D);
    }
    const Rate decay(KIND == kDecay ? p.decay[cc] : 0.0f);
    float a0 = adjoint_behind(p, cut, q, cc, ends), dd = 0.0f;
    ox.template clear<CH>(n, all, q.cb * CH, p.D);
    ou.template clear<CH>(n, all, q.cb * CH, p.D);
    if (KIND != kCoupled) ov.template clear<CH>(n, all, q.cb * CH, p.D);
    const int last = (n - 1) / kTile * kTile;
    auto start = [&](int t0) { return p.starts[(q.b * nc + (s0 + t0) / kChunk) * p.D + cc]; };   // the state before row t0
    T rx[kRows], ru[kRows], rv[kRows], rg[kRows];      // the tile under way
    float rh = 0.0f;
    if (n > 0) {
        const auto tu = wu.tile(last, n - last, n), tv = wv.tile(last, n - last, n), tx = wx.tile(last, n - last, n),
                   tg = wg.tile(last, n - last, n);
        rh = start(last);
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
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
        Gate g[kRows];
        T ax[kRows], ag[kRows];                        // x and dy as they were loaded
        float h = rh;
        rh = start(t1);
#pragma unroll
        for (int r0 = 0; r0 < kRows; r0 += kGroup) {
            float u[kGroup], v[kGroup];
#pragma unroll
            for (int i = 0; i < kGroup; ++i) {         // the next tile's rows into the registers of those taken
                const int r = r0 + i;
                u[i] = to_float(ru[r]);
                ru[r] = wu.load(tu, r, l);
                if (KIND != kCoupled) {
                    v[i] = to_float(rv[r]);
                    rv[r] = wv.load(tv, r, l);
                }
                ax[r] = rx[r];
                rx[r] = wx.load(tx, r, l);
                ag[r] = rg[r];
                rg[r] = wg.load(tg, r, l);
            }
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int i = 0; i < kGroup; ++i) g[r0 + i] = gate_of<T, KIND>(u[i], KIND != kCoupled ? v[i] : 0.0f, decay);
        }
        if (rows < kTile) {                            // rows behind the end change nothing
            const int end = (int)hidden((unsigned)rows);   // a branch, not selections in every tile
#pragma unroll
            for (int r = 0; r < kRows; ++r)
                if (l.row + r >= end) {
                    g[r].f = 1.0f;
                    g[r].i = 0.0f;
                    ax[r] = ag[r] = from_float<T>(0.0f);
                    if (KIND == kDecay) g[r].r = 0.0f;     // nothing for ddecay
                }
        }
        float x[kRows], dy[kRows];
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            x[r] = to_float(ax[r]);
            dy[r] = to_float(ag[r]);
        }
        float F = 1.0f, H = 0.0f, A = 0.0f;
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            H = g[r].f * H + g[r].i * x[r];
            F *= g[r].f;
        }
#pragma unroll
        for (int r = kRows - 1; r >= 0; --r) A = g[r].f * (dy[r] + A);
        float pf = 1.0f, ph = 0.0f, qf = 1.0f, qa = 0.0f;   // the map before the lane's rows, the adjoint's behind them
        join_both<CH>(lane, &F, &H, &A, &pf, &ph, &qf, &qa);
        if (first) {
            totf[buf][wave][col] = f32x2{F, H};
            tota[buf][wave][col] = A;
        }
        __syncthreads();
        float a;
#pragma unroll
        for (int w = kWaves - 1; w >= 0; --w) {
            if (w == wave) a = a0;
            a0 = totf[buf][w][col][0] * a0 + tota[buf][w][col];
        }
        for (int w = 0; w < wave; ++w) {
            const f32x2 m = totf[buf][w][col];
            h = m[0] * h + m[1];
        }
        h = pf * h + ph;
        a = qf * a + qa;
        float before[kRows];
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            before[r] = h;
            h = g[r].f * h + g[r].i * x[r];
        }
        const auto tdx = ox.tile(t0, rows, n), tdu = ou.tile(t0, rows, n), tdv = ov.tile(t0, rows, n);
#pragma unroll
        for (int r = kRows - 1; r >= 0; --r) {
            const float gr = dy[r] + a;
            const GateGrads o = grads_of<KIND>(g[r], x[r], before[r], gr, decay);
            a = g[r].f * gr;
            dd += o.dd;
            ox.store(tdx, o.dx, r, l);
            ou.store(tdu, o.du, r, l);
            if (KIND != kCoupled) ov.store(tdv, o.dv, r, l);
        }
    }
    if (p.dstate && q.seg == 0 && wave == 0 && first && l.live) p.dstate[q.b * p.D + l.c] = a0;
    if (KIND != kDecay) return;
    __syncthreads();
    dd = sum_groups<CH>(dd);
    if (first) tota[0][wave][col] = dd;
    __syncthreads();
    const int c = q.cb * CH + (int)threadIdx.x;
    if (threadIdx.x >= CH || c >= p.D) return;
    float s = 0.0f;
    for (int w = 0; w < kWaves; ++w) s += tota[0][w][threadIdx.x];
    part[(q.b * cut.nseg + q.seg) * p.D + c] = s;
}

// The adjoint maps of all segments but the first.
template <typename T, int KIND, bool BUF>
__global__ __launch_bounds__(64 * kWaves, 2) void diag_adjoint_kernel(DiagProblem p, Cut cut, f32x2* __restrict__ ends)
{
    constexpr int CH = 64, kTile = Shape<CH>::tile;
    __shared__ f32x2 tot[2][kWaves][CH];
    Place q;
    if (!place(p, cut, &q) || q.seg == 0) return;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const Lane l = lane_of<CH>(p, q);
    const int s0 = q.seg * cut.len, all = min(cut.len, p.T - s0);
    const int n = __builtin_amdgcn_readfirstlane(min(max(clamp_len(p.lengths, (int)q.b, p.T) - s0, 0), all));
    Walk<T, BUF, 0> wu, wg;
    wu.open(p.fgate, q.b, s0, l, p.D);
    wg.open(p.dy, q.b, s0, l, p.D);
    const Rate decay(KIND == kDecay ? p.decay[min(l.c, p.D - 1)] : 0.0f);
    float a0 = 0.0f, f0 = 1.0f;
    T ru[kRows], rg[kRows];
    const int last = (n - 1) / kTile * kTile;
    if (n > 0) {
        const auto tu = wu.tile(last, n - last, n), tg = wg.tile(last, n - last, n);
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            ru[r] = wu.load(tu, r, l);
            rg[r] = wg.load(tg, r, l);
        }
    }
    int buf = 0;
    for (int t0 = last; n > 0 && t0 >= 0; t0 -= kTile, buf ^= 1) {
        const int rows = min(n - t0, kTile), t1 = max(t0 - kTile, 0), rows1 = t0 ? kTile : 0;
        const auto tu = wu.tile(t1, rows1, n), tg = wg.tile(t1, rows1, n);
        float f[kRows], dy[kRows];
#pragma unroll
        for (int r0 = 0; r0 < kRows; r0 += kGroup) {
            float u[kGroup];
#pragma unroll
            for (int i = 0; i < kGroup; ++i) {
                const int r = r0 + i;
                u[i] = to_float(ru[r]);
                ru[r] = wu.load(tu, r, l);
                dy[r] = to_float(rg[r]);
                rg[r] = wg.load(tg, r, l);
            }
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int i = 0; i < kGroup; ++i) f[r0 + i] = forget_of<T, KIND>(u[i], decay);
        }
        if (rows < kTile) {
            const int end = (int)hidden((unsigned)rows);
#pragma unroll
            for (int r = 0; r < kRows; ++r)
                if (l.row + r >= end) {
                    f[r] = 1.0f;
                    dy[r] = 0.0f;
                }
        }
        float F = 1.0f, A = 0.0f;
#pragma unroll
        for (int r = kRows - 1; r >= 0; --r) {
            A = f[r] * (dy[r] + A);
            F *= f[r];
        }
        tot[buf][wave][lane] = f32x2{F, A};
        __syncthreads();
#pragma unroll
        for (int w = kWaves - 1; w >= 0; --w) {
            const f32x2 m = tot[buf][w][lane];
            a0 = m[0] * a0 + m[1];
            f0 *= m[0];
        }
    }
    if (wave == 0 && l.live) ends[(q.b * cut.nseg + q.seg) * p.D + l.c] = f32x2{f0, a0};
}

__global__ __launch_bounds__(1024) void diag_params_kernel(DiagProblem p, const float* part, int64_t parts)
{
    __shared__ float red[16][64];
    const int64_t i = (int64_t)blockIdx.x * 64 + threadIdx.x;
    const float s = part_sum(part, parts, p.D, p.D, blockIdx.x, red);
    if (threadIdx.x < 64 && i < p.D) p.ddecay[i] = s;
}

template <typename T, int KIND, int CH, bool BUF, bool NT>
hipError_t bwd_c(const DiagProblem& p, const Cut& cut, hipStream_t stream)
{
    f32x2* ends = (f32x2*)p.ws;
    const int64_t parts = (int64_t)p.B * cut.nseg;
    float* part = parts == 1 ? p.ddecay : (float*)(p.ws + ends_bytes(p, cut));
    hipError_t e;
    if constexpr (CH == 64) {
        if (cut.nseg > 1) {
            diag_adjoint_kernel<T, KIND, BUF><<<grid_of(cut.blocks), 64 * kWaves, 0, stream>>>(p, cut, ends);
            if ((e = hipGetLastError()) != hipSuccess) return e;
        }
    }
    diag_bwd_kernel<T, KIND, CH, BUF, NT><<<grid_of(cut.blocks), 64 * kWaves, 0, stream>>>(p, cut, ends, part);
    if ((e = hipGetLastError()) != hipSuccess || KIND != kDecay || parts == 1) return e;
    diag_params_kernel<<<(unsigned)((p.D + 63) / 64), 1024, 0, stream>>>(p, part, parts);
    return hipGetLastError();
}

template <typename T, int KIND>
hipError_t bwd_k(const DiagProblem& p, hipStream_t stream)
{
    bool buf = true, lines = true;
    for (const Rows* m : {&p.x, &p.fgate, &p.igate, &p.dy, &p.dx, &p.dfgate, &p.digate}) {
        buf = buf && walks(*m, p);
        lines = lines && on_lines(*m, p);
    }
    const Cut cut = cut_of(p, buf, true, lines);
    if (!buf) return bwd_c<T, KIND, 64, false, false>(p, cut, stream);
    switch (cut.ch) {
    case 64: return lines ? bwd_c<T, KIND, 64, true, true>(p, cut, stream) : bwd_c<T, KIND, 64, true, false>(p, cut, stream);
    case 32: return bwd_c<T, KIND, 32, true, false>(p, cut, stream);
    default: return bwd_c<T, KIND, 16, true, false>(p, cut, stream);
    }
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
