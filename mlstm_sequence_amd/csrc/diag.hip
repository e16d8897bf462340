// diag.hip -- gated linear recurrence of channels, forward (diag_impl.hpp).
//
// Rows of a tile are affine maps of the state, h -> F h + H, and maps compose:
// a lane forms the map of its rows, the halves of a wave and the eight waves
// join theirs (lane swaps, LDS, one barrier a tile), and each lane then runs
// its rows again from the state before them, kept in registers all along.
// The next tile's loads are under way meanwhile.  Each input is read once and
// y written once: bound by memory.
//
// A long axis over few channels is cut into segments: their maps first (one
// more reading of the inputs), then each from the state that the maps before
// it give.
#include "diag_impl.hpp"

#include <algorithm>

namespace tfla {
namespace {

using namespace diag;

constexpr int kGroup = 4;   // rows whose gates a lane forms together
constexpr int kAhead = 2;   // tiles under way (even: two LDS buffers in turn)

// OUT: outputs; else the segment's map.
template <typename T, int KIND, int CH, int V, bool BUF, bool OUT>
__global__ __launch_bounds__(64 * kWaves, 2) void diag_fwd_kernel(DiagProblem p, Cut sg, f32x2* __restrict__ ends)
{
    typedef Shape<CH, V> S;
    constexpr int R = S::R, kTile = S::tile, LA = CH == 64 ? kStreamed : 0, SA = 0;
    __shared__ f32x2 tot[2][kWaves][CH];
    Place q;
    if (!place(p, sg, &q) || (!OUT && q.seg == sg.nseg - 1)) return;   // no segment starts from the last one's map
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const Lane l = lane_of<CH, V>(p, q);
    const bool first = lane < S::lanes;                // of the lanes that share channels
    const int col = lane % S::lanes * V;
    const int s0 = q.seg * sg.len, all = min(sg.len, p.T - s0);
    // rows of this segment; the same for all lanes, which the compiler cannot tell of a loaded value
    const int n = __builtin_amdgcn_readfirstlane(min(max(clamp_len(p.lengths, (int)q.b, p.T) - s0, 0), all));
    const int cc = min(l.c, l.last);
    Walk<T, V, BUF, LA> wx, wu, wv;
    Walk<T, V, BUF, SA> wy;
    wx.open(p.x, q.b, s0, l);
    wu.open(p.fgate, q.b, s0, l);
    if (KIND != kCoupled) wv.open(p.igate, q.b, s0, l);
    if (OUT) wy.open(p.y, q.b, s0, l);
    Rate decay[V];
    float h0[V], f0[V];                                // the state before the tile; !OUT: the map so far
#pragma unroll
    for (int k = 0; k < V; ++k) {
        decay[k] = Rate(KIND == kDecay ? p.decay[cc + k] : 0.0f);
        h0[k] = OUT && p.state ? p.state[q.b * p.D + cc + k] : 0.0f;
        f0[k] = 1.0f;
    }
    if (OUT) {
        constexpr int LINKS = 8;                       // in batches, whose loads are under way together
        const f32x2* e = ends + q.b * sg.nseg * p.D + cc;
        for (int j0 = 0; j0 < q.seg; j0 += LINKS) {
            f32x2 m[LINKS][V];
#pragma unroll
            for (int j = 0; j < LINKS; ++j)
#pragma unroll
                for (int k = 0; k < V; ++k) m[j][k] = e[(int64_t)min(j0 + j, q.seg - 1) * p.D + k];
#pragma unroll
            for (int j = 0; j < LINKS; ++j)
                if (j0 + j < q.seg)
#pragma unroll
                    for (int k = 0; k < V; ++k) h0[k] = m[j][k][0] * h0[k] + m[j][k][1];
        }
    }
    struct Raw {
        typename RawOf<sizeof(T) * V>::type x[R], u[R], v[R];
    };
    Raw raw[kAhead];                                   // the tiles under way
    if (n > 0)
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int t = i * kTile, rows = min(n - t, kTile);
            const auto tu = wu.tile(t, rows, n), tv = wv.tile(t, rows, n), tx = wx.tile(t, rows, n);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                raw[i].u[r] = wu.load(tu, r, l);
                if (KIND != kCoupled) raw[i].v[r] = wv.load(tv, r, l);
                raw[i].x[r] = wx.load(tx, r, l);
            }
        }
    auto tile = [&](int t0, int buf, Raw& raw) {
        const int rows = min(n - t0, kTile), t1 = t0 + kAhead * kTile, rows1 = min(n - t1, kTile);
        const auto tu = wu.tile(t1, rows1, n), tv = wv.tile(t1, rows1, n), tx = wx.tile(t1, rows1, n);
        float f[R][V], b[R][V];
#pragma unroll
        for (int r0 = 0; r0 < R; r0 += kGroup) {
            float u[kGroup][V], v[kGroup][V], x[kGroup][V];
#pragma unroll
            for (int i = 0; i < kGroup; ++i) {         // a later tile's rows into the registers of those taken
                decode<T, V>(raw.u[r0 + i], u[i]);
                raw.u[r0 + i] = wu.load(tu, r0 + i, l);
                if (KIND != kCoupled) {
                    decode<T, V>(raw.v[r0 + i], v[i]);
                    raw.v[r0 + i] = wv.load(tv, r0 + i, l);
                }
                decode<T, V>(raw.x[r0 + i], x[i]);
                raw.x[r0 + i] = wx.load(tx, r0 + i, l);
            }
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int i = 0; i < kGroup; ++i)
#pragma unroll
                for (int k = 0; k < V; ++k) {
                    const Gate g = gate_of<T, KIND>(u[i][k], KIND != kCoupled ? v[i][k] : 0.0f, decay[k]);
                    f[r0 + i][k] = g.f;
                    b[r0 + i][k] = g.i * x[i][k];
                }
        }
        if (rows < kTile) {                            // rows behind the end change nothing
            const int end = (int)hidden((unsigned)rows);   // a branch, not selections in every tile
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int k = 0; k < V; ++k)
                    if (l.row + r >= end) {
                        f[r][k] = 1.0f;
                        b[r][k] = 0.0f;
                    }
        }
        float F[V], H[V], fl[V], hl[V];                // the lane's map, then the wave's; the map before the lane's rows
#pragma unroll
        for (int k = 0; k < V; ++k) {
            F[k] = f[0][k];
            H[k] = b[0][k];
#pragma unroll
            for (int r = 1; r < R; ++r) {
                H[k] = f[r][k] * H[k] + b[r][k];
                F[k] *= f[r][k];
            }
            fl[k] = 1.0f;
            hl[k] = 0.0f;
            join<S::lanes>(lane, &F[k], &H[k], &fl[k], &hl[k]);
        }
        if (first)
#pragma unroll
            for (int k = 0; k < V; ++k) tot[buf][wave][col + k] = f32x2{F[k], H[k]};
        __syncthreads();
        float h[V];
#pragma unroll
        for (int w = 0; w < kWaves; ++w)
#pragma unroll
            for (int k = 0; k < V; ++k) {
                const f32x2 m = tot[buf][w][col + k];
                if (w == wave) h[k] = h0[k];
                h0[k] = m[0] * h0[k] + m[1];
                if (!OUT) f0[k] *= m[0];
            }
        if (!OUT) return;
        if (p.starts && wave * S::rows % kChunk == 0 && first && l.live && t0 + wave * S::rows < all) {
            const int64_t nc = (p.T + kChunk - 1) / kChunk;
#pragma unroll
            for (int k = 0; k < V; ++k)
                p.starts[(q.b * nc + (s0 + t0 + wave * S::rows) / kChunk) * p.D + l.c + k] = h[k];
        }
#pragma unroll
        for (int k = 0; k < V; ++k) h[k] = fl[k] * h[k] + hl[k];
        const auto ty = wy.tile(t0, rows, n);
#pragma unroll
        for (int r = 0; r < R; ++r) {
#pragma unroll
            for (int k = 0; k < V; ++k) h[k] = f[r][k] * h[k] + b[r][k];
            wy.store(ty, encode<T, V>(h), r, l);
        }
    };
    for (int t0 = 0; t0 < n; t0 += kAhead * kTile)
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            if (t0 + i * kTile < n) tile(t0 + i * kTile, i & 1, raw[i]);
    if (!OUT) {
        if (wave == 0 && first && l.live)
#pragma unroll
            for (int k = 0; k < V; ++k) ends[(q.b * sg.nseg + q.seg) * p.D + l.c + k] = f32x2{f0[k], h0[k]};
        return;
    }
    wy.template clear<CH>(n, all, q.cb * CH, p.D);
    if (wave != 0 || !first || !l.live) return;
    if (p.starts) {                                    // of chunks behind the last tile
        const int64_t nc = (p.T + kChunk - 1) / kChunk;
        for (int t = (n + kTile - 1) / kTile * kTile; t < all; t += kChunk)
#pragma unroll
            for (int k = 0; k < V; ++k) p.starts[(q.b * nc + (s0 + t) / kChunk) * p.D + l.c + k] = h0[k];
    }
    if (p.state_out && q.seg == sg.nseg - 1)
#pragma unroll
        for (int k = 0; k < V; ++k) p.state_out[q.b * p.D + l.c + k] = h0[k];
}

// Single tokens and very short calls: a thread to a channel.
template <typename T, int KIND>
__global__ __launch_bounds__(256) void diag_step_kernel(DiagProblem p)
{
    const int nb = (p.D + 255) / 256, c = (int)(block_id() % nb) * 256 + threadIdx.x;
    const int64_t b = block_id() / nb;
    if (b >= p.B || c >= p.D) return;
    const int len = clamp_len(p.lengths, (int)b, p.T);
    const T* x = (const T*)p.x.p + b * p.x.batch + c;
    const T* u = (const T*)p.fgate.p + b * p.fgate.batch + c;
    const T* v = KIND != kCoupled ? (const T*)p.igate.p + b * p.igate.batch + c : nullptr;
    T* y = (T*)p.y.p + b * p.y.batch + c;
    const Rate decay(KIND == kDecay ? p.decay[c] : 0.0f);
    float h = p.state ? p.state[b * p.D + c] : 0.0f;
    if (p.starts) p.starts[b * p.D + c] = h;
    for (int64_t t = 0; t < p.T; ++t) {
        if (t < len) {
            const Gate g = gate_of<T, KIND>(to_float(u[t * p.fgate.row]), v ? to_float(v[t * p.igate.row]) : 0.0f, decay);
            h = g.f * h + g.i * to_float(x[t * p.x.row]);
        }
        y[t * p.y.row] = from_float<T>(t < len ? h : 0.0f);
    }
    if (p.state_out) p.state_out[b * p.D + c] = h;
}

// Calls of up to this many rows go to the step kernel.
constexpr int kStepRows = 4;

template <typename T, int KIND, int CH, int V, bool BUF>
hipError_t fwd_v(const DiagProblem& p, const Cut& cut, hipStream_t stream)
{
    f32x2* ends = (f32x2*)p.ws;
    if constexpr (CH == 64) {
        if (cut.nseg > 1) {
            diag_fwd_kernel<T, KIND, CH, V, BUF, false><<<grid_of(cut.blocks), 64 * kWaves, 0, stream>>>(p, cut, ends);
            const hipError_t e = hipGetLastError();
            if (e != hipSuccess) return e;
        }
    }
    diag_fwd_kernel<T, KIND, CH, V, BUF, true><<<grid_of(cut.blocks), 64 * kWaves, 0, stream>>>(p, cut, ends);
    return hipGetLastError();
}

template <typename T, int KIND, int V>
hipError_t fwd_c(const DiagProblem& p, hipStream_t stream)
{
    const Cut cut = cut_of(p, true, false);
    switch (cut.ch) {
    case 64: return fwd_v<T, KIND, 64, V, true>(p, cut, stream);
    case 32: return fwd_v<T, KIND, 32, V, true>(p, cut, stream);
    default: return fwd_v<T, KIND, 16, V, true>(p, cut, stream);
    }
}

template <typename T, int KIND>
hipError_t fwd_k(const DiagProblem& p, hipStream_t stream)
{
    if (p.T <= kStepRows) {
        diag_step_kernel<T, KIND><<<grid_of((int64_t)p.B * ((p.D + 255) / 256)), 256, 0, stream>>>(p);
        return hipGetLastError();
    }
    bool buf = true, two = sizeof(T) == 2 && p.D % 2 == 0;
    for (const Rows* m : {&p.x, &p.fgate, &p.igate, (const Rows*)&p.y}) {
        buf = buf && walks(*m, p);
        two = two && aligned(*m, p, 2 * sizeof(T));
    }
    if (!buf) return fwd_v<T, KIND, 64, 1, false>(p, cut_of(p, false, false), stream);
    return two ? fwd_c<T, KIND, 2>(p, stream) : fwd_c<T, KIND, 1>(p, stream);
}

template <typename T>
hipError_t fwd_t(const DiagProblem& p, hipStream_t stream)
{
    switch (p.kind) {
    case kCoupled: return fwd_k<T, kCoupled>(p, stream);
    case kSigmoid: return fwd_k<T, kSigmoid>(p, stream);
    default: return fwd_k<T, kDecay>(p, stream);
    }
}

}  // namespace

// For whichever way the call's strides allow.
size_t diag_workspace(const DiagProblem& p)
{
    return p.T <= kStepRows ? 0 : std::max(ends_bytes(p, cut_of(p, true, false)), ends_bytes(p, cut_of(p, false, false)));
}

hipError_t launch_diag_fwd(const DiagProblem& p, hipStream_t stream)
{
    return p.bf16 ? fwd_t<bf16>(p, stream) : fwd_t<float>(p, stream);
}

}  // namespace tfla
