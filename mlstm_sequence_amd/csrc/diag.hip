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

namespace tfla {
namespace {

using namespace diag;

constexpr int kPer = 32, kTile = kWaves * kPer;   // rows of a wave, of a tile

// OUT: outputs; else the segment's map.
template <typename T, int KIND, int V, bool BUF, bool OUT>
__global__ __launch_bounds__(64 * kWaves, 2) void diag_fwd_kernel(DiagProblem p, Segments sg, f32x2* __restrict__ ends)
{
    constexpr int R = kPer / V;
    __shared__ f32x2 tot[2][kWaves][64];
    Place q;
    if (!place(p, sg, &q) || (!OUT && q.seg == sg.nseg - 1)) return;   // no segment starts from the last one's map
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    int half;
    const Lane l = lane_of<V, kPer>(p, q, &half);
    const int s0 = q.seg * sg.len, all = min(sg.len, p.T - s0);
    const int n = min(max(clamp_len(p.lengths, (int)q.b, p.T) - s0, 0), all);   // rows of this segment
    const int cc = min(l.c, l.last);
    Walk<T, V, BUF> wx, wu, wv, wy;
    wx.open(p.x, q.b, s0, l);
    wu.open(p.fgate, q.b, s0, l);
    if (KIND != kCoupled) wv.open(p.igate, q.b, s0, l);
    if (OUT) wy.open(p.y, q.b, s0, l);
    float decay[V], h0[V], f0[V];                      // the state before the tile; !OUT: the map so far
#pragma unroll
    for (int k = 0; k < V; ++k) {
        decay[k] = KIND == kDecay ? p.decay[cc + k] : 0.0f;
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
    typename Walk<T, V, BUF>::raw rx[R], ru[R], rv[R];
    auto fetch = [&](int t0) {
        const int rows = min(n - t0, kTile);
        wu.template load<R>(ru, t0, rows, n, l);
        if (KIND != kCoupled) wv.template load<R>(rv, t0, rows, n, l);
        wx.template load<R>(rx, t0, rows, n, l);
    };
    if (n > 0) fetch(0);
    int buf = 0;
    for (int t0 = 0; t0 < n; t0 += kTile, buf ^= 1) {
        const int rows = min(n - t0, kTile);
        float f[R][V], b[R][V];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            float u[V], v[V], x[V];
            decode<T, V>(ru[r], u);
            if (KIND != kCoupled) decode<T, V>(rv[r], v);
            decode<T, V>(rx[r], x);
#pragma unroll
            for (int k = 0; k < V; ++k) {
                const Gate g = gate_of<T, KIND>(u[k], KIND != kCoupled ? v[k] : 0.0f, decay[k]);
                f[r][k] = g.f;
                b[r][k] = g.i * x[k];
            }
        }
        fetch(t0 + kTile);
        if (rows < kTile)                              // rows behind the end change nothing
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int k = 0; k < V; ++k)
                    if (l.row + r >= rows) {
                        f[r][k] = 1.0f;
                        b[r][k] = 0.0f;
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
            if (V == 2) {
                float lf, uf, lh, uh;
                halves(F[k], &lf, &uf);
                halves(H[k], &lh, &uh);
                F[k] = lf * uf;
                H[k] = uf * lh + uh;
                fl[k] = half ? lf : 1.0f;
                hl[k] = half ? lh : 0.0f;
            }
        }
        if (half == 0)
#pragma unroll
            for (int k = 0; k < V; ++k) tot[buf][wave][lane * V + k] = f32x2{F[k], H[k]};
        __syncthreads();
        float h[V];
#pragma unroll
        for (int w = 0; w < kWaves; ++w)
#pragma unroll
            for (int k = 0; k < V; ++k) {
                const f32x2 m = tot[buf][w][lane % (64 / V) * V + k];
                if (w == wave) h[k] = h0[k];
                h0[k] = m[0] * h0[k] + m[1];
                if (!OUT) f0[k] *= m[0];
            }
        if (!OUT) continue;
        if (p.starts && wave * kPer % kChunk == 0 && half == 0 && l.live && t0 + wave * kPer < all) {
            const int64_t nc = (p.T + kChunk - 1) / kChunk;
#pragma unroll
            for (int k = 0; k < V; ++k)
                p.starts[(q.b * nc + (s0 + t0 + wave * kPer) / kChunk) * p.D + l.c + k] = h[k];
        }
#pragma unroll
        for (int k = 0; k < V; ++k)
            if (V == 2) h[k] = fl[k] * h[k] + hl[k];
#pragma unroll
        for (int r = 0; r < R; ++r) {
#pragma unroll
            for (int k = 0; k < V; ++k) h[k] = f[r][k] * h[k] + b[r][k];
            wy.store(encode<T, V>(h), r, t0, rows, l);
        }
    }
    if (!OUT) {
        if (wave == 0 && half == 0 && l.live)
#pragma unroll
            for (int k = 0; k < V; ++k) ends[(q.b * sg.nseg + q.seg) * p.D + l.c + k] = f32x2{f0[k], h0[k]};
        return;
    }
    wy.clear(n, all, q.cb * 64, p.D);
    if (wave != 0 || half != 0 || !l.live) return;
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
    const float decay = KIND == kDecay ? p.decay[c] : 0.0f;
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

template <typename T, int KIND, int V, bool BUF>
hipError_t fwd_v(const DiagProblem& p, hipStream_t stream)
{
    const Segments sg = segments_of(p, kTile);
    f32x2* ends = (f32x2*)p.ws;
    const dim3 grid = grid_of((int64_t)p.B * sg.nseg * sg.ncb);
    if (sg.nseg > 1) {
        diag_fwd_kernel<T, KIND, V, BUF, false><<<grid, 64 * kWaves, 0, stream>>>(p, sg, ends);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    diag_fwd_kernel<T, KIND, V, BUF, true><<<grid, 64 * kWaves, 0, stream>>>(p, sg, ends);
    return hipGetLastError();
}

template <typename T, int KIND>
hipError_t fwd_k(const DiagProblem& p, hipStream_t stream)
{
    if (p.T <= kStepRows) {
        diag_step_kernel<T, KIND><<<grid_of((int64_t)p.B * ((p.D + 255) / 256)), 256, 0, stream>>>(p);
        return hipGetLastError();
    }
    bool buf = true, two = p.D % 2 == 0;
    for (const Rows* m : {&p.x, &p.fgate, &p.igate, (const Rows*)&p.y}) {
        buf = buf && walks(*m, p, kTile);
        two = two && aligned(*m, p, 2 * sizeof(T));
    }
    if (!buf) return fwd_v<T, KIND, 1, false>(p, stream);
    return two ? fwd_v<T, KIND, 2, true>(p, stream) : fwd_v<T, KIND, 1, true>(p, stream);
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

size_t diag_workspace(const DiagProblem& p) { return p.T <= kStepRows ? 0 : ends_bytes(p, segments_of(p, kTile)); }

hipError_t launch_diag_fwd(const DiagProblem& p, hipStream_t stream)
{
    return p.bf16 ? fwd_t<bf16>(p, stream) : fwd_t<float>(p, stream);
}

}  // namespace tfla
