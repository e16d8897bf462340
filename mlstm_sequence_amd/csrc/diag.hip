// diag.hip -- gated linear recurrence of channels, forward (diag_impl.hpp).
//
// Rows of a tile are affine maps of the state, h -> F h + H, and maps compose:
// a lane forms the map of its rows, the row groups of a wave and the eight
// waves join theirs (lane swaps, LDS, one barrier a tile), and each lane then
// runs its rows again from the state before them, the gates kept in registers
// all along.  Two tiles' loads are under way meanwhile, a row's issued as the
// row before it in the same register is taken.  Each input is read once and y
// written once: bound by memory.  B=4 T=4096 D=4096 bf16, coupled gates 403 MB
// in 80 us, two gates or a decay 537 MB in 109 and 111 (5.0 to 4.8 TB/s, where
// a copy moves 5.0; 4.2 with loads through the caches); fp32 139, 194, 196.
//
// A long axis over few channels is cut into segments: their maps first (one
// more reading of the inputs), then each from the state that the maps before
// it give.  B=1 T=8192 D=4096 bf16: 74, 92 and 99 us.
#include "diag_impl.hpp"

#include <algorithm>

namespace tfla {
namespace {

using namespace diag;

constexpr int kAhead = 2;   // tiles under way (even: two LDS buffers in turn)

// OUT: outputs; else the segment's map.  No segment starts from the last one's map: in its place the first pass leaves
// the state before the first row, since the second may update that in place (one workgroup writes it at its end, which
// may be before another begins).  The first reading of a segmented walk goes through the caches, for the second
// (B=1 T=30000 D=1024 bf16, coupled: 63 us and 68 past them).
template <typename T, int KIND, int CH, bool BUF, bool NT, bool OUT>
__global__ __launch_bounds__(64 * kWaves, 2) void diag_fwd_kernel(DiagProblem p, Cut cut, f32x2* __restrict__ ends)
{
    typedef Shape<CH> S;
    typedef Walk<T, BUF, NT && OUT ? kStreamed : 0> In;
    constexpr int kTile = S::tile;
    __shared__ f32x2 tot[2][kWaves][CH];
    Place q;
    if (!place(p, cut, &q)) return;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const Lane l = lane_of<CH>(p, q);
    const int col = lane % CH, cc = min(l.c, p.D - 1);
    const bool first = lane < CH;                      // of the lanes that share a channel
    const int s0 = q.seg * cut.len, all = min(cut.len, p.T - s0);
    // rows of this segment; the same for all lanes, which the compiler cannot tell of a loaded value
    const int n = __builtin_amdgcn_readfirstlane(min(max(clamp_len(p.lengths, (int)q.b, p.T) - s0, 0), all));
    const int64_t nc = (p.T + kChunk - 1) / kChunk;
    f32x2* e = ends + q.b * cut.nseg * p.D + cc;       // of the lane's channel, a segment p.D apart
    if (!OUT && q.seg == cut.nseg - 1) {
        if (wave == 0 && first && l.live) e[(int64_t)q.seg * p.D] = f32x2{1.0f, p.state ? p.state[q.b * p.D + cc] : 0.0f};
        return;
    }
    In wx, wu, wv;
    Walk<T, BUF, 0> wy;
    wx.open(p.x, q.b, s0, l, p.D);
    wu.open(p.fgate, q.b, s0, l, p.D);
    if (KIND != kCoupled) wv.open(p.igate, q.b, s0, l, p.D);
    if (OUT) wy.open(p.y, q.b, s0, l, p.D);
    const Rate decay(KIND == kDecay ? p.decay[cc] : 0.0f);
    float h0 = 0.0f, f0 = 1.0f;                        // the state before the tile; !OUT: the map so far
    if (OUT) {
        constexpr int LINKS = 8;                       // in batches, whose loads are under way together
        if (cut.nseg > 1) h0 = e[(int64_t)(cut.nseg - 1) * p.D][1];
        else if (p.state) h0 = p.state[q.b * p.D + cc];
        for (int j0 = 0; j0 < q.seg; j0 += LINKS) {
            f32x2 m[LINKS];
#pragma unroll
            for (int j = 0; j < LINKS; ++j) m[j] = e[(int64_t)min(j0 + j, q.seg - 1) * p.D];
#pragma unroll
            for (int j = 0; j < LINKS; ++j)
                if (j0 + j < q.seg) h0 = m[j][0] * h0 + m[j][1];
        }
    }
    struct Raw {
        T x[kRows], u[kRows], v[kRows];
    };
    Raw raw[kAhead];                                   // the tiles under way, as they were loaded
    if (n > 0)
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int t = i * kTile, rows = min(n - t, kTile);
            const auto tu = wu.tile(t, rows, n), tv = wv.tile(t, rows, n), tx = wx.tile(t, rows, n);
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                raw[i].u[r] = wu.load(tu, r, l);
                if (KIND != kCoupled) raw[i].v[r] = wv.load(tv, r, l);
                raw[i].x[r] = wx.load(tx, r, l);
            }
        }
    auto tile = [&](int t0, int buf, Raw& raw) {
        const int rows = min(n - t0, kTile), t1 = t0 + kAhead * kTile, rows1 = min(n - t1, kTile);
        const auto tu = wu.tile(t1, rows1, n), tv = wv.tile(t1, rows1, n), tx = wx.tile(t1, rows1, n);
        float f[kRows], b[kRows];
#pragma unroll
        for (int r0 = 0; r0 < kRows; r0 += kGroup) {
            float u[kGroup], v[kGroup], x[kGroup];
#pragma unroll
            for (int i = 0; i < kGroup; ++i) {         // a later tile's rows into the registers of those taken
                const int r = r0 + i;
                u[i] = to_float(raw.u[r]);
                raw.u[r] = wu.load(tu, r, l);
                if (KIND != kCoupled) {
                    v[i] = to_float(raw.v[r]);
                    raw.v[r] = wv.load(tv, r, l);
                }
                x[i] = to_float(raw.x[r]);
                raw.x[r] = wx.load(tx, r, l);
            }
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int i = 0; i < kGroup; ++i) {
                const Gate g = gate_of<T, KIND>(u[i], KIND != kCoupled ? v[i] : 0.0f, decay);
                f[r0 + i] = g.f;
                b[r0 + i] = g.i * x[i];
            }
        }
        if (rows < kTile) {                            // rows behind the end change nothing
            const int end = (int)hidden((unsigned)rows);   // a branch, not selections in every tile
#pragma unroll
            for (int r = 0; r < kRows; ++r)
                if (l.row + r >= end) {
                    f[r] = 1.0f;
                    b[r] = 0.0f;
                }
        }
        float F = f[0], H = b[0], pf = 1.0f, ph = 0.0f;   // the lane's map, then the wave's; the map before the lane's rows
#pragma unroll
        for (int r = 1; r < kRows; ++r) {
            H = f[r] * H + b[r];
            F *= f[r];
        }
        join<CH>(lane, &F, &H, &pf, &ph);
        if (first) tot[buf][wave][col] = f32x2{F, H};
        __syncthreads();
        float h;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            const f32x2 m = tot[buf][w][col];
            if (w == wave) h = h0;
            h0 = m[0] * h0 + m[1];
            if (!OUT) f0 *= m[0];
        }
        if (!OUT) return;
        const int tw = t0 + wave * S::rows;            // the wave's first row
        if (p.starts && wave * S::rows % kChunk == 0 && first && l.live && tw < all)
            p.starts[(q.b * nc + (s0 + tw) / kChunk) * p.D + l.c] = h;
        h = pf * h + ph;
        const auto ty = wy.tile(t0, rows, n);
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            h = f[r] * h + b[r];
            wy.store(ty, h, r, l);
        }
    };
    for (int t0 = 0; t0 < n; t0 += kAhead * kTile)
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            if (t0 + i * kTile < n) tile(t0 + i * kTile, i & 1, raw[i]);
    if (!OUT) {
        if (wave == 0 && first && l.live) e[(int64_t)q.seg * p.D] = f32x2{f0, h0};
        return;
    }
    wy.template clear<CH>(n, all, q.cb * CH, p.D);
    if (wave != 0 || !first || !l.live) return;
    if (p.starts)                                      // of chunks behind the last tile
        for (int t = (n + kTile - 1) / kTile * kTile; t < all; t += kChunk)
            p.starts[(q.b * nc + (s0 + t) / kChunk) * p.D + l.c] = h0;
    if (p.state_out && q.seg == cut.nseg - 1) p.state_out[q.b * p.D + l.c] = h0;
}

// Single tokens and short axes: a thread to a channel, N rows' loads under way together.  No row is computed twice and
// no tile is part empty, but it takes many channels to fill the chip.  B=64 T=1 D=4096: 3.3 us, the least that a launch
// takes; N rows of four and eight are equal to 10 %, one row at a time is not (B=8 T=32 D=4096 bf16, coupled: 8.8 us,
// eight 6.7).
template <typename T, int KIND, int N>
__global__ __launch_bounds__(256) void diag_short_kernel(DiagProblem p)
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
    float* starts = p.starts ? p.starts + b * ((p.T + kChunk - 1) / kChunk) * p.D + c : nullptr;
    static_assert(kChunk % N == 0, "chunks start where batches do");
    for (int t0 = 0; t0 < p.T; t0 += N) {
        if (starts && t0 % kChunk == 0) starts[(int64_t)(t0 / kChunk) * p.D] = h;
        T rx[N], ru[N], rv[N];
#pragma unroll
        for (int i = 0; i < N; ++i) {                  // behind the last row: the last
            const int64_t t = min(t0 + i, p.T - 1);
            ru[i] = u[t * p.fgate.row];
            if (KIND != kCoupled) rv[i] = v[t * p.igate.row];
            rx[i] = x[t * p.x.row];
        }
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int t = t0 + i;
            if (t >= p.T) break;
            if (t < len) {
                const Gate g = gate_of<T, KIND>(to_float(ru[i]), KIND != kCoupled ? to_float(rv[i]) : 0.0f, decay);
                h = g.f * h + g.i * to_float(rx[i]);
            }
            y[(int64_t)t * p.y.row] = from_float<T>(t < len ? h : 0.0f);
        }
    }
    if (p.state_out) p.state_out[b * p.D + c] = h;
}

// Whether a call goes to the kernel above: up to 16 rows (B=1 T=16 D=1024 bf16, coupled: 4.4 us, tiles 5.5; T=32 6.4 and
// 5.5), and where b blocks of 64 channels are 16 for each row (B=16 T=64 D=4096 bf16, coupled and with a decay: 14.3 and
// 17.7 us, tiles 14.5 and 26.3; B=8 T=64 11 and 17, tiles 8 and 14) as long as tiles, whose arithmetic counts, do not
// catch up: bf16 with coupled gates 256 rows (B=128 D=4096 T=256: 158 us, tiles 173; T=512 322 and 330), else 512 (T=512
// with a decay 433 and 515; T=1024 873 and 923, but B=64 438 and 466, B=32 317 and 237), fp32 64 (T=64 88 and 103; T=128
// 172 and 143) and 256 (T=192 with a decay 328 and 414; T=512 901 and 856).
bool is_short(const DiagProblem& p)
{
    const int64_t most = p.bf16 ? (p.kind == kCoupled ? 256 : 512) : (p.kind == kCoupled ? 64 : 256);
    return p.T <= std::max<int64_t>(16, std::min(most, blocks_of(p, 64) / 16));
}

template <typename T, int KIND, int CH, bool BUF, bool NT>
hipError_t fwd_c(const DiagProblem& p, const Cut& cut, hipStream_t stream)
{
    f32x2* ends = (f32x2*)p.ws;
    if constexpr (CH == 64) {
        if (cut.nseg > 1) {
            diag_fwd_kernel<T, KIND, CH, BUF, NT, false><<<grid_of(cut.blocks), 64 * kWaves, 0, stream>>>(p, cut, ends);
            const hipError_t e = hipGetLastError();
            if (e != hipSuccess) return e;
        }
    }
    diag_fwd_kernel<T, KIND, CH, BUF, NT, true><<<grid_of(cut.blocks), 64 * kWaves, 0, stream>>>(p, cut, ends);
    return hipGetLastError();
}

template <typename T, int KIND>
hipError_t fwd_k(const DiagProblem& p, hipStream_t stream)
{
    if (is_short(p)) {
        const dim3 grid = grid_of((int64_t)p.B * ((p.D + 255) / 256));
        if (p.T == 1) diag_short_kernel<T, KIND, 1><<<grid, 256, 0, stream>>>(p);
        else diag_short_kernel<T, KIND, 8><<<grid, 256, 0, stream>>>(p);
        return hipGetLastError();
    }
    bool buf = true, lines = true;
    for (const Rows* m : {&p.x, &p.fgate, &p.igate, &p.y}) {
        buf = buf && walks(*m, p);
        lines = lines && on_lines(*m, p);
    }
    const Cut cut = cut_of(p, buf, false, lines);
    if (!buf) return fwd_c<T, KIND, 64, false, false>(p, cut, stream);
    switch (cut.ch) {
    case 64: return lines ? fwd_c<T, KIND, 64, true, true>(p, cut, stream) : fwd_c<T, KIND, 64, true, false>(p, cut, stream);
    case 32: return fwd_c<T, KIND, 32, true, false>(p, cut, stream);
    default: return fwd_c<T, KIND, 16, true, false>(p, cut, stream);
    }
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
    return is_short(p) ? 0 : std::max(ends_bytes(p, cut_of(p, true, false)), ends_bytes(p, cut_of(p, false, false)));
}

hipError_t launch_diag_fwd(const DiagProblem& p, hipStream_t stream)
{
    return p.bf16 ? fwd_t<bf16>(p, stream) : fwd_t<float>(p, stream);
}

}  // namespace tfla
