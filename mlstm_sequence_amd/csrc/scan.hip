// scan.hip -- forward pass of the selective scan (scan_impl.hpp).
//
// A workgroup walks its segment in tiles: while one is walked, the next
// tile's inputs load into registers and are published into the other of two
// LDS buffers, (delta, delta x) for each channel and B and C as fp32 for the
// whole group; after a barrier the tile's outputs are finished (the sum over
// the waves' shares of C h, the skip, the gate).  All lanes of a wave read the
// same four values of B and C, so these reads cost LDS 16 of about 136 cycles
// a wave and step.  Read by scalar loads instead they cost none, but the
// scalar cache misses on every row and a wait for one such load is a wait for
// all: with one wave on a SIMD a step took 512 cycles.
// The arithmetic bounds it: 6 issue slots a state and step (four products and
// an exponential of two), 24 of about 35 that a wave of four states spends on
// a step; the rest is softplus, gate and conversions.  B=1 T=8192 D=4096 N=16
// bf16 with a gate, in segments: 216 to 238 us (the walk for the end states
// 103, the walk for the outputs 143, profiled apart, each with 93 % of the
// issue slots taken); B=8 T=2048, one walk: 315 us.
//
// A long axis over few sequences and channels is cut into segments: every
// segment is first walked from a zero state for its end state (no outputs),
// the start states follow from those (a decay over a segment is
// exp(A sum delta)), and the second walk starts from them.  The last segment's
// end state is formed like the others' and not used.
#include "scan_impl.hpp"

namespace tfla {
namespace {

using namespace scan;

// Steps of a tile.  One or two waves prepare 8 or 16 steps each in a tile of 16 and run out of registers
// (B=4 T=1024 D=2048, N=8: 67 us with 16, 52 with 8); four or more gain from fewer barriers (N=16, B=8 T=2048
// D=4096: 315 against 337 us).
constexpr int tile_steps(int W) { return W > 2 ? 16 : 8; }
constexpr int U = 1;     // steps fetched from LDS together (2 cost registers and 4 % at N=16)
constexpr int kVm0 = 0x0f70;   // s_waitcnt: no vector load outstanding
constexpr int AHEAD = 2; // tiles whose inputs are under way (even: two LDS buffers in turn)

struct SegWs {
    float* ends;   // [B][nseg][D][N]
    float* sums;   // [B][nseg][D]
};

// OUT: the outputs; else the end state and the sum of the steps.  GATED: y times z sigmoid(z).
// Four waves to a SIMD are asked for (16 waves fill it as they are): left alone, the gated kernel takes 166
// registers and three fit.  With N up to 4, where a wave prepares a whole tile, it keeps 3 to 5 values in scratch
// for that, and three waves without them would be faster (B=1 T=8192 D=4096 N=4: 143 us against 152; B=4 T=1024
// D=2048: 50.5 and 52).
template <typename T, int W, bool OUT, bool GATED>
__global__ __launch_bounds__(64 * W, W == 16 ? 1 : 4) void scan_fwd_kernel(ScanProblem p, Segments sg, SegWs ws)
{
    constexpr int TS = tile_steps(W), OWN = TS / W;                       // steps of a tile that a wave prepares and finishes
    constexpr int NP = W * kStates, BC = OUT ? 2 : 1;  // states with padding; B alone, or B and C
    constexpr int PER = (TS * BC * NP + 64 * W - 1) / (64 * W);
    __shared__ f32x2 du[2][TS][64];                   // delta, delta x
    __shared__ f32x4 bc[2][TS][BC][W];                // B, C
    __shared__ float part[OUT ? W : 1][OUT ? TS : 1][64];
    const Place q = place(p, sg);
    const int all = clamp_len(p.lengths, q.b, p.T);
    const int s0 = q.seg * sg.len, s1 = min(s0 + sg.len, p.T);
    const int len = max(0, min(all, s1) - s0);        // steps of this segment
    const int n0 = q.wave * kStates;
    const int ns = min(kStates, p.N - n0);            // the wave's states (<= 0: it only shares the steps' work)
    const T* xp = (const T*)p.x.p + q.b * p.x.batch + s0 * p.x.row;
    const T* dp = (const T*)p.dt.p + q.b * p.dt.batch + s0 * p.dt.row;
    const T* zp = GATED ? (const T*)p.z.p + q.b * p.z.batch + s0 * p.z.row : nullptr;
    T* yp = OUT ? (T*)p.y.p + q.b * p.y.batch + s0 * p.y.row : nullptr;
    const unsigned c = q.c;
    const int own = q.wave * OWN;                     // the wave's steps of a tile: own .. own + OWN - 1
    // this thread's elements of the tile's B and C: element e of the tile is step, matrix, state in that order
    MatCursor<T> mat[PER];
    bool mv[PER];                                     // padding is 0
#pragma unroll
    for (int k = 0; k < PER; ++k) {
        const int e = threadIdx.x + k * 64 * W, n = e % NP, isc = e / NP % BC;
        mv[k] = n < p.N;
        mat[k].set(isc ? p.cmat : p.bmat, q.b, s0, q.g * p.N + min(n, p.N - 1), min(e / NP / BC, TS - 1), 0, TS, len);
    }
    const int softplus = __builtin_amdgcn_readfirstlane(p.softplus);
    const float skip = OUT && p.skip ? p.skip[q.c] : 0.0f;
    const float bias = p.dt_bias ? p.dt_bias[q.c] : 0.0f;
    const size_t srow = ((size_t)q.b * p.D + q.c) * p.N + n0;
    const size_t erow = (((size_t)q.b * sg.nseg + q.seg) * p.D + q.c) * p.N + n0;

    // the start: the folded one of a segmented walk's second pass, else the caller's; 0 in its first pass
    float A[kStates], h[kStates];
    {
        const float* st = !OUT ? nullptr : sg.nseg > 1 ? ws.ends + erow : p.state ? p.state + srow : nullptr;
        const f32x4 av = load_states(p.a + (size_t)q.c * p.N + n0, ns);
        const f32x4 hv = st ? load_states(st, ns) : f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int n = 0; n < kStates; ++n) {
            A[n] = av[n] * kLog2e;
            h[n] = hv[n];
        }
    }
    float dsum = 0.0f;                                // this wave's steps

    // The inputs of the next AHEAD tiles, as they were loaded: a conversion beside the load would wait for it
    // there.  A tile's walk is shorter than a trip to memory, so with few waves on a SIMD one tile ahead is late.
    struct Raw {
        T x[OWN], dt[OWN], z[OWN], m[PER];
    };
    Raw raw[AHEAD];
    T fx[OWN], fz[OWN];                     // what the current tile's finish needs
    // No branch stands around a load (rows behind the end are read as the last one, and never used): where
    // paths with and without the load meet, its register would be copied, which waits for it.
    auto fetch = [&](Raw& r, int t0) {
#pragma unroll
        for (int i = 0; i < OWN; ++i) {
            const int64_t t = min(t0 + own + i, len - 1);
            r.x[i] = (xp + t * p.x.row)[c];
            r.dt[i] = (dp + t * p.dt.row)[c];
            if (GATED) r.z[i] = (zp + t * p.z.row)[c];
        }
#pragma unroll
        for (int k = 0; k < PER; ++k) r.m[k] = mat[k].next(t0, len);
    };
    auto publish = [&](const Raw& r, int t0, int buf) {
#pragma unroll
        for (int i = 0; i < OWN; ++i) {
            const float u = to_float(r.dt[i]) + bias;
            const float d = softplus ? softplus_t<T>(u) : u;
            du[buf][own + i][q.lane] = f32x2{d, d * to_float(r.x[i])};   // behind the end: never read
            if (!OUT && t0 + own + i < len) dsum += d;
        }
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            const int e = threadIdx.x + k * 64 * W;
            if (e < TS * BC * NP) ((float*)bc[buf])[e] = mv[k] ? to_float(r.m[k]) : 0.0f;
        }
    };
    auto finish = [&](int t0) {
        const int n = len - t0 - own;
#pragma unroll
        for (int i = 0; i < OWN; ++i) {
            float o = skip * to_float(fx[i]);
#pragma unroll
            for (int w = 0; w < W; ++w) o += part[w][own + i][q.lane];
            if (GATED) {
                const float z = to_float(fz[i]);
                o *= z * sigmoid_t<T>(z);
            }
            if (q.live && i < n) (yp + (int64_t)(t0 + own + i) * p.y.row)[c] = from_float<T>(o);
        }
    };
    auto step = [&](const f32x2 v, const f32x4 Bv, const f32x4 Cv) {
        float o = 0.0f;
#pragma unroll
        for (int n = 0; n < kStates; ++n) {
            h[n] = exp2_fast(v[0] * A[n]) * h[n] + v[1] * Bv[n];
            if (OUT) o += Cv[n] * h[n];
        }
        return o;
    };

    // Everything loaded so far arrives before the walk's own loads start: a value still under way at the loop's
    // head would make every tile wait there for all loads, the next tiles' among them.
    __builtin_amdgcn_s_waitcnt(kVm0);
    __builtin_amdgcn_sched_barrier(0);
    if (len > 0) {
#pragma unroll
        for (int a = 0; a < AHEAD; ++a) fetch(raw[a], a * TS);
        publish(raw[0], 0, 0);
    }
    auto tile = [&](int t0, Raw& r, const Raw& next, int buf) {
        const int cnt = min(TS, len - t0);
#pragma unroll
        for (int i = 0; i < OWN; ++i) {
            fx[i] = r.x[i];
            if (GATED) fz[i] = r.z[i];
        }
        fetch(r, t0 + AHEAD * TS);
        __syncthreads();
        if (cnt == TS) {
            f32x4 Bv[2][U], Cv[2][U];
            f32x2 v[2][U];
            auto load = [&](int slot, int s) {
#pragma unroll
                for (int j = 0; j < U; ++j) {
                    v[slot][j] = du[buf][s + j][q.lane];
                    Bv[slot][j] = bc[buf][s + j][0][q.wave];
                    if (OUT) Cv[slot][j] = bc[buf][s + j][BC - 1][q.wave];
                }
            };
            load(0, 0);
#pragma unroll
            for (int g = 0; g < TS / U; ++g) {
                if (g + 1 < TS / U) load((g + 1) & 1, (g + 1) * U);
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int j = 0; j < U; ++j) {
                    const float o = step(v[g & 1][j], Bv[g & 1][j], OUT ? Cv[g & 1][j] : Bv[g & 1][j]);
                    if (OUT) part[q.wave][g * U + j][q.lane] = o;
                }
            }
        } else {
            for (int s = 0; s < cnt; ++s) {
                const float o = step(du[buf][s][q.lane], bc[buf][s][0][q.wave], bc[buf][s][BC - 1][q.wave]);
                if (OUT) part[q.wave][s][q.lane] = o;
            }
        }
        publish(next, t0 + TS, buf ^ 1);
        if (OUT) {
            __syncthreads();
            finish(t0);
        }
    };
    for (int t0 = 0; t0 < len; t0 += AHEAD * TS) {
#pragma unroll
        for (int a = 0; a < AHEAD; ++a)
            if (t0 + a * TS < len) tile(t0 + a * TS, raw[a], raw[(a + 1) % AHEAD], a & 1);
    }
    if (OUT) {
        for (int t = len + q.wave; t < s1 - s0; t += W)
            if (q.live) (yp + t * p.y.row)[c] = from_float<T>(0.0f);
        if (p.state_out && q.seg == sg.nseg - 1 && q.live)
            store_states(p.state_out + srow, ns, f32x4{h[0], h[1], h[2], h[3]});
    } else {
        if (q.live) store_states(ws.ends + erow, ns, f32x4{h[0], h[1], h[2], h[3]});
        __syncthreads();
        float* red = &part[0][0][0];               // [64], one wave after another in order
        for (int w = 0; w < W; ++w) {
            if (q.wave == w) red[q.lane] = (w ? red[q.lane] : 0.0f) + dsum;
            __syncthreads();
        }
        if (q.wave == 0 && q.live) ws.sums[((size_t)q.b * sg.nseg + q.seg) * p.D + q.c] = red[q.lane];
    }
}

__global__ __launch_bounds__(256) void scan_starts_kernel(ScanProblem p, Segments sg, float* __restrict__ ends,
                                                          const float* __restrict__ sums)
{
    const int64_t DN = (int64_t)p.D * p.N;
    const int64_t i = block_id() * 256 + threadIdx.x;
    if (i >= p.B * DN) return;
    const int64_t b = i / DN, k = i % DN;
    const int c = (int)(k / p.N);
    const float A = p.a[k] * kLog2e;
    float h = p.state ? p.state[i] : 0.0f;
    float* e = ends + b * sg.nseg * DN + k;
    const float* s = sums + b * sg.nseg * p.D + c;
    constexpr int LINKS = 8;                          // in batches, whose loads are under way together
    for (int j0 = 0; j0 < sg.nseg; j0 += LINKS) {
        float d[LINKS], v[LINKS];
#pragma unroll
        for (int k = 0; k < LINKS; ++k) {
            const int64_t j = min(j0 + k, sg.nseg - 1);
            d[k] = s[j * p.D];
            v[k] = e[j * DN];
        }
#pragma unroll
        for (int k = 0; k < LINKS; ++k) {
            if (j0 + k < sg.nseg) e[(j0 + k) * DN] = h;
            h = exp2_fast(d[k] * A) * h + v[k];
        }
    }
}

// Segments: a single walk costs one pass over the states' arithmetic, a segmented one about 1.8, and a SIMD needs
// two waves or more to hide a step's latencies.  With two on each (2048 waves) a single walk is faster (B=8 T=2048
// D=4096 N=16: 315 against 419 us), with one it is not (B=4: 259 against 214 us).  A segmented walk has waves for
// what the CUs hold, and 64 steps at least to a segment.
Segments segments_of(const ScanProblem& p)
{
    const int W = waves_of(p.N), TS = tile_steps(W);
    const int64_t waves = (int64_t)p.B * channel_blocks(p) * W;
    const int tiles = (p.T + TS - 1) / TS;
    int64_t n = waves >= 2048 ? 1 : (W > 8 ? 4096 : 8192) / waves;
    if (n > p.T / 64) n = p.T / 64;
    if (n < 1) n = 1;
    const int per = (int)((tiles + n - 1) / n);
    return Segments{per * TS, (tiles + per - 1) / per};
}

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

SegWs seg_ws(const ScanProblem& p, const Segments& sg, char* base, size_t* bytes)
{
    SegWs w{nullptr, nullptr};
    *bytes = 0;
    if (sg.nseg <= 1) return w;
    const size_t e = align256((size_t)p.B * sg.nseg * p.D * p.N * 4), s = align256((size_t)p.B * sg.nseg * p.D * 4);
    w.ends = (float*)base;
    w.sums = (float*)(base + e);
    *bytes = e + s;
    return w;
}

// Single tokens and very short calls: moving the states is all there is.  L lanes share a channel, kStates states
// each, so a wave reads and writes its states in whole lines, and the lanes' shares of C h meet by lane swaps.
// B=64 T=1 D=4096 N=16: 36 MB in 12.5 us (2.9 TB/s); nothing is left to have under way meanwhile.
template <typename T, int L>
__global__ __launch_bounds__(256) void scan_step_kernel(ScanProblem p, int per_seq)
{
    const int64_t blk = block_id();
    if (blk >= (int64_t)p.B * per_seq) return;
    const int b = (int)(blk / per_seq), i = (int)(blk % per_seq) * 256 + threadIdx.x;
    const int c = min(i / L, p.D - 1), n0 = (i % L) * kStates;
    const bool live = i / L < p.D;
    const int ns = min(kStates, p.N - n0);
    const int len = clamp_len(p.lengths, b, p.T);
    const T* xp = (const T*)p.x.p + b * p.x.batch + c;
    const T* dp = (const T*)p.dt.p + b * p.dt.batch + c;
    const T* zp = p.z.p ? (const T*)p.z.p + b * p.z.batch + c : nullptr;
    T* yp = (T*)p.y.p + b * p.y.batch + c;
    const int g = c / (p.D / p.G);
    const T* Bp = (const T*)p.bmat.p + b * p.bmat.batch + g * p.N + n0;
    const T* Cp = (const T*)p.cmat.p + b * p.cmat.batch + g * p.N + n0;
    const size_t srow = ((size_t)b * p.D + c) * p.N + n0;
    const float skip = p.skip ? p.skip[c] : 0.0f, bias = p.dt_bias ? p.dt_bias[c] : 0.0f;
    const f32x4 A = load_states(p.a + (size_t)c * p.N + n0, ns);
    f32x4 h = {0.0f, 0.0f, 0.0f, 0.0f};
    if (p.state) h = load_states(p.state + srow, ns);
    for (int t = 0; t < p.T; ++t) {
        float o = 0.0f;
        if (t < len) {
            const float x = to_float(xp[t * p.x.row]), u = to_float(dp[t * p.dt.row]) + bias;
            const float d = p.softplus ? softplus_t<T>(u) : u;
            float Bv[kStates], Cv[kStates];
#pragma unroll
            for (int n = 0; n < kStates; ++n) {
                Bv[n] = n < ns ? to_float(Bp[t * p.bmat.row + n]) : 0.0f;
                Cv[n] = n < ns ? to_float(Cp[t * p.cmat.row + n]) : 0.0f;
            }
#pragma unroll
            for (int n = 0; n < kStates; ++n) {
                h[n] = exp2_fast(d * (A[n] * kLog2e)) * h[n] + d * x * Bv[n];
                o += Cv[n] * h[n];
            }
#pragma unroll
            for (int k = 1; k < L; k <<= 1) o += __shfl_xor(o, k);
            o += skip * x;
            if (zp) {
                const float z = to_float(zp[t * p.z.row]);
                o *= z * sigmoid_t<T>(z);
            }
        }
        if (live && n0 == 0) yp[t * p.y.row] = from_float<T>(o);
    }
    if (p.state_out && live) store_states(p.state_out + srow, ns, h);
}

template <typename T, int L>
hipError_t step_l(const ScanProblem& p, hipStream_t stream)
{
    const int per_seq = (int)(((int64_t)p.D * L + 255) / 256);
    scan_step_kernel<T, L><<<grid_of((int64_t)p.B * per_seq), 256, 0, stream>>>(p, per_seq);
    return hipGetLastError();
}

// Calls of up to this many steps go to the step kernel.
constexpr int kStepRows = 4;

template <typename T, int W>
hipError_t fwd_w(const ScanProblem& p, hipStream_t stream)
{
    const Segments sg = segments_of(p);
    size_t bytes;
    const SegWs ws = seg_ws(p, sg, p.ws, &bytes);
    const unsigned blocks = (unsigned)p.B * sg.nseg * channel_blocks(p);
    if (sg.nseg > 1) {
        scan_fwd_kernel<T, W, false, false><<<blocks, 64 * W, 0, stream>>>(p, sg, ws);
        hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        const int64_t n = (int64_t)p.B * p.D * p.N;
        scan_starts_kernel<<<grid_of((n + 255) / 256), 256, 0, stream>>>(p, sg, ws.ends, ws.sums);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    if (p.z.p) scan_fwd_kernel<T, W, true, true><<<blocks, 64 * W, 0, stream>>>(p, sg, ws);
    else scan_fwd_kernel<T, W, true, false><<<blocks, 64 * W, 0, stream>>>(p, sg, ws);
    return hipGetLastError();
}

template <typename T>
hipError_t fwd_t(const ScanProblem& p, hipStream_t stream)
{
    if (p.T <= kStepRows) switch (waves_of(p.N)) {
        case 1: return step_l<T, 1>(p, stream);
        case 2: return step_l<T, 2>(p, stream);
        case 4: return step_l<T, 4>(p, stream);
        case 8: return step_l<T, 8>(p, stream);
        default: return step_l<T, 16>(p, stream);
        }
    switch (waves_of(p.N)) {
    case 1: return fwd_w<T, 1>(p, stream);
    case 2: return fwd_w<T, 2>(p, stream);
    case 4: return fwd_w<T, 4>(p, stream);
    case 8: return fwd_w<T, 8>(p, stream);
    default: return fwd_w<T, 16>(p, stream);
    }
}

}  // namespace

size_t scan_workspace(const ScanProblem& p)
{
    size_t bytes;
    seg_ws(p, segments_of(p), nullptr, &bytes);
    return bytes;
}

hipError_t launch_scan_fwd(const ScanProblem& p, hipStream_t stream)
{
    return p.bf16 ? fwd_t<bf16>(p, stream) : fwd_t<float>(p, stream);
}

}  // namespace tfla
