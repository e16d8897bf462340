// scan.hip -- forward pass of the selective scan (scan_impl.hpp).
//
// A workgroup walks its segment in tiles of TS steps, with one barrier a
// tile: the waves publish the next tile's (delta, delta x) into the other of
// two LDS buffers while the current tile is walked, and finish the previous
// tile's outputs (the sum over the waves' shares of C h, the skip, the gate)
// from the other of two buffers of shares.  Inside a tile, B, C and the
// published steps of the next four steps are fetched before the current four
// are computed, so no product waits for a load.
//
// A long axis over few sequences and channels is cut into segments: every
// segment is first walked from a zero state for its end state (no outputs),
// the start states follow from those (a decay over a segment is
// exp(A sum delta)), and the second walk starts from them.
#include "scan_impl.hpp"

namespace tfla {
namespace {

using namespace scan;

constexpr int TS = 16;   // steps of a tile
constexpr int U4 = 4;    // steps fetched together

struct SegWs {
    float* ends;   // [B][nseg][D][N]
    float* sums;   // [B][nseg][D]
};

// OUT: the outputs; else the end state and the sum of the steps.
template <typename T, int W, bool OUT>
__global__ __launch_bounds__(64 * W) void scan_fwd_kernel(ScanProblem p, Segments sg, SegWs ws)
{
    constexpr int OWN = TS / W;                       // steps of a tile that a wave prepares and finishes
    __shared__ f32x2 du[2][TS][64];                   // delta, delta x
    __shared__ float part[OUT ? 2 : 1][OUT ? W : 1][OUT ? TS : 1][64];
    const Place q = place(p, sg);
    const int all = clamp_len(p.lengths, q.b, p.T);
    const int s0 = q.seg * sg.len, s1 = min(s0 + sg.len, p.T);
    const int len = max(0, min(all, s1) - s0);        // steps of this segment
    const int n0 = q.wave * kStates;
    const bool has = n0 < p.N;                        // a wave behind the last state only shares the steps' work
    const int nn = has ? n0 : 0;
    // Rows are addressed as a uniform pointer to the tile and 32-bit byte offsets within it
    // (the host refuses row strides for which those would not do).
    constexpr unsigned E = sizeof(T);
    const unsigned xr = (unsigned)p.x.row * E, dr = (unsigned)p.dt.row * E, zr = (unsigned)p.z.row * E,
                   yr = (unsigned)p.y.row * E, br = (unsigned)p.bmat.row * E, cr = (unsigned)p.cmat.row * E;
    const char* xp = (const char*)p.x.p + (q.b * p.x.batch + s0 * p.x.row) * E;
    const char* dp = (const char*)p.dt.p + (q.b * p.dt.batch + s0 * p.dt.row) * E;
    const bool gated = OUT && p.z.p;
    const char* zp = gated ? (const char*)p.z.p + (q.b * p.z.batch + s0 * p.z.row) * E : nullptr;
    char* yp = OUT ? (char*)p.y.p + (q.b * p.y.batch + s0 * p.y.row) * E : nullptr;
    const char* Bp = (const char*)p.bmat.p + (q.b * p.bmat.batch + s0 * p.bmat.row + q.g * p.N + nn) * E;
    const char* Cp = (const char*)p.cmat.p + (q.b * p.cmat.batch + s0 * p.cmat.row + q.g * p.N + nn) * E;
    const unsigned c = q.c * E, own = q.wave * OWN;   // the wave's steps of a tile: own .. own + OWN - 1
    auto in = [&](const char* base, unsigned row, int s) { return *(const T*)(base + (s * row + c)); };
    const float skip = OUT && p.skip ? p.skip[q.c] : 0.0f;
    const float bias = p.dt_bias ? p.dt_bias[q.c] : 0.0f;
    const size_t srow = ((size_t)q.b * p.D + q.c) * p.N + nn;
    const size_t erow = (((size_t)q.b * sg.nseg + q.seg) * p.D + q.c) * p.N + nn;

    float A[kStates], h[kStates] = {0.0f, 0.0f, 0.0f, 0.0f};
    {
        const f32x4 av = *(const f32x4u*)(p.a + (size_t)q.c * p.N + nn);
        // the start: the folded one of a segmented walk's second pass, else the caller's; 0 in its first pass
        const float* st = !OUT ? nullptr : sg.nseg > 1 ? ws.ends + erow : p.state ? p.state + srow : nullptr;
        f32x4 hv = {0.0f, 0.0f, 0.0f, 0.0f};
        if (st) hv = *(const f32x4u*)st;
#pragma unroll
        for (int n = 0; n < kStates; ++n) {
            A[n] = av[n] * kLog2e;
            h[n] = hv[n];
        }
    }
    float dsum = 0.0f;                                // this wave's steps

    // The next tile's inputs, and those that the current tile's finish needs, as they were loaded: a
    // conversion beside the load would wait for it there.
    T rx[OWN] = {}, rd[OWN] = {}, rz[OWN] = {}, fx[OWN] = {}, fz[OWN] = {};
    auto fetch = [&](int t0) {                        // the tile at xp, dp, zp, then on to the next
        if (t0 + TS <= len) {
#pragma unroll
            for (int i = 0; i < OWN; ++i) {
                rx[i] = in(xp, xr, own + i);
                rd[i] = in(dp, dr, own + i);
                if (gated) rz[i] = in(zp, zr, own + i);
            }
        } else {
#pragma unroll
            for (int i = 0; i < OWN; ++i)
                if (t0 + own + i < (unsigned)len) {
                    rx[i] = in(xp, xr, own + i);
                    rd[i] = in(dp, dr, own + i);
                    if (gated) rz[i] = in(zp, zr, own + i);
                }
        }
        xp += (uint64_t)TS * xr;
        dp += (uint64_t)TS * dr;
        if (gated) zp += (uint64_t)TS * zr;
    };
    auto publish = [&](int t0, int buf) {
#pragma unroll
        for (int i = 0; i < OWN; ++i) {
            const float u = to_float(rd[i]) + bias;
            const float d = p.softplus ? softplus_t<T>(u) : u;
            du[buf][own + i][q.lane] = f32x2{d, d * to_float(rx[i])};   // behind the end: never read
            if (!OUT && t0 + own + i < (unsigned)len) dsum += d;
        }
    };
    auto finish = [&](int t0, int buf) {              // the tile at yp, then on to the next
        const int n = len - t0 - (int)own;
#pragma unroll
        for (int i = 0; i < OWN; ++i) {
            float o = skip * to_float(fx[i]);
            const float z = to_float(fz[i]);
#pragma unroll
            for (int w = 0; w < W; ++w) o += part[buf][w][own + i][q.lane];
            if (gated) o *= z * sigmoid_t<T>(z);
            if (q.live && i < n) *(T*)(yp + ((own + i) * yr + c)) = from_float<T>(o);
        }
        yp += (uint64_t)TS * yr;
    };
    auto step = [&](const f32x2 v, const Uniform4<T>& Bv, const Uniform4<T>& Cv) {
        float o = 0.0f;
#pragma unroll
        for (int n = 0; n < kStates; ++n) {
            h[n] = exp2_fast(v[0] * A[n]) * h[n] + v[1] * Bv.get(n);
            if (OUT) o += Cv.get(n) * h[n];
        }
        return o;
    };

    fetch(0);
    publish(0, 0);
    for (int t0 = 0, k = 0; t0 < len; t0 += TS, ++k) {
        const int buf = k & 1, cnt = min(TS, len - t0);
        T nx[OWN], nz[OWN];
#pragma unroll
        for (int i = 0; i < OWN; ++i) {
            nx[i] = rx[i];
            nz[i] = rz[i];
        }
        fetch(t0 + TS);
        __syncthreads();
        if (OUT && k > 0) finish(t0 - TS, buf ^ 1);
#pragma unroll
        for (int i = 0; i < OWN; ++i) {
            fx[i] = nx[i];
            fz[i] = nz[i];
        }
        if (has && cnt == TS) {
            const char *Bt = Bp, *Ct = Cp;
            Uniform4<T> Bv[2][U4], Cv[2][U4];
            f32x2 v[2][U4];
#pragma unroll
            for (int j = 0; j < U4; ++j) {
                Bv[0][j].load((const T*)(Bt + j * br));
                if (OUT) Cv[0][j].load((const T*)(Ct + j * cr));
                v[0][j] = du[buf][j][q.lane];
            }
#pragma unroll
            for (int g = 0; g < TS / U4; ++g) {
                if (g + 1 < TS / U4) {
                    Bt += (uint64_t)U4 * br;
                    Ct += (uint64_t)U4 * cr;
#pragma unroll
                    for (int j = 0; j < U4; ++j) {
                        Bv[(g + 1) & 1][j].load((const T*)(Bt + j * br));
                        if (OUT) Cv[(g + 1) & 1][j].load((const T*)(Ct + j * cr));
                        v[(g + 1) & 1][j] = du[buf][(g + 1) * U4 + j][q.lane];
                    }
                }
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int j = 0; j < U4; ++j) {
                    const float o = step(v[g & 1][j], Bv[g & 1][j], Cv[g & 1][j]);
                    if (OUT) part[buf][q.wave][g * U4 + j][q.lane] = o;
                }
            }
        } else if (has) {
            for (int s = 0; s < cnt; ++s) {
                Uniform4<T> Bv, Cv;
                Bv.load((const T*)(Bp + s * br));
                if (OUT) Cv.load((const T*)(Cp + s * cr));
                const float o = step(du[buf][s][q.lane], Bv, Cv);
                if (OUT) part[buf][q.wave][s][q.lane] = o;
            }
        } else if (OUT) {
            for (int s = 0; s < cnt; ++s) part[buf][q.wave][s][q.lane] = 0.0f;
        }
        Bp += (uint64_t)TS * br;
        Cp += (uint64_t)TS * cr;
        publish(t0 + TS, buf ^ 1);
    }
    if (OUT) {
        __syncthreads();
        if (len > 0) finish((len - 1) / TS * TS, ((len - 1) / TS) & 1);
        T* y0 = (T*)p.y.p + q.b * p.y.batch + s0 * p.y.row + q.c;
        for (int t = len + q.wave; t < s1 - s0; t += W)
            if (q.live) y0[t * p.y.row] = from_float<T>(0.0f);
        if (p.state_out && q.seg == sg.nseg - 1 && has && q.live)
            *(f32x4u*)(p.state_out + srow) = f32x4{h[0], h[1], h[2], h[3]};
    } else {
        if (has && q.live) *(f32x4u*)(ws.ends + erow) = f32x4{h[0], h[1], h[2], h[3]};
        __syncthreads();
        float* red = &part[0][0][0][0];               // [64], one wave after another in order
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
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= p.B * DN) return;
    const int64_t b = i / DN, k = i % DN;
    const int c = (int)(k / p.N);
    const float A = p.a[k] * kLog2e;
    float h = p.state ? p.state[i] : 0.0f;
    float* e = ends + b * sg.nseg * DN + k;
    const float* s = sums + b * sg.nseg * p.D + c;
    for (int j = 0; j < sg.nseg; ++j) {
        const float next = exp2_fast(s[(int64_t)j * p.D] * A) * h + e[j * DN];
        e[j * DN] = h;
        h = next;
    }
}

// Segments: enough workgroups to fill the chip.  A single walk costs one pass
// over the states' arithmetic, a segmented one about 1.8, so an axis is cut
// only where a single walk leaves most of the chip idle.
Segments segments_of(const ScanProblem& p)
{
    const int W = waves_of(p.N);
    const int64_t waves = (int64_t)p.B * channel_blocks(p) * W;
    const int tiles = (p.T + TS - 1) / TS;
    int64_t n = waves >= 1024 ? 1 : 3072 / waves;
    if (n > tiles / 8) n = tiles / 8;                 // 128 steps at least
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

template <typename T, int W>
hipError_t fwd_w(const ScanProblem& p, hipStream_t stream)
{
    const Segments sg = segments_of(p);
    size_t bytes;
    const SegWs ws = seg_ws(p, sg, p.ws, &bytes);
    const unsigned blocks = (unsigned)p.B * sg.nseg * channel_blocks(p);
    if (sg.nseg > 1) {
        scan_fwd_kernel<T, W, false><<<blocks, 64 * W, 0, stream>>>(p, sg, ws);
        hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        const int64_t n = (int64_t)p.B * p.D * p.N;
        scan_starts_kernel<<<(unsigned)((n + 255) / 256), 256, 0, stream>>>(p, sg, ws.ends, ws.sums);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    scan_fwd_kernel<T, W, true><<<blocks, 64 * W, 0, stream>>>(p, sg, ws);
    return hipGetLastError();
}

template <typename T>
hipError_t fwd_t(const ScanProblem& p, hipStream_t stream)
{
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
