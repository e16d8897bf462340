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
    const T* xp = (const T*)p.x.p + q.b * p.x.batch + s0 * p.x.row + q.c;
    const T* dp = (const T*)p.dt.p + q.b * p.dt.batch + s0 * p.dt.row + q.c;
    const bool gated = OUT && p.z.p;
    const T* zp = gated ? (const T*)p.z.p + q.b * p.z.batch + s0 * p.z.row + q.c : nullptr;
    T* yp = OUT ? (T*)p.y.p + q.b * p.y.batch + s0 * p.y.row + q.c : nullptr;
    const T* Bp = (const T*)p.bmat.p + q.b * p.bmat.batch + s0 * p.bmat.row + q.g * p.N + nn;
    const T* Cp = (const T*)p.cmat.p + q.b * p.cmat.batch + s0 * p.cmat.row + q.g * p.N + nn;
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

    float rx[OWN], rd[OWN], rz[OWN];                  // the next tile's inputs
    float fx[OWN], fz[OWN];                           // inputs the current tile's finish needs
    auto fetch = [&](int t0) {
#pragma unroll
        for (int i = 0; i < OWN; ++i) {
            const int t = t0 + q.wave + i * W;
            if (t < len) {
                rx[i] = to_float(xp[t * p.x.row]);
                rd[i] = to_float(dp[t * p.dt.row]);
                if (gated) rz[i] = to_float(zp[t * p.z.row]);
            }
        }
    };
    auto publish = [&](int t0, int buf) {
#pragma unroll
        for (int i = 0; i < OWN; ++i) {
            const int s = q.wave + i * W;
            if (t0 + s < len) {
                const float u = rd[i] + bias;
                const float d = p.softplus ? softplus_f(u) : u;
                du[buf][s][q.lane] = f32x2{d, d * rx[i]};
                if (!OUT) dsum += d;
            }
        }
    };
    auto finish = [&](int t0, int buf) {
#pragma unroll
        for (int i = 0; i < OWN; ++i) {
            const int s = q.wave + i * W;
            if (t0 + s < len) {
                float o = skip * fx[i];
#pragma unroll
                for (int w = 0; w < W; ++w) o += part[buf][w][s][q.lane];
                if (gated) o *= fz[i] * sigmoid_f(fz[i]);
                if (q.live) yp[(t0 + s) * p.y.row] = from_float<T>(o);
            }
        }
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
        float nx[OWN], nz[OWN];
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
            const T* Bt = Bp + t0 * p.bmat.row;
            const T* Ct = Cp + t0 * p.cmat.row;
            Uniform4<T> Bv[2][U4], Cv[2][U4];
            f32x2 v[2][U4];
#pragma unroll
            for (int j = 0; j < U4; ++j) {
                Bv[0][j].load(Bt + j * p.bmat.row);
                if (OUT) Cv[0][j].load(Ct + j * p.cmat.row);
                v[0][j] = du[buf][j][q.lane];
            }
#pragma unroll
            for (int g = 0; g < TS / U4; ++g) {
                if (g + 1 < TS / U4) {
#pragma unroll
                    for (int j = 0; j < U4; ++j) {
                        const int s = (g + 1) * U4 + j;
                        Bv[(g + 1) & 1][j].load(Bt + s * p.bmat.row);
                        if (OUT) Cv[(g + 1) & 1][j].load(Ct + s * p.cmat.row);
                        v[(g + 1) & 1][j] = du[buf][s][q.lane];
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
                Bv.load(Bp + (t0 + s) * p.bmat.row);
                if (OUT) Cv.load(Cp + (t0 + s) * p.cmat.row);
                const float o = step(du[buf][s][q.lane], Bv, Cv);
                if (OUT) part[buf][q.wave][s][q.lane] = o;
            }
        } else if (OUT) {
            for (int s = 0; s < cnt; ++s) part[buf][q.wave][s][q.lane] = 0.0f;
        }
        publish(t0 + TS, buf ^ 1);
    }
    if (OUT) {
        __syncthreads();
        if (len > 0) finish((len - 1) / TS * TS, ((len - 1) / TS) & 1);
        for (int t = len + q.wave; t < s1 - s0; t += W)
            if (q.live) yp[t * p.y.row] = from_float<T>(0.0f);
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
