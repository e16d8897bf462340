// scan.hip -- forward pass of the selective scan (scan_impl.hpp).
#include "scan_impl.hpp"

namespace tfla {
namespace {

using namespace scan;

constexpr int TS = 16;   // steps of a tile

// W waves of kStates states.  Per tile of TS steps: each wave prepares its
// own steps' (delta, delta x); all walk the tile and leave their share of
// sum_n C h; each wave finishes its own steps.
template <typename T, int W>
__global__ __launch_bounds__(64 * W) void scan_fwd_kernel(ScanProblem p)
{
    __shared__ f32x2 du[TS][64];        // delta, delta x
    __shared__ float part[W][TS][64];
    const Place q = place(p);
    const int len = clamp_len(p.lengths, q.b, p.T);
    const int n0 = q.wave * kStates;
    const bool has = n0 < p.N;          // a wave behind the last state only shares the steps' work
    const int nn = has ? n0 : 0;
    const T* xp = (const T*)p.x.p + q.b * p.x.batch + q.c;
    const T* dp = (const T*)p.dt.p + q.b * p.dt.batch + q.c;
    const T* zp = p.z.p ? (const T*)p.z.p + q.b * p.z.batch + q.c : nullptr;
    T* yp = (T*)p.y.p + q.b * p.y.batch + q.c;
    const T* Bp = (const T*)p.bmat.p + q.b * p.bmat.batch + q.g * p.N + nn;
    const T* Cp = (const T*)p.cmat.p + q.b * p.cmat.batch + q.g * p.N + nn;
    const float skip = p.skip ? p.skip[q.c] : 0.0f;
    const float bias = p.dt_bias ? p.dt_bias[q.c] : 0.0f;
    const size_t srow = ((size_t)q.b * p.D + q.c) * p.N + nn;

    float A[kStates], h[kStates];
#pragma unroll
    for (int n = 0; n < kStates; ++n) {
        A[n] = p.a[(size_t)q.c * p.N + nn + n] * kLog2e;
        h[n] = p.state ? p.state[srow + n] : 0.0f;
    }
    for (int t0 = 0; t0 < len; t0 += TS) {
        const int cnt = min(TS, len - t0);
        float xv[TS / W > 0 ? TS / W : 1];
        for (int i = 0; i < TS / W; ++i) {
            const int s = q.wave + i * W;
            if (s < cnt) {
                xv[i] = to_float(xp[(t0 + s) * p.x.row]);
                const float u = to_float(dp[(t0 + s) * p.dt.row]) + bias;
                const float d = p.softplus ? softplus_f(u) : u;
                du[s][q.lane] = f32x2{d, d * xv[i]};
            }
        }
        __syncthreads();
        if (has) {
            for (int s = 0; s < cnt; ++s) {
                const f32x2 v = du[s][q.lane];
                Uniform4<T> Bv, Cv;
                Bv.load(Bp + (t0 + s) * p.bmat.row);
                Cv.load(Cp + (t0 + s) * p.cmat.row);
                float o = 0.0f;
#pragma unroll
                for (int n = 0; n < kStates; ++n) {
                    h[n] = exp2_fast(v[0] * A[n]) * h[n] + v[1] * Bv.v[n];
                    o += Cv.v[n] * h[n];
                }
                part[q.wave][s][q.lane] = o;
            }
        } else {
            for (int s = 0; s < cnt; ++s) part[q.wave][s][q.lane] = 0.0f;
        }
        __syncthreads();
        for (int i = 0; i < TS / W; ++i) {
            const int s = q.wave + i * W;
            if (s < cnt) {
                float o = skip * xv[i];
#pragma unroll
                for (int w = 0; w < W; ++w) o += part[w][s][q.lane];
                if (zp) {
                    const float z = to_float(zp[(t0 + s) * p.z.row]);
                    o *= z * sigmoid_f(z);
                }
                if (q.live) yp[(t0 + s) * p.y.row] = from_float<T>(o);
            }
        }
    }
    for (int t = len + q.wave; t < p.T; t += W)
        if (q.live) yp[t * p.y.row] = from_float<T>(0.0f);
    if (p.state_out && has && q.live)
#pragma unroll
        for (int n = 0; n < kStates; ++n) p.state_out[srow + n] = h[n];
}

template <typename T, int W>
hipError_t fwd_w(const ScanProblem& p, hipStream_t stream)
{
    const int per = p.D / p.G;
    const unsigned blocks = (unsigned)p.B * p.G * ((per + 63) / 64);
    scan_fwd_kernel<T, W><<<blocks, 64 * W, 0, stream>>>(p);
    return hipGetLastError();
}

template <typename T>
hipError_t fwd_t(const ScanProblem& p, hipStream_t stream)
{
    const int w = (p.N + kStates - 1) / kStates;
    if (w <= 1) return fwd_w<T, 1>(p, stream);
    if (w <= 2) return fwd_w<T, 2>(p, stream);
    if (w <= 4) return fwd_w<T, 4>(p, stream);
    if (w <= 8) return fwd_w<T, 8>(p, stream);
    return fwd_w<T, 16>(p, stream);
}

}  // namespace

size_t scan_workspace(const ScanProblem&) { return 0; }

hipError_t launch_scan_fwd(const ScanProblem& p, hipStream_t stream)
{
    return p.bf16 ? fwd_t<bf16>(p, stream) : fwd_t<float>(p, stream);
}

}  // namespace tfla
