// conv.hip -- causal depthwise convolution over [B,T,D] with channels last.
//
//   u_t = bias + sum_{j<K} w_j X_{t-K+1+j},  y_t = u_t or SiLU(u_t)
//
// X is the carried state's K-1 rows, then x.  A thread owns VEC neighbouring
// channels and a run of rows: the K-1 rows before it in registers, each row
// of x loaded once.  2 K flops an element against 2 elements moved: bound by
// memory.
#include "act.hpp"
#include "blocks.hpp"

namespace tfla {
namespace {

__device__ __forceinline__ int clamp_len(const int* lengths, int b, int T)
{
    return lengths ? min(max(lengths[b], 0), T) : T;
}

struct ConvGeom {
    int B, T, D, nv;      // nv: vectors of VEC channels in a row
    int run, nrun;        // rows of a run, runs of a sequence
};

// One thread: channels c0 .. c0+VEC-1, rows t0 .. t0+run-1 of sequence b.
template <typename T, int VEC, int K>
__global__ __launch_bounds__(256) void conv_fwd_kernel(ConvGeom g, const T* __restrict__ x, int64_t xb, int64_t xr,
                                                       const float* __restrict__ w, const float* __restrict__ bias,
                                                       const T* state, const int* __restrict__ lengths,
                                                       T* __restrict__ y, int64_t yb, int64_t yr, T* state_out,
                                                       int silu)
{
    const int64_t item = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (item >= (int64_t)g.B * g.nrun * g.nv) return;
    const int c0 = (int)(item % g.nv) * VEC;
    const int64_t rb = item / g.nv;
    const int r = (int)(rb % g.nrun), b = (int)(rb / g.nrun);
    const int t0 = r * g.run, t1 = min(t0 + g.run, g.T);
    const int len = clamp_len(lengths, b, g.T);
    x += b * xb + c0;
    y += b * yb + c0;
    const size_t srow = ((size_t)b * (K - 1)) * g.D + c0;

    float wk[K][VEC], bs[VEC], win[K][VEC];   // win[j]: X[t-K+1+j]
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
        bs[v] = bias ? bias[c0 + v] : 0.0f;
#pragma unroll
        for (int j = 0; j < K; ++j) wk[j][v] = w[(size_t)(c0 + v) * K + j];
    }
#pragma unroll
    for (int j = 0; j + 1 < K; ++j) {
        const int p = t0 - (K - 1) + j;
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            float s = 0.0f;
            if (p < 0) s = state ? to_float(state[srow + (size_t)(p + K - 1) * g.D + v]) : 0.0f;
            else if (p < len) s = to_float(x[p * xr + v]);
            win[j][v] = s;
        }
    }
    for (int t = t0; t < t1; ++t) {
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            float o = 0.0f;
            if (t < len) {
                win[K - 1][v] = to_float(x[t * xr + v]);
                float u = bs[v];
#pragma unroll
                for (int j = 0; j < K; ++j) u += wk[j][v] * win[j][v];
                o = silu ? u * sigmoid_f(u) : u;
#pragma unroll
                for (int j = 0; j + 1 < K; ++j) win[j][v] = win[j + 1][v];
            }
            y[t * yr + v] = from_float<T>(o);
        }
    }
    // The thread that read the state's rows also writes the new ones, in
    // ascending order from rows at or after the one written: in place is safe.
    if (state_out && r == 0) {
#pragma unroll
        for (int i = 0; i + 1 < K; ++i) {
            const int p = len - (K - 1) + i;
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                T s = from_float<T>(0.0f);
                if (p >= 0) s = x[p * xr + v];
                else if (state) s = state[srow + (size_t)(p + K - 1) * g.D + v];
                state_out[srow + (size_t)i * g.D + v] = s;
            }
        }
    }
}

// Backward.  du_t = dy_t act'(u_t); dX_p = sum_i w_{K-1-i} du_{p+i};
// dw_j = sum_t du_t X_{t-K+1+j}.  A thread walks t over its run and the K-1
// rows behind it (whose du it recomputes), so dX_p is complete at
// t = p+K-1; run 0 also yields the rows of the carried state.  Weight
// gradients of the run's own rows go to `part`, one row of sums for each
// block row, and are summed over the runs in a fixed order afterwards.
template <typename T, int VEC, int K>
__global__ __launch_bounds__(256) void conv_bwd_kernel(ConvGeom g, const T* __restrict__ x, int64_t xb, int64_t xr,
                                                       const float* __restrict__ w, const float* __restrict__ bias,
                                                       const T* state, const int* __restrict__ lengths,
                                                       const T* __restrict__ dy, int64_t gb, int64_t gr,
                                                       const T* dso, T* __restrict__ dx, int64_t db, int64_t dr,
                                                       T* dstate, float* __restrict__ part, int silu)
{
    const int64_t item = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (item >= (int64_t)g.B * g.nrun * g.nv) return;
    const int c0 = (int)(item % g.nv) * VEC;
    const int64_t rb = item / g.nv;
    const int r = (int)(rb % g.nrun), b = (int)(rb / g.nrun);
    const int t0 = r * g.run, t1 = min(t0 + g.run, g.T);
    const int len = clamp_len(lengths, b, g.T);
    x += b * xb + c0;
    dy += b * gb + c0;
    dx += b * db + c0;
    const size_t srow = ((size_t)b * (K - 1)) * g.D + c0;

    float wk[K][VEC], bs[VEC], win[K][VEC], dw[K + 1][VEC];
    float du[K][VEC];                         // du[i]: du_{t-K+1+i}
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
        bs[v] = bias ? bias[c0 + v] : 0.0f;
        dw[K][v] = 0.0f;
#pragma unroll
        for (int j = 0; j < K; ++j) {
            wk[j][v] = w[(size_t)(c0 + v) * K + j];
            dw[j][v] = 0.0f;
            du[j][v] = 0.0f;
        }
    }
#pragma unroll
    for (int j = 0; j + 1 < K; ++j) {
        const int p = t0 - (K - 1) + j;
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            float s = 0.0f;
            if (p < 0) s = state ? to_float(state[srow + (size_t)(p + K - 1) * g.D + v]) : 0.0f;
            else if (p < len) s = to_float(x[p * xr + v]);
            win[j][v] = s;
        }
    }
    const int first = r == 0 ? -(K - 1) : t0;   // rows of X this thread writes: first .. t1-1
    for (int t = t0; t < t1 + K - 1; ++t) {
        const bool live = t < len, own = t < t1;
        const int p = t - (K - 1);
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            float d = 0.0f;
            if (live) {
                win[K - 1][v] = to_float(x[t * xr + v]);
                d = to_float(dy[t * gr + v]);
                if (silu) {
                    float u = bs[v];
#pragma unroll
                    for (int j = 0; j < K; ++j) u += wk[j][v] * win[j][v];
                    const float sg = sigmoid_f(u);
                    d *= sg * (1.0f + u * (1.0f - sg));
                }
                if (own) {
#pragma unroll
                    for (int j = 0; j < K; ++j) dw[j][v] += d * win[j][v];
                    dw[K][v] += d;
                }
#pragma unroll
                for (int j = 0; j + 1 < K; ++j) win[j][v] = win[j + 1][v];
            }
            du[K - 1][v] = d;
            if (p >= first && p < t1) {
                float o = 0.0f;
                if (p < len) {
#pragma unroll
                    for (int i = 0; i < K; ++i) o += wk[K - 1 - i][v] * du[i][v];
                    const int q = p - (len - (K - 1));   // row of state_out that is X_p
                    if (dso && q >= 0) o += to_float(dso[srow + (size_t)q * g.D + v]);
                }
                if (p >= 0) dx[p * dr + v] = from_float<T>(o);
                else if (dstate) dstate[srow + (size_t)(p + K - 1) * g.D + v] = from_float<T>(o);
            }
#pragma unroll
            for (int i = 0; i + 1 < K; ++i) du[i][v] = du[i + 1][v];
        }
    }
#pragma unroll
    for (int v = 0; v < VEC; ++v)
#pragma unroll
        for (int j = 0; j <= K; ++j) part[((size_t)rb * (K + 1) + j) * g.D + c0 + v] = dw[j][v];
}

// dweight [D,K] and dbias [D] from the runs' sums [parts][K+1][D]
__global__ __launch_bounds__(256) void conv_params_kernel(const float* __restrict__ part, int parts, int D, int K,
                                                          float* __restrict__ dweight, float* __restrict__ dbias)
{
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= (int64_t)(K + 1) * D) return;
    const int j = (int)(i / D), c = (int)(i % D);
    float s = 0.0f;
    for (int r = 0; r < parts; ++r) s += part[(size_t)r * (K + 1) * D + i];
    if (j < K) dweight[(size_t)c * K + j] = s;
    else if (dbias) dbias[c] = s;
}

int run_rows(int B, int T, int D)
{
    (void)B;
    (void)D;
    return T < 64 ? T : 64;
}

template <typename T, int K>
hipError_t fwd_t(const ConvProblem& p, hipStream_t stream)
{
    ConvGeom g{p.B, p.T, p.D, p.D, run_rows(p.B, p.T, p.D), 0};
    g.nrun = (p.T + g.run - 1) / g.run;
    const int64_t items = (int64_t)p.B * g.nrun * g.nv;
    conv_fwd_kernel<T, 1, K><<<dim3((unsigned)((items + 255) / 256)), 256, 0, stream>>>(
        g, (const T*)p.x.p, p.x.batch, p.x.row, p.weight, p.bias, (const T*)p.state, p.lengths, (T*)p.y.p, p.y.batch,
        p.y.row, (T*)p.state_out, p.silu);
    return hipGetLastError();
}

template <typename T, int K>
hipError_t bwd_t(const ConvProblem& p, hipStream_t stream)
{
    ConvGeom g{p.B, p.T, p.D, p.D, run_rows(p.B, p.T, p.D), 0};
    g.nrun = (p.T + g.run - 1) / g.run;
    const int64_t items = (int64_t)p.B * g.nrun * g.nv;
    conv_bwd_kernel<T, 1, K><<<dim3((unsigned)((items + 255) / 256)), 256, 0, stream>>>(
        g, (const T*)p.x.p, p.x.batch, p.x.row, p.weight, p.bias, (const T*)p.state, p.lengths, (const T*)p.dy.p,
        p.dy.batch, p.dy.row, (const T*)p.dstate_out, (T*)p.dx.p, p.dx.batch, p.dx.row, (T*)p.dstate, p.part, p.silu);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int64_t n = (int64_t)(K + 1) * p.D;
    conv_params_kernel<<<dim3((unsigned)((n + 255) / 256)), 256, 0, stream>>>(p.part, p.B * g.nrun, p.D, K, p.dweight,
                                                                             p.dbias);
    return hipGetLastError();
}

template <typename T, bool BWD>
hipError_t by_taps(const ConvProblem& p, hipStream_t stream)
{
    switch (p.K) {
#define TFLA_TAPS(k) case k: return BWD ? bwd_t<T, k>(p, stream) : fwd_t<T, k>(p, stream)
    TFLA_TAPS(1);
    TFLA_TAPS(2);
    TFLA_TAPS(3);
    TFLA_TAPS(4);
    TFLA_TAPS(5);
    TFLA_TAPS(6);
    TFLA_TAPS(7);
    default: return BWD ? bwd_t<T, 8>(p, stream) : fwd_t<T, 8>(p, stream);
#undef TFLA_TAPS
    }
}

}  // namespace

size_t conv_bwd_workspace(int B, int T, int D, int K, bool bf16)
{
    (void)bf16;
    const int run = run_rows(B, T, D);
    return (size_t)B * ((T + run - 1) / run) * (K + 1) * D * sizeof(float);
}

hipError_t launch_conv_fwd(const ConvProblem& p, hipStream_t stream)
{
    return p.bf16 ? by_taps<bf16, false>(p, stream) : by_taps<float, false>(p, stream);
}

hipError_t launch_conv_bwd(const ConvProblem& p, hipStream_t stream)
{
    return p.bf16 ? by_taps<bf16, true>(p, stream) : by_taps<float, true>(p, stream);
}

}  // namespace tfla
