// conv.hip -- causal depthwise convolution over [B,T,D] with channels last.
//
//   u_t = bias + sum_{j<K} w_j X_{t-K+1+j},  y_t = u_t or SiLU(u_t)
//
// X is the carried state's K-1 rows, then x.  A thread owns VEC neighbouring
// channels and a run of rows, loads each row of its run once, kRows at a time
// and one such group ahead, and keeps the K-1 rows before a group in
// registers, so what is read twice is K-1 rows a run (from the caches).
// 2 K + 6 flops an element against 2 elements moved: bound by memory
// (B=4 T=4096 D=4096 bf16, K=4: forward 268 MB in 48 us, 5.6 TB/s, where a copy
// moves 5.1; backward 403 MB in 82 us, whose 33 issue slots an element
// take 69 % of what there is).
//
// VEC is 8 bytes (4 in the backward pass, whose sums take the registers)
// where the number of channels, the addresses and the strides allow it, else
// 1 element (B=4 T=4096 D=4096 with rows an element longer: bf16 85 us where
// aligned rows take 47, backward 138 and 79; fp32 171 and 94, 231 and 177).
// 16 bytes leave too few waves for short calls (padded prompts,
// B=6 T=1531 D=2048: 23 us against 17) and gain nothing on long ones.
#include "act.hpp"
#include "blocks.hpp"
#include "sums.hpp"

#include <type_traits>

namespace tfla {
namespace {

constexpr int kRows = 4;   // rows loaded together

__device__ __forceinline__ int clamp_len(const int* lengths, int b, int T)
{
    return lengths ? min(max(lengths[b], 0), T) : T;
}

// VEC elements as they lie in memory
template <typename T, int VEC> struct Pack {
    typedef T vec __attribute__((ext_vector_type(VEC)));
    vec v;
    __device__ __forceinline__ void load(const T* p) { v = *(const vec*)p; }
    // non-temporal: this launch does not read it again (B=4 T=4096 D=4096 backward: 94 us with plain stores, 81 so;
    // padded prompts 17.8 and 15.9)
    __device__ __forceinline__ void store(T* p) const { __builtin_nontemporal_store(v, (vec*)p); }
    __device__ __forceinline__ float get(int i) const { return to_float((T)v[i]); }
    __device__ __forceinline__ void set(int i, float x) { v[i] = from_float<T>(x); }
};
template <typename T> struct Pack<T, 1> {
    T v;
    __device__ __forceinline__ void load(const T* p) { v = *p; }
    __device__ __forceinline__ void store(T* p) const { *p = v; }
    __device__ __forceinline__ float get(int) const { return to_float(v); }
    __device__ __forceinline__ void set(int, float x) { v = from_float<T>(x); }
};

// A wave owns 64 vectors of channels and a run of rows (so all that depends on
// the row alone is scalar), a workgroup four runs of the same channels.
struct ConvGeom {
    int nv;               // vectors of VEC channels in a row
    int run, nrun;        // rows of a run, runs of a sequence
    int ncb;              // workgroups across a row
    int64_t groups;       // and down the runs
};

// The wave's run and the lane's channels; false: none.
struct ConvPlace {
    int64_t group, rb;
    int cb, cv, lane, wave;
    __device__ __forceinline__ bool set(const ConvProblem& p, const ConvGeom& g)
    {
        group = block_id() / g.ncb;
        cb = (int)(block_id() % g.ncb);
        lane = threadIdx.x & 63;
        wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        cv = cb * 64 + lane;
        rb = group * 4 + wave;
        return cv < g.nv && rb < (int64_t)p.B * g.nrun;
    }
};

// The K-1 rows before row t0 (r > 0: none of them from the state).
template <typename T, int VEC, int K>
__device__ __forceinline__ void history(float (*xr)[VEC], const T* x, int64_t row, int t0, int len, const T* state, int D)
{
#pragma unroll
    for (int j = 0; j + 1 < K; ++j) {
        const int p = t0 - (K - 1) + j;
        Pack<T, VEC> v;
        v.load(x + max(min(p, len - 1), 0) * row);
        const bool in = p >= 0 && p < len;
#pragma unroll
        for (int i = 0; i < VEC; ++i) xr[j][i] = in ? v.get(i) : 0.0f;
        if (p < 0 && state) {
            v.load(state + (size_t)(p + K - 1) * D);
#pragma unroll
            for (int i = 0; i < VEC; ++i) xr[j][i] = v.get(i);
        }
    }
}

template <typename T, int VEC, int K, bool SILU>
__global__ __launch_bounds__(256) void conv_fwd_kernel(ConvProblem p, ConvGeom g)
{
    ConvPlace q;
    if (!q.set(p, g)) return;
    const int c0 = q.cv * VEC;
    const int r = (int)(q.rb % g.nrun), b = (int)(q.rb / g.nrun);
    const int t0 = r * g.run, t1 = min(t0 + g.run, p.T);
    const int len = clamp_len(p.lengths, b, p.T);
    const T* x = (const T*)p.x.p + b * p.x.batch + c0;
    T* y = (T*)p.y.p + b * p.y.batch + c0;
    const size_t srow = ((size_t)b * (K - 1)) * p.D + c0;
    const T* state = p.state ? (const T*)p.state + srow : nullptr;

    Pack<T, VEC> raw[kRows];
    // rows behind the end are read as the last (or first) one and not used: no branch stands around a load
    auto fetch = [&](int t) {
#pragma unroll
        for (int k = 0; k < kRows; ++k) raw[k].load(x + max(min(t + k, len - 1), 0) * p.x.row);
    };
    fetch(t0);
    float wk[K][VEC], bs[VEC], xr[K - 1 + kRows][VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
        bs[v] = p.bias ? p.bias[c0 + v] : 0.0f;
#pragma unroll
        for (int j = 0; j < K; ++j) wk[j][v] = p.weight[(size_t)(c0 + v) * K + j];
    }
    history<T, VEC, K>(xr, x, p.x.row, t0, len, state, p.D);
    // ALL: every row of the group is one of the run's, before the end
    auto rows = [&](auto ALL, int t) {
        constexpr bool all = decltype(ALL)::value;
#pragma unroll
        for (int k = 0; k < kRows; ++k)
#pragma unroll
            for (int v = 0; v < VEC; ++v) xr[K - 1 + k][v] = raw[k].get(v);
        fetch(t + kRows);
#pragma unroll
        for (int k = 0; k < kRows; ++k) {
            Pack<T, VEC> o;
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                float u = bs[v];
#pragma unroll
                for (int j = 0; j < K; ++j) u += wk[j][v] * xr[k + j][v];
                if (SILU) u *= sigmoid_t<T>(u);
                o.set(v, all || t + k < len ? u : 0.0f);
            }
            if (all || t + k < t1) o.store(y + (t + k) * p.y.row);
        }
#pragma unroll
        for (int j = 0; j + 1 < K; ++j)
#pragma unroll
            for (int v = 0; v < VEC; ++v) xr[j][v] = xr[j + kRows][v];
    };
    for (int t = t0; t < t1; t += kRows) {
        if (t + kRows <= min(t1, len)) rows(std::true_type{}, t);
        else rows(std::false_type{}, t);
    }
    // The thread that read the state's rows also writes the new ones, in
    // ascending order from rows at or after the one written: in place is safe.
    if (p.state_out && r == 0) {
        T* out = (T*)p.state_out + srow;
#pragma unroll
        for (int i = 0; i + 1 < K; ++i) {
            const int q = len - (K - 1) + i;
            Pack<T, VEC> s;
#pragma unroll
            for (int v = 0; v < VEC; ++v) s.set(v, 0.0f);
            if (q >= 0) s.load(x + q * p.x.row);
            else if (state) s.load(state + (size_t)(q + K - 1) * p.D);
            s.store(out + (size_t)i * p.D);
        }
    }
}

// Backward.  du_t = dy_t act'(u_t); dX_p = sum_i w_{K-1-i} du_{p+i};
// dw_j = sum_t du_t X_{t-K+1+j}.  A thread walks t over its run and the K-1
// rows behind it (whose du it recomputes), so dX_p is complete at
// t = p+K-1; run 0 also yields the rows of the carried state.  The weight
// gradients of a workgroup's runs (each thread its own run's rows only) meet
// in LDS and go to `part`; the workgroups' sums are added in a fixed order
// afterwards.
template <typename T, int VEC, int K, bool SILU>
__global__ __launch_bounds__(256) void conv_bwd_kernel(ConvProblem p, ConvGeom g)
{
    __shared__ float red[256 * VEC];
    ConvPlace q;
    const bool live = q.set(p, g);
    if (q.group >= g.groups) return;
    float dw[K + 1][VEC];
#pragma unroll
    for (int j = 0; j <= K; ++j)
#pragma unroll
        for (int v = 0; v < VEC; ++v) dw[j][v] = 0.0f;
    const int c0 = min(q.cv, g.nv - 1) * VEC;
    if (live) {
        const int r = (int)(q.rb % g.nrun), b = (int)(q.rb / g.nrun);
        const int t0 = r * g.run, t1 = min(t0 + g.run, p.T);
        const int len = clamp_len(p.lengths, b, p.T);
        const T* x = (const T*)p.x.p + b * p.x.batch + c0;
        const T* dy = (const T*)p.dy.p + b * p.dy.batch + c0;
        T* dx = (T*)p.dx.p + b * p.dx.batch + c0;
        const size_t srow = ((size_t)b * (K - 1)) * p.D + c0;
        const T* state = p.state ? (const T*)p.state + srow : nullptr;
        const T* dso = p.dstate_out ? (const T*)p.dstate_out + srow : nullptr;
        T* dst = p.dstate ? (T*)p.dstate + srow : nullptr;

        Pack<T, VEC> rx[kRows], rd[kRows];
        auto fetch = [&](int t) {
#pragma unroll
            for (int k = 0; k < kRows; ++k) {
                const int64_t s = max(min(t + k, len - 1), 0);
                rx[k].load(x + s * p.x.row);
                rd[k].load(dy + s * p.dy.row);
            }
        };
        fetch(t0);
        float wk[K][VEC], bs[VEC], xr[K - 1 + kRows][VEC], du[K - 1 + kRows][VEC];
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            bs[v] = p.bias ? p.bias[c0 + v] : 0.0f;
#pragma unroll
            for (int j = 0; j < K; ++j) wk[j][v] = p.weight[(size_t)(c0 + v) * K + j];
#pragma unroll
            for (int j = 0; j + 1 < K; ++j) du[j][v] = 0.0f;
        }
        history<T, VEC, K>(xr, x, p.x.row, t0, len, state, p.D);
        const int first = r == 0 ? -(K - 1) : t0;   // rows of X this thread writes: first .. t1-1
        // ALL: every row of the group is one of the run's, before the end, and completes one that it writes to dx
        // without a part of dstate_out
        auto rows = [&](auto ALL, int t) {
            constexpr bool all = decltype(ALL)::value;
#pragma unroll
            for (int k = 0; k < kRows; ++k)
#pragma unroll
                for (int v = 0; v < VEC; ++v) {
                    xr[K - 1 + k][v] = all || t + k < len ? rx[k].get(v) : 0.0f;
                    du[K - 1 + k][v] = all || t + k < len ? rd[k].get(v) : 0.0f;
                }
            fetch(t + kRows);
#pragma unroll
            for (int k = 0; k < kRows; ++k) {
                const int s = t + k - (K - 1);              // the row of X completed here
                float o[VEC];
#pragma unroll
                for (int v = 0; v < VEC; ++v) {
                    float d = du[K - 1 + k][v];
                    if (SILU) {
                        float u = bs[v];
#pragma unroll
                        for (int j = 0; j < K; ++j) u += wk[j][v] * xr[k + j][v];
                        const float sg = sigmoid_t<T>(u);
                        d *= sg + u * sg * (1.0f - sg);
                        // behind the end d is 0, and 0 times a slope that overflowed must stay 0
                        if (!all && t + k >= len) d = 0.0f;
                        du[K - 1 + k][v] = d;
                    }
                    const float e = all || t + k < t1 ? d : 0.0f;
#pragma unroll
                    for (int j = 0; j < K; ++j) dw[j][v] += e * xr[k + j][v];
                    dw[K][v] += e;
                    o[v] = 0.0f;
#pragma unroll
                    for (int i = 0; i < K; ++i) o[v] += wk[K - 1 - i][v] * du[k + i][v];
                }
                Pack<T, VEC> w;
                if (all) {
#pragma unroll
                    for (int v = 0; v < VEC; ++v) w.set(v, o[v]);
                    w.store(dx + s * p.dx.row);
                } else if (s >= first && s < t1) {
                    const int e = s - (len - (K - 1));      // the row of state_out that is X_s
                    Pack<T, VEC> a;
#pragma unroll
                    for (int v = 0; v < VEC; ++v) a.set(v, 0.0f);
                    if (dso && e >= 0 && s < len) a.load(dso + (size_t)e * p.D);
#pragma unroll
                    for (int v = 0; v < VEC; ++v) w.set(v, s < len ? o[v] + a.get(v) : 0.0f);
                    if (s >= 0) w.store(dx + s * p.dx.row);
                    else if (dst) w.store(dst + (size_t)(s + K - 1) * p.D);
                }
            }
#pragma unroll
            for (int j = 0; j + 1 < K; ++j)
#pragma unroll
                for (int v = 0; v < VEC; ++v) {
                    xr[j][v] = xr[j + kRows][v];
                    du[j][v] = du[j + kRows][v];
                }
        };
        for (int t = t0; t < t1 + K - 1; t += kRows) {
            // rows t-K+1 .. t+kRows-K of X are completed
            if (t > t0 && t - (K - 1) >= t0 && t + kRows <= t1 && t + kRows - K < len - (K - 1)) rows(std::true_type{}, t);
            else rows(std::false_type{}, t);
        }
    }
#pragma unroll
    for (int j = 0; j <= K; ++j) {
        __syncthreads();
#pragma unroll
        for (int v = 0; v < VEC; ++v) red[(q.wave * VEC + v) * 64 + q.lane] = dw[j][v];
        __syncthreads();
        for (int i = threadIdx.x; i < VEC * 64; i += 256) {
            const int c = q.cb * 64 + (i & 63), v = i >> 6;
            const float s = (red[i] + red[i + VEC * 64]) + (red[i + 2 * VEC * 64] + red[i + 3 * VEC * 64]);
            if (c < g.nv) p.part[((size_t)q.group * (K + 1) + j) * p.D + (size_t)c * VEC + v] = s;
        }
    }
}

// dweight [D,K] and dbias [D] from the workgroups' sums [parts][K+1][D]
__global__ __launch_bounds__(1024) void conv_params_kernel(const float* __restrict__ part, int64_t parts, int D, int K,
                                                           float* __restrict__ dweight, float* __restrict__ dbias)
{
    __shared__ float red[16][64];
    const int64_t n = (int64_t)(K + 1) * D, i = (int64_t)blockIdx.x * 64 + threadIdx.x;
    const float s = part_sum(part, parts, n, n, blockIdx.x, red);
    if (threadIdx.x >= 64 || i >= n) return;
    const int j = (int)(i / D), c = (int)(i % D);
    if (j < K) dweight[(size_t)c * K + j] = s;
    else if (dbias) dbias[c] = s;
}

bool fits(const void* p, int64_t batch, int64_t row, const ConvProblem& c, size_t bytes)
{
    const size_t e = c.bf16 ? 2 : 4;
    return (uintptr_t)p % bytes == 0 && (c.B == 1 || batch * e % bytes == 0) && (c.T == 1 || row * e % bytes == 0);
}

// Elements of a vector: `bytes` of them where the rows, states and widths allow it and fill a wave, else 1.
int vec_of(const ConvProblem& p, size_t bytes, bool bwd)
{
    const size_t e = p.bf16 ? 2 : 4;
    const int v = (int)(bytes / e);
    bool ok = p.D % v == 0 && p.D >= 64 * v && fits(p.x.p, p.x.batch, p.x.row, p, bytes) && (uintptr_t)p.state % bytes == 0;
    if (bwd) ok = ok && fits(p.dy.p, p.dy.batch, p.dy.row, p, bytes) && fits(p.dx.p, p.dx.batch, p.dx.row, p, bytes) &&
                  (uintptr_t)p.dstate_out % bytes == 0 && (uintptr_t)p.dstate % bytes == 0;
    else ok = ok && fits(p.y.p, p.y.batch, p.y.row, p, bytes) && (uintptr_t)p.state_out % bytes == 0;
    return ok ? v : 1;
}

// Rows of a run, 8 at least (no run but the first then reaches into the state): as long as about `threads` threads
// remain, up to `most`.
int run_rows(int64_t rows, int T, int64_t nv, int64_t threads, int most)
{
    int run = 8;
    while (run < most && rows * nv / (2 * run) >= threads) run *= 2;
    return run < T ? run : T;
}

ConvGeom geom(const ConvProblem& p, int vec, bool bwd)
{
    ConvGeom g;
    g.nv = p.D / vec;
    g.run = run_rows((int64_t)p.B * p.T, p.T, g.nv, bwd ? 1 << 17 : 1 << 18, bwd ? 128 : 32);
    g.nrun = (p.T + g.run - 1) / g.run;
    g.ncb = (g.nv + 63) / 64;
    g.groups = ((int64_t)p.B * g.nrun + 3) / 4;
    return g;
}

template <typename T, int VEC, int K>
hipError_t fwd_v(const ConvProblem& p, hipStream_t stream)
{
    const ConvGeom g = geom(p, VEC, false);
    const dim3 blocks = grid_of(g.groups * g.ncb);
    if (p.silu) conv_fwd_kernel<T, VEC, K, true><<<blocks, 256, 0, stream>>>(p, g);
    else conv_fwd_kernel<T, VEC, K, false><<<blocks, 256, 0, stream>>>(p, g);
    return hipGetLastError();
}

template <typename T, int VEC, int K>
hipError_t bwd_v(const ConvProblem& p, hipStream_t stream)
{
    const ConvGeom g = geom(p, VEC, true);
    const dim3 blocks = grid_of(g.groups * g.ncb);
    if (p.silu) conv_bwd_kernel<T, VEC, K, true><<<blocks, 256, 0, stream>>>(p, g);
    else conv_bwd_kernel<T, VEC, K, false><<<blocks, 256, 0, stream>>>(p, g);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int64_t n = (int64_t)(K + 1) * p.D;
    conv_params_kernel<<<(unsigned)((n + 63) / 64), 1024, 0, stream>>>(p.part, g.groups, p.D, K, p.dweight, p.dbias);
    return hipGetLastError();
}

constexpr size_t kFwdBytes = 8, kBwdBytes = 4;

template <typename T, int K, bool BWD>
hipError_t by_width(const ConvProblem& p, hipStream_t stream)
{
    constexpr int V = (int)((BWD ? kBwdBytes : kFwdBytes) / sizeof(T));
    const bool wide = vec_of(p, BWD ? kBwdBytes : kFwdBytes, BWD) == V;
    if constexpr (BWD) return wide ? bwd_v<T, V, K>(p, stream) : bwd_v<T, 1, K>(p, stream);
    else return wide ? fwd_v<T, V, K>(p, stream) : fwd_v<T, 1, K>(p, stream);
}

template <typename T, bool BWD>
hipError_t by_taps(const ConvProblem& p, hipStream_t stream)
{
    switch (p.K) {
    case 1: return by_width<T, 1, BWD>(p, stream);
    case 2: return by_width<T, 2, BWD>(p, stream);
    case 3: return by_width<T, 3, BWD>(p, stream);
    case 4: return by_width<T, 4, BWD>(p, stream);
    case 5: return by_width<T, 5, BWD>(p, stream);
    case 6: return by_width<T, 6, BWD>(p, stream);
    case 7: return by_width<T, 7, BWD>(p, stream);
    default: return by_width<T, 8, BWD>(p, stream);
    }
}

}  // namespace

// For whichever width the call's addresses allow.
size_t conv_bwd_workspace(int B, int T, int D, int K, bool bf16)
{
    ConvProblem p{};
    p.B = B;
    p.T = T;
    p.D = D;
    p.K = K;
    p.bf16 = bf16;
    size_t most = 0;
    for (const int v : {1, (int)(kBwdBytes / (bf16 ? 2 : 4))}) {
        if (D % v) continue;
        const size_t n = (size_t)geom(p, v, true).groups * (K + 1) * D * sizeof(float);
        if (n > most) most = n;
    }
    return most;
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
