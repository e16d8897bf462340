// norm.hip -- group norm over [B,T,G,C] with channels last, and the
// activation or gate behind it.
//
//   xh = (x - mean) rstd,  u = xh w + bias,  y = act(u) or u act(gate)
//   v = du w,  dx = rstd (v - mean(v) - xh mean(v xh))
//
// A set is what shares one mean: the C channels of a token's group, or the
// T x C values of a sequence's group.
#include "act.hpp"
#include "blocks.hpp"

namespace tfla {
namespace {

__device__ __forceinline__ float act_f(float u, int act)
{
    if (act == kActNone) return u;
    const float s = sigmoid_f(u);
    return act == kActSilu ? u * s : s;
}

__device__ __forceinline__ float act_grad(float u, int act)
{
    if (act == kActNone) return 1.0f;
    const float s = sigmoid_f(u);
    return act == kActSilu ? s * (1.0f + u * (1.0f - s)) : s * (1.0f - s);
}

__device__ __forceinline__ int64_t at(const Heads& h, int b, int t, int g, int c)
{
    return b * h.batch + t * h.row + g * h.group + c;
}

__device__ __forceinline__ float block_sum(float v)
{
    __shared__ float s[4];
#pragma unroll
    for (int o = 32; o; o >>= 1) v += __shfl_xor(v, o);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
    __syncthreads();
    return (s[0] + s[1]) + (s[2] + s[3]);
}

struct Set {
    int b, t0, t1, g;
    int64_t id;
};

// Block -> set: token sets [B,T,G], sequence sets [B,G].
__device__ __forceinline__ Set set_of(const NormProblem& p)
{
    Set s;
    int64_t i = blockIdx.x;
    s.id = i;
    s.g = (int)(i % p.G);
    i /= p.G;
    if (p.sequence) {
        s.b = (int)i;
        s.t0 = 0;
        s.t1 = p.T;
    } else {
        s.b = (int)(i / p.T);
        s.t0 = (int)(i % p.T);
        s.t1 = s.t0 + 1;
    }
    return s;
}

template <typename T>
__global__ __launch_bounds__(256) void norm_fwd_kernel(NormProblem p)
{
    const Set s = set_of(p);
    const T* x = (const T*)p.x.p;
    const T* z = (const T*)p.gate.p;
    T* y = (T*)p.y.p;
    const int64_t n = (int64_t)(s.t1 - s.t0) * p.C;
    float m = 0.0f;
    for (int64_t i = threadIdx.x; i < n; i += 256) m += to_float(x[at(p.x, s.b, s.t0 + (int)(i / p.C), s.g, (int)(i % p.C))]);
    m = block_sum(m) / (float)n;
    float q = 0.0f;
    for (int64_t i = threadIdx.x; i < n; i += 256) {
        const float d = to_float(x[at(p.x, s.b, s.t0 + (int)(i / p.C), s.g, (int)(i % p.C))]) - m;
        q += d * d;
    }
    const float r = 1.0f / sqrtf(block_sum(q) / (float)n + p.eps);
    if (threadIdx.x == 0) {
        if (p.mean) p.mean[s.id] = m;
        if (p.rstd) p.rstd[s.id] = r;
    }
    for (int64_t i = threadIdx.x; i < n; i += 256) {
        const int t = s.t0 + (int)(i / p.C), c = (int)(i % p.C);
        const float w = p.weight ? p.weight[s.g * p.C + c] : 1.0f, bs = p.bias ? p.bias[s.g * p.C + c] : 0.0f;
        const float u = (to_float(x[at(p.x, s.b, t, s.g, c)]) - m) * r * w + bs;
        const float o = z ? u * act_f(to_float(z[at(p.gate, s.b, t, s.g, c)]), p.act) : act_f(u, p.act);
        y[at(p.y, s.b, t, s.g, c)] = from_float<T>(o);
    }
}

// xh, u, du and dgate's factor of one element
struct Elem1 {
    float xh, u, du, dz;
};
template <typename T>
__device__ __forceinline__ Elem1 elem(const NormProblem& p, float m, float r, int b, int t, int g, int c)
{
    Elem1 e;
    const float w = p.weight ? p.weight[g * p.C + c] : 1.0f, bs = p.bias ? p.bias[g * p.C + c] : 0.0f;
    e.xh = (to_float(((const T*)p.x.p)[at(p.x, b, t, g, c)]) - m) * r;
    e.u = e.xh * w + bs;
    const float dy = to_float(((const T*)p.dy.p)[at(p.dy, b, t, g, c)]);
    if (p.gate.p) {
        const float z = to_float(((const T*)p.gate.p)[at(p.gate, b, t, g, c)]);
        e.du = dy * act_f(z, p.act);
        e.dz = dy * e.u * act_grad(z, p.act);
    } else {
        e.du = dy * act_grad(e.u, p.act);
        e.dz = 0.0f;
    }
    return e;
}

template <typename T>
__global__ __launch_bounds__(256) void norm_bwd_kernel(NormProblem p)
{
    const Set s = set_of(p);
    const int64_t n = (int64_t)(s.t1 - s.t0) * p.C;
    const float m = p.mean[s.id], r = p.rstd[s.id];
    float s1 = 0.0f, s2 = 0.0f;
    for (int64_t i = threadIdx.x; i < n; i += 256) {
        const int t = s.t0 + (int)(i / p.C), c = (int)(i % p.C);
        const Elem1 e = elem<T>(p, m, r, s.b, t, s.g, c);
        const float v = e.du * (p.weight ? p.weight[s.g * p.C + c] : 1.0f);
        s1 += v;
        s2 += v * e.xh;
    }
    s1 = block_sum(s1) / (float)n;
    s2 = block_sum(s2) / (float)n;
    for (int64_t i = threadIdx.x; i < n; i += 256) {
        const int t = s.t0 + (int)(i / p.C), c = (int)(i % p.C);
        const Elem1 e = elem<T>(p, m, r, s.b, t, s.g, c);
        const float v = e.du * (p.weight ? p.weight[s.g * p.C + c] : 1.0f);
        ((T*)p.dx.p)[at(p.dx, s.b, t, s.g, c)] = from_float<T>(r * (v - s1 - e.xh * s2));
        if (p.dgate.p) ((T*)p.dgate.p)[at(p.dgate, s.b, t, s.g, c)] = from_float<T>(e.dz);
    }
}

// dweight, dbias: sums of a run of rows into ws [parts][2][G C], then over the parts
constexpr int kRun = 64;

template <typename T>
__global__ __launch_bounds__(256) void norm_params_kernel(NormProblem p)
{
    const int W = p.G * p.C, nb = (W + 255) / 256;
    const int64_t part = blockIdx.x / nb;
    const int i = (int)(blockIdx.x % nb) * 256 + threadIdx.x;
    if (i >= W) return;
    const int g = i / p.C, c = i % p.C;
    float s1 = 0.0f, s2 = 0.0f;
    const int64_t r1 = min((part + 1) * kRun, (int64_t)p.B * p.T);
    for (int64_t r = part * kRun; r < r1; ++r) {
        const int b = (int)(r / p.T), t = (int)(r % p.T);
        const int64_t id = (p.sequence ? b : r) * p.G + g;
        const Elem1 e = elem<T>(p, p.mean[id], p.rstd[id], b, t, g, c);
        s1 += e.du * e.xh;
        s2 += e.du;
    }
    float* o = (float*)p.ws + part * 2 * W;
    o[i] = s1;
    o[W + i] = s2;
}

__global__ __launch_bounds__(256) void norm_sums_kernel(NormProblem p, int64_t parts)
{
    const int W = p.G * p.C;
    const int i = blockIdx.x * 256 + threadIdx.x;
    if (i >= 2 * W) return;
    const float* src = (const float*)p.ws;
    float s = 0.0f;
    for (int64_t r = 0; r < parts; ++r) s += src[r * 2 * W + i];
    if (i < W) {
        if (p.dweight) p.dweight[i] = s;
    } else if (p.dbias) {
        p.dbias[i - W] = s;
    }
}

int64_t parts_of(const NormProblem& p) { return ((int64_t)p.B * p.T + kRun - 1) / kRun; }

template <typename T>
hipError_t bwd_t(const NormProblem& p, hipStream_t stream)
{
    const unsigned sets = (unsigned)p.B * (p.sequence ? 1 : p.T) * p.G;
    norm_bwd_kernel<T><<<sets, 256, 0, stream>>>(p);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || (!p.dweight && !p.dbias)) return e;
    const int W = p.G * p.C;
    const int64_t parts = parts_of(p);
    norm_params_kernel<T><<<(unsigned)(parts * ((W + 255) / 256)), 256, 0, stream>>>(p);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    norm_sums_kernel<<<(2 * W + 255) / 256, 256, 0, stream>>>(p, parts);
    return hipGetLastError();
}

}  // namespace

size_t norm_workspace(const NormProblem&) { return 0; }

hipError_t launch_norm_fwd(const NormProblem& p, hipStream_t stream)
{
    const unsigned sets = (unsigned)p.B * (p.sequence ? 1 : p.T) * p.G;
    if (p.bf16) norm_fwd_kernel<bf16><<<sets, 256, 0, stream>>>(p);
    else norm_fwd_kernel<float><<<sets, 256, 0, stream>>>(p);
    return hipGetLastError();
}

size_t norm_bwd_workspace(const NormProblem& p) { return (size_t)parts_of(p) * 2 * p.G * p.C * 4; }

hipError_t launch_norm_bwd(const NormProblem& p, hipStream_t stream)
{
    return p.bf16 ? bwd_t<bf16>(p, stream) : bwd_t<float>(p, stream);
}

}  // namespace tfla
