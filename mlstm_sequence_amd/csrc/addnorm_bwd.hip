// addnorm_bwd.hip -- residual sum with a layer or RMS norm, backward.
//
//   th = (t - mean) rstd,  v = dy weight
//   dt = rstd (v - mean(v) - th mean(v th)) + dtotal,  dweight = sum dy th,  dbias = sum dy
#include "gfx950.hpp"

#include "norm_impl.hpp"
#include "sums.hpp"

namespace tfla {
namespace {

constexpr int kRun = 64;   // rows of a part of the weights' gradients

// A workgroup to a row; its statistics go to the workspace.
template <typename T, typename S>
__global__ __launch_bounds__(256) void addnorm_bwd_kernel(AddNormProblem p)
{
    __shared__ float red[4];
    const int64_t id = block_id();
    if (id >= (int64_t)p.B * p.T) return;
    const int64_t b = id / p.T, t = id % p.T;
    const S* x = (const S*)p.total.p + b * p.total.batch + t * p.total.row;
    const T* g = (const T*)p.dy.p + b * p.dy.batch + t * p.dy.row;
    const S* e = p.dtotal.p ? (const S*)p.dtotal.p + b * p.dtotal.batch + t * p.dtotal.row : nullptr;
    T* dx = (T*)p.dx.p + b * p.dx.batch + t * p.dx.row;
    S* dr = p.dresidual.p ? (S*)p.dresidual.p + b * p.dresidual.batch + t * p.dresidual.row : nullptr;
    const float inv = 1.0f / (float)p.C;
    auto sum = [&](float v) { return norm::row_sum<true>(v, 256, red); };
    float s = 0.0f, q = 0.0f, s1 = 0.0f, s2 = 0.0f;
    for (int c = threadIdx.x; c < p.C; c += 256) s += to_float(x[c]);
    const float mean = p.rms ? 0.0f : sum(s) * inv;
    for (int c = threadIdx.x; c < p.C; c += 256) {
        const float d = to_float(x[c]) - mean, v = to_float(g[c]) * (p.weight ? p.weight[c] : 1.0f);
        q += d * d;
        s1 += v;
        s2 += v * d;
    }
    const float rstd = 1.0f / sqrtf(sum(q) * inv + p.eps);
    s1 = p.rms ? 0.0f : sum(s1) * inv;
    s2 = sum(s2) * inv * rstd * rstd;
    for (int c = threadIdx.x; c < p.C; c += 256) {
        const float d = to_float(x[c]) - mean, v = to_float(g[c]) * (p.weight ? p.weight[c] : 1.0f);
        const float o = rstd * (v - s1 - d * s2) + (e ? to_float(e[c]) : 0.0f);
        dx[c] = from_float<T>(o);
        if (dr) dr[c] = from_float<S>(o);
    }
    if (threadIdx.x == 0 && p.ws) {
        ((f32x2*)p.ws)[id] = f32x2{mean, rstd};
    }
}

size_t stats_bytes(const AddNormProblem& p) { return ((size_t)p.B * p.T * 8 + 255) & ~size_t(255); }

template <typename T, typename S>
__global__ __launch_bounds__(256) void addnorm_columns_kernel(AddNormProblem p, float* part)
{
    const int nb = (p.C + 255) / 256;
    const int64_t run = block_id() / nb, rows = (int64_t)p.B * p.T;
    const int c = (int)(block_id() % nb) * 256 + threadIdx.x;
    if (c >= p.C || run * kRun >= rows) return;
    float dw = 0.0f, db = 0.0f;
    for (int64_t i = run * kRun; i < min(rows, (run + 1) * kRun); ++i) {
        const int64_t b = i / p.T, t = i % p.T;
        const f32x2 st = ((const f32x2*)p.ws)[i];
        const float g = to_float(((const T*)p.dy.p)[b * p.dy.batch + t * p.dy.row + c]);
        dw += g * ((to_float(((const S*)p.total.p)[b * p.total.batch + t * p.total.row + c]) - st[0]) * st[1]);
        db += g;
    }
    part[run * 2 * p.C + c] = dw;
    part[run * 2 * p.C + p.C + c] = db;
}

__global__ __launch_bounds__(1024) void addnorm_params_kernel(AddNormProblem p, const float* part, int64_t parts)
{
    __shared__ float red[16][64];
    const int64_t W = p.C, i = (int64_t)blockIdx.x * 64 + threadIdx.x;
    const float s = part_sum(part, parts, 2 * W, 2 * W, blockIdx.x, red);
    if (threadIdx.x >= 64 || i >= 2 * W) return;
    if (i < W) {
        if (p.dweight) p.dweight[i] = s;
    } else if (p.dbias) {
        p.dbias[i - W] = s;
    }
}

template <typename T, typename S>
hipError_t bwd_t(const AddNormProblem& p, hipStream_t stream)
{
    addnorm_bwd_kernel<T, S><<<grid_of((int64_t)p.B * p.T), 256, 0, stream>>>(p);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || (!p.dweight && !p.dbias)) return e;
    float* part = (float*)(p.ws + stats_bytes(p));
    const int64_t runs = ((int64_t)p.B * p.T + kRun - 1) / kRun;
    addnorm_columns_kernel<T, S><<<grid_of(runs * ((p.C + 255) / 256)), 256, 0, stream>>>(p, part);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    addnorm_params_kernel<<<(unsigned)((2 * (int64_t)p.C + 63) / 64), 1024, 0, stream>>>(p, part, runs);
    return hipGetLastError();
}

}  // namespace

size_t addnorm_bwd_workspace(const AddNormProblem& p)
{
    const int64_t runs = ((int64_t)p.B * p.T + kRun - 1) / kRun;
    return stats_bytes(p) + (size_t)runs * 2 * p.C * sizeof(float);
}

hipError_t launch_addnorm_bwd(const AddNormProblem& p, hipStream_t stream)
{
    if (!p.bf16) return bwd_t<float, float>(p, stream);
    return p.sum_fp32 ? bwd_t<bf16, float>(p, stream) : bwd_t<bf16, bf16>(p, stream);
}

}  // namespace tfla
