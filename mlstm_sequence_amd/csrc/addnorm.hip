// addnorm.hip -- residual sum with a layer or RMS norm, forward.
//
//   t = x + residual,  y = (t - mean) rstd weight + bias   (RMS: mean taken as 0)
#include "gfx950.hpp"

#include "norm_impl.hpp"

namespace tfla {
namespace {

// A workgroup to a row.  T: activations, S: the stream.
template <typename T, typename S>
__global__ __launch_bounds__(256) void addnorm_fwd_kernel(AddNormProblem p)
{
    __shared__ float red[4];
    const int64_t id = block_id();
    if (id >= (int64_t)p.B * p.T) return;
    const int64_t b = id / p.T, t = id % p.T;
    const T* x = (const T*)p.x.p + b * p.x.batch + t * p.x.row;
    const S* r = p.residual.p ? (const S*)p.residual.p + b * p.residual.batch + t * p.residual.row : nullptr;
    T* y = (T*)p.y.p + b * p.y.batch + t * p.y.row;
    S* o = p.total.p ? (S*)p.total.p + b * p.total.batch + t * p.total.row : nullptr;
    auto sum = [&](float v) { return norm::row_sum<true>(v, 256, red); };
    auto at = [&](int c) { return to_float(x[c]) + (r ? to_float(r[c]) : 0.0f); };
    float s = 0.0f, q = 0.0f;
    for (int c = threadIdx.x; c < p.C; c += 256) s += at(c);
    const float mean = p.rms ? 0.0f : sum(s) / (float)p.C;
    for (int c = threadIdx.x; c < p.C; c += 256) {
        const float d = at(c) - mean;
        q += d * d;
    }
    const float rstd = 1.0f / sqrtf(sum(q) / (float)p.C + p.eps);
    for (int c = threadIdx.x; c < p.C; c += 256) {
        const float v = at(c);
        y[c] = from_float<T>((v - mean) * rstd * (p.weight ? p.weight[c] : 1.0f) + (p.bias ? p.bias[c] : 0.0f));
        if (o) o[c] = from_float<S>(v);   // last: it may be r
    }
}

}  // namespace

hipError_t launch_addnorm_fwd(const AddNormProblem& p, hipStream_t stream)
{
    const dim3 grid = grid_of((int64_t)p.B * p.T);
    if (!p.bf16) addnorm_fwd_kernel<float, float><<<grid, 256, 0, stream>>>(p);
    else if (p.sum_fp32) addnorm_fwd_kernel<bf16, float><<<grid, 256, 0, stream>>>(p);
    else addnorm_fwd_kernel<bf16, bf16><<<grid, 256, 0, stream>>>(p);
    return hipGetLastError();
}

}  // namespace tfla
