// act.hpp -- exponentials, activations and their slopes for the operators
// around the recurrences, on the transcendental unit (v_exp_f32, v_log_f32,
// v_rcp_f32: 1 ulp each).
#pragma once

#include "gfx950.hpp"

namespace tfla {

// e^x.  The product x log2(e) is carried in two parts, so every normal
// result keeps its relative accuracy (about 3 half-steps); without the low
// part the error would grow with |x|.  The low part is used where 2^p is
// finite and not 0 only: an infinity times it, or times 0, would be NaN.
// Beyond stand infinity (x above 88.7), 0 and NaN as they come.
__device__ __forceinline__ float exp_f(float x)
{
    constexpr float kLn2 = 0.6931471805599453f;
    constexpr float kLog2eLow = 1.9259629911266175e-08f;   // log2(e) - (float)log2(e)
    const float p = x * kLog2e;
    const float lo = fmaf(x, kLog2eLow, fmaf(x, kLog2e, -p)) * kLn2;
    const float e = exp2_fast(p);
    return fabsf(p) < 128.0f ? fmaf(e, lo, e) : e;
}

__device__ __forceinline__ float sigmoid_f(float u) { return __builtin_amdgcn_rcpf(1.0f + exp_f(-u)); }

// softplus(u) = max(u, 0) + log1p(y), y = e^{-|u|}.  With v = 1 + y rounded,
// log1p(y) = log(v) + (y - (v - 1)) / v: the last term is what rounding took
// from y, at most half a step of v, and leaving out its division by v changes
// the sum by less than half a step of y.
__device__ __forceinline__ float softplus_of(float u, float y)
{
    constexpr float kLn2 = 0.6931471805599453f;
    const float v = 1.0f + y;
    // the median of u, 0 and infinity is max(u, 0) in one instruction; a NaN comes back through y
    return __builtin_amdgcn_fmed3f(u, 0.0f, __builtin_inff()) + fmaf(__builtin_amdgcn_logf(v), kLn2, y - (v - 1.0f));
}
__device__ __forceinline__ float softplus_f(float u) { return softplus_of(u, exp_f(-fabsf(u))); }

// The same for bf16 data, whose own half step (2^-8) is far above the
// exponential's error of |x| 2^-24 without the product's low part.  fp32
// results of bf16 data (weights' gradients, states) carry that error too,
// below what the data's half steps leave in them.
__device__ __forceinline__ float sigmoid_fast(float u)
{
    return __builtin_amdgcn_rcpf(1.0f + exp2_fast(u * -kLog2e));
}
__device__ __forceinline__ float softplus_fast(float u) { return softplus_of(u, exp2_fast(fabsf(u) * -kLog2e)); }

template <typename T> __device__ __forceinline__ float sigmoid_t(float u) { return sizeof(T) == 2 ? sigmoid_fast(u) : sigmoid_f(u); }
template <typename T> __device__ __forceinline__ float softplus_t(float u) { return sizeof(T) == 2 ? softplus_fast(u) : softplus_f(u); }

}  // namespace tfla
