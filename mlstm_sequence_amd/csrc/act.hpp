// act.hpp -- exponentials, activations and their slopes for the operators
// around the recurrences, on the transcendental unit (v_exp_f32, v_log_f32,
// v_rcp_f32: 1 ulp each).
#pragma once

#include "gfx950.hpp"

namespace tfla {

// e^x.  The product x log2(e) is carried in two parts, so the result keeps
// its relative accuracy (about 3 half-steps) at any size of x; without the
// low part the error would grow with |x|.  Infinities and NaN go through.
__device__ __forceinline__ float exp_f(float x)
{
    constexpr float kLn2 = 0.6931471805599453f;
    constexpr float kLog2eLow = 1.9259629911266175e-08f;   // log2(e) - (float)log2(e)
    const float p = x * kLog2e;
    float lo = fmaf(x, kLog2eLow, fmaf(x, kLog2e, -p));
    lo = fabsf(p) < 256.0f ? lo * kLn2 : 0.0f;
    const float e = exp2_fast(p);
    return fmaf(e, lo, e);
}

__device__ __forceinline__ float sigmoid_f(float u) { return __builtin_amdgcn_rcpf(1.0f + exp_f(-u)); }

// softplus(u) = max(u, 0) + log1p(e^{-|u|}); log1p as in log_sigmoid_fast.
__device__ __forceinline__ float softplus_f(float u)
{
    constexpr float kLn2 = 0.6931471805599453f;
    const float y = exp_f(-fabsf(u));
    const float v = 1.0f + y;
    const float l = v == 1.0f ? y : __builtin_amdgcn_logf(v) * kLn2 * (y * __builtin_amdgcn_rcpf(v - 1.0f));
    return fmaxf(u, 0.0f) + l;
}

}  // namespace tfla
