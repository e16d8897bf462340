// diag_impl.hpp -- gates of the gated linear recurrence of channels.
//
//   h_t = f_t h_{t-1} + i_t x_t
//   g_t = dy_t + f_{t+1} g_{t+1},  dx = i g,  df = h_{t-1} g,  di = x g
//
//   coupled   f = s(u), i = 1 - f:         du = (df - di) f i
//   sigmoid   f = s(u), i = s(v):          du = df f (1 - f),  dv = di i (1 - i)
//   decay     f = e^{-w}, w = decay s(u), i = m s(v), m = sqrt(1 - f^2):
//             dw = di s(v) f^2 / m - df f,  du = dw w (1 - s(u)),  ddecay = sum dw s(u),  dv = di i (1 - s(v))
#pragma once

#include "act.hpp"
#include "blocks.hpp"

namespace tfla {
namespace diag {

constexpr int kChunk = 128;   // TFLA_DIAG_CHUNK

__device__ __forceinline__ int clamp_len(const int* lengths, int b, int T)
{
    return lengths ? min(max(lengths[b], 0), T) : T;
}

template <typename T> __device__ __forceinline__ float exp_t(float x) { return sizeof(T) == 2 ? exp2_fast(x * kLog2e) : exp_f(x); }

// 1 - e^{-2w}: the series where the difference would cancel (w below 1/4; the first term left out is 2^-26 of it).
__device__ __forceinline__ float one_minus_square(float w, float f)
{
    const float z = 2.0f * w;
    float s = fmaf(z, -2.4801587e-5f, 1.9841270e-4f);
    s = fmaf(z, -s, 1.3888889e-3f);
    s = fmaf(z, -s, 8.3333333e-3f);
    s = fmaf(z, -s, 4.1666667e-2f);
    s = fmaf(z, -s, 1.6666667e-1f);
    s = fmaf(z, -s, 0.5f);
    s = fmaf(z, -s, 1.0f);
    return z < 0.5f ? z * s : fmaf(-f, f, 1.0f);
}

// The gates of a step; r = s(u), s = s(v) and m where the kind has them.
struct Gate {
    float f, i, r, s, m;
};

template <typename T, int KIND> __device__ __forceinline__ Gate gate_of(float u, float v, float decay)
{
    Gate g;
    if (KIND == kCoupled) {
        const float e = exp_t<T>(-u);
        g.f = __builtin_amdgcn_rcpf(1.0f + e);
        g.i = e == __builtin_inff() ? 1.0f : e * g.f;   // 1 - f without its cancellation
    } else {
        g.s = sigmoid_t<T>(v);
        g.r = sigmoid_t<T>(u);
        if (KIND == kSigmoid) {
            g.f = g.r;
            g.i = g.s;
        } else {
            const float w = decay * g.r;
            g.f = exp_t<T>(-w);
            g.m = __builtin_amdgcn_sqrtf(one_minus_square(w, g.f));
            g.i = g.m * g.s;
        }
    }
    return g;
}

struct GateGrads {
    float dx, du, dv, dd;
};

// Gradients of a step from its gates, x, the state before it and g.
template <int KIND> __device__ __forceinline__ GateGrads grads_of(const Gate& k, float x, float before, float g, float decay)
{
    GateGrads o;
    o.dx = k.i * g;
    const float df = before * g, di = x * g;
    o.dv = o.dd = 0.0f;
    if (KIND == kCoupled) {
        o.du = (df - di) * (k.f * k.i);
    } else if (KIND == kSigmoid) {
        o.du = df * (k.f * (1.0f - k.f));
        o.dv = di * (k.i * (1.0f - k.i));
    } else {
        const float dm = k.m > 0.0f ? k.f * k.f * __builtin_amdgcn_rcpf(k.m) : 0.0f;
        const float dw = di * k.s * dm - df * k.f;
        o.dd = dw * k.r;
        o.du = o.dd * decay * (1.0f - k.r);
        o.dv = di * k.i * (1.0f - k.s);
    }
    return o;
}

}  // namespace diag
}  // namespace tfla
