// scan_impl.hpp -- what the selective scan's forward and backward kernels
// share.
//
//   delta_t = softplus(dt_t + dt_bias),   a_t = exp(delta_t A[c,n])
//   h_t = a_t h_{t-1} + delta_t x_t B_t[n],   y_t = sum_n C_t[n] h_t + skip x_t
//
// Lanes are channels: a workgroup owns 64 channels of one group and one
// sequence, and its W waves split the N states, kStates to a wave, held in
// fp32 registers along the whole walk.  B_t and C_t are then the same for
// every lane of a wave: they are read by scalar loads and enter the products
// as scalar operands, at no cost in vector registers or vector loads.  What
// belongs to a channel and a step alone (softplus, the gate, their gradients)
// is done once, by the wave that owns the step in the tile, and handed to the
// others through LDS.
#pragma once

#include "blocks.hpp"
#include "gfx950.hpp"

namespace tfla {
namespace scan {

constexpr int kStates = 4;    // states of a wave

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// kStates values of B or C at a wave-uniform address (scalar loads; the data
// is read-only during the launch).
template <typename T> struct Uniform4;
template <> struct Uniform4<bf16> {
    float v[4];
    __device__ __forceinline__ void load(const bf16* p)
    {
        typedef const u32x2 __attribute__((address_space(4))) cvec;
        const u32x2 r = *(cvec*)(uintptr_t)p;
        v[0] = __builtin_bit_cast(float, r[0] << 16);
        v[1] = __builtin_bit_cast(float, r[0] & 0xffff0000u);
        v[2] = __builtin_bit_cast(float, r[1] << 16);
        v[3] = __builtin_bit_cast(float, r[1] & 0xffff0000u);
    }
};
template <> struct Uniform4<float> {
    float v[4];
    __device__ __forceinline__ void load(const float* p)
    {
        typedef const f32x4 __attribute__((address_space(4))) cvec;
        const f32x4 r = *(cvec*)(uintptr_t)p;
        v[0] = r[0];
        v[1] = r[1];
        v[2] = r[2];
        v[3] = r[3];
    }
};

__device__ __forceinline__ int clamp_len(const int* lengths, int b, int T)
{
    return lengths ? min(max(lengths[b], 0), T) : T;
}

__device__ __forceinline__ float sigmoid_f(float u) { return 1.0f / (1.0f + expf(-u)); }

// softplus(u) = max(u, 0) + log1p(e^{-|u|})
__device__ __forceinline__ float softplus_f(float u) { return fmaxf(u, 0.0f) + log1pf(expf(-fabsf(u))); }

// Where a workgroup stands: sequence, channels, states.
struct Place {
    int b, g, cb, lane, wave, c;   // c: the lane's channel (clamped to a valid one when !live)
    bool live;
};

__device__ __forceinline__ Place place(const ScanProblem& p)
{
    Place q;
    const int per = p.D / p.G;
    const int ncb = (per + 63) / 64;
    int blk = blockIdx.x;
    q.cb = blk % ncb;
    blk /= ncb;
    q.g = blk % p.G;
    q.b = blk / p.G;
    q.lane = threadIdx.x & 63;
    q.wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int i = q.cb * 64 + q.lane;
    q.live = i < per;
    q.c = q.g * per + min(i, per - 1);
    return q;
}

}  // namespace scan
}  // namespace tfla
