// norm_impl.hpp -- what the group norm's kernels share.
//
//   xh = (x - mean) rstd,  u = xh w + bias,  y = act(u) or u act(gate)
//   v = du w,  dx = rstd (v - mean(v) - xh mean(v xh))
//
// A set is what shares one mean: the C channels of a token's group, or the
// T x C values of a sequence's group.
#pragma once

#include "act.hpp"
#include "blocks.hpp"
#include "sums.hpp"

namespace tfla {
namespace norm {

// VEC elements as they lie in memory
template <typename T, int VEC> struct Pack {
    typedef T vec __attribute__((ext_vector_type(VEC)));
    vec v;
    __device__ __forceinline__ void load(const T* p) { v = *(const vec*)p; }
    __device__ __forceinline__ void store(T* p) const { *(vec*)p = v; }
    template <bool NT> __device__ __forceinline__ void load_t(const T* p)
    {
        if (NT) v = __builtin_nontemporal_load((const vec*)p);
        else load(p);
    }
    template <bool NT> __device__ __forceinline__ void store_t(T* p) const
    {
        if (NT) __builtin_nontemporal_store(v, (vec*)p);
        else store(p);
    }
    __device__ __forceinline__ float get(int i) const { return to_float((T)v[i]); }
    __device__ __forceinline__ void set(int i, float x) { v[i] = from_float<T>(x); }
};
template <typename T> struct Pack<T, 1> {
    T v;
    __device__ __forceinline__ void load(const T* p) { v = *p; }
    __device__ __forceinline__ void store(T* p) const { *p = v; }
    template <bool> __device__ __forceinline__ void load_t(const T* p) { load(p); }
    template <bool> __device__ __forceinline__ void store_t(T* p) const { store(p); }
    __device__ __forceinline__ float get(int) const { return to_float(v); }
    __device__ __forceinline__ void set(int, float x) { v = from_float<T>(x); }
};

// ACTIVE: SiLU (silu) or sigmoid; else the identity.
template <typename T, bool ACTIVE> __device__ __forceinline__ float act_f(float u, bool silu)
{
    if (!ACTIVE) return u;
    const float s = sigmoid_t<T>(u);
    return silu ? u * s : s;
}
template <typename T, bool ACTIVE> __device__ __forceinline__ void act_both(float u, bool silu, float* f, float* slope)
{
    if (!ACTIVE) {
        *f = u;
        *slope = 1.0f;
        return;
    }
    const float s = sigmoid_t<T>(u), us = u * s;
    *f = silu ? us : s;
    *slope = silu ? s + us * (1.0f - s) : s * (1.0f - s);
}

__device__ __forceinline__ int64_t at(const Heads& h, int b, int t, int g, int c)
{
    return b * h.batch + t * h.row + g * h.group + c;
}

template <int CTRL> __device__ __forceinline__ float dpp_add(float v)
{
    return v + __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), CTRL, 0xf, 0xf, true));
}
__device__ __forceinline__ float fold16(float v)
{
    const unsigned u = __builtin_bit_cast(unsigned, v);
    const auto r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    const unsigned lo = r[0], hi = r[1];
    return __builtin_bit_cast(float, lo) + __builtin_bit_cast(float, hi);
}
__device__ __forceinline__ float fold32(float v)
{
    const unsigned u = __builtin_bit_cast(unsigned, v);
    const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    const unsigned lo = r[0], hi = r[1];
    return __builtin_bit_cast(float, lo) + __builtin_bit_cast(float, hi);
}

// Sum over the aligned group of L lanes a lane is in, in each of them (L a power of two, uniform).
__device__ __forceinline__ float lane_sum(float v, int L)
{
    if (L > 1) v = dpp_add<0xb1>(v);    // lane ^ 1
    if (L > 2) v = dpp_add<0x4e>(v);    // lane ^ 2
    if (L > 4) v = dpp_add<0x141>(v);   // lane ^ 7
    if (L > 8) v = dpp_add<0x140>(v);   // lane ^ 15
    if (L > 16) v = fold16(v);
    if (L > 32) v = fold32(v);
    return v;
}

// How the rows [B,T,G] of token sets fall to waves.  L lanes hold a row, one
// vector each, so a wave holds 64 / L: consecutive groups of a token where
// those divide G (`by_group`), else consecutive tokens of a group.  A row of
// more than 64 vectors falls to a whole workgroup (L = 128 or 256 threads), up
// to 4 vectors a lane.  A wave (workgroup) keeps its groups and walks `per` token steps, so
// its weights stay in registers.  Rows are counted in 32 bits: a division
// by T in 64 costs more than a row of 512 channels.
struct TokenMap {
    int L, slots, ng, step;     // rows of a wave; sets of groups; tokens of a step
    bool by_group, block;
    int nv;                     // vectors of a row
    unsigned tokens, per, chunks;
};

inline TokenMap token_map(const NormProblem& p, int vec, int64_t waves, int most)
{
    TokenMap m;
    m.nv = p.C / vec;
    m.block = m.nv > 64;
    m.L = !m.block ? 1 : m.nv > 128 ? 256 : 128;
    while (m.L < 64 && m.L < m.nv) m.L *= 2;
    m.slots = m.block ? 1 : 64 / m.L;
    m.by_group = p.G % m.slots == 0;
    m.ng = m.by_group ? p.G / m.slots : p.G;
    m.step = m.by_group ? 1 : m.slots;
    m.tokens = (unsigned)p.B * (unsigned)p.T;
    const int64_t steps = ((int64_t)m.tokens + m.step - 1) / m.step;
    int64_t per = steps * m.ng / (m.block ? waves * 64 / m.L : waves);
    if (per < 1) per = 1;
    if (per > most) per = most;
    m.per = (unsigned)per;
    m.chunks = (unsigned)((steps + per - 1) / per);
    return m;
}

inline bool fits(const Heads& h, const NormProblem& p, size_t bytes)
{
    const size_t e = p.bf16 ? 2 : 4;
    return !h.p || ((uintptr_t)h.p % bytes == 0 && (p.B == 1 || h.batch * e % bytes == 0) &&
                    (p.T == 1 || h.row * e % bytes == 0) && (p.G == 1 || h.group * e % bytes == 0));
}

// Elements of a vector: 16 bytes where channels, addresses and strides allow, else 1 (gated [4,8192,8,512] with rows
// an element longer, aligned rows after the comma: bf16 264, 160 us, backward 365, 272; fp32 352, 342 and 593, 570).
inline int vec_of(const NormProblem& p, bool bwd)
{
    const int v = p.bf16 ? 8 : 4;
    bool ok = p.C % v == 0 && fits(p.x, p, 16) && fits(p.gate, p, 16);
    if (bwd) ok = ok && fits(p.dy, p, 16) && fits(p.dx, p, 16) && fits(p.dgate, p, 16);
    else ok = ok && fits(p.y, p, 16);
    return ok ? v : 1;
}

// Whether a call moves far more than the last-level cache holds (256 MB): its loads (and, backward, its stores) are
// then non-temporal.  Gated norm of [4,8192,8,512] bf16, 807 MB: 186 us without, 171 so; backward of
// [8,4096,32,128], 1.35 GB: 292 and 278; but gated norm of [1,2000,8,512], 49 MB, 20.2 and 22.2.
inline bool streams(const NormProblem& p, int tensors)
{
    return (int64_t)p.B * p.T * p.G * p.C * (p.bf16 ? 2 : 4) * tensors >= (int64_t(512) << 20);
}

// Vectors that a lane holds of a row (rounded to what is built), or 0: too many.
inline int lane_vectors(const TokenMap& m)
{
    const int v = (m.nv + m.L - 1) / m.L;
    return v <= 1 ? 1 : v <= 2 ? 2 : v <= 4 ? 4 : 0;
}

// Sum over the lanes of a row; for a workgroup's row through LDS (two barriers; `red` of 4 floats).
template <bool BLOCK> __device__ __forceinline__ float row_sum(float v, int L, float* red)
{
    if (!BLOCK) return lane_sum(v, L);
    v = lane_sum(v, 64);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    const float s = red[0] + red[1];
    return L > 128 ? s + (red[2] + red[3]) : s;
}

// Sequence sets (norm_seq.hip)
hipError_t launch_seq_fwd(const NormProblem& p, hipStream_t stream);
hipError_t launch_seq_bwd(const NormProblem& p, hipStream_t stream);
size_t seq_workspace(const NormProblem& p);
size_t seq_bwd_workspace(const NormProblem& p);

}  // namespace norm
}  // namespace tfla
