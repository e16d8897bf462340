// addnorm_impl.hpp -- what the residual sum's kernels share.
//
// A row lives in the registers of L lanes, a few vectors each: part of a wave,
// a wave, or up to 16 waves.  A vector is 16 bytes of the wider type, so that
// each load of a wave covers whole lines.  Rows are walked
// with the next one's loads under way, so the weights stay in registers.
#pragma once

#include "norm_impl.hpp"

namespace tfla {
namespace addnorm {

// VEC elements as they lie in memory; NT: loads past the caches
template <typename T, int VEC, bool NT> struct Pack {
    typedef T vec __attribute__((ext_vector_type(VEC)));
    vec v;
    __device__ __forceinline__ void load(const T* p)
    {
        if (NT) v = __builtin_nontemporal_load((const vec*)p);
        else v = *(const vec*)p;
    }
    __device__ __forceinline__ void store(T* p) const { *(vec*)p = v; }
    __device__ __forceinline__ float get(int i) const { return to_float((T)v[i]); }
    __device__ __forceinline__ void set(int i, float x) { v[i] = from_float<T>(x); }
};
template <typename T, bool NT> struct Pack<T, 1, NT> {
    T v;
    __device__ __forceinline__ void load(const T* p) { v = *p; }
    __device__ __forceinline__ void store(T* p) const { *p = v; }
    __device__ __forceinline__ float get(int) const { return to_float(v); }
    __device__ __forceinline__ void set(int, float x) { v = from_float<T>(x); }
};

// L lanes to a row, slots rows to a workgroup of `threads`, `blocks` workgroups taking rows in turn.
struct RowMap {
    int L, nv, slots, threads;
    unsigned rows, blocks;
};

// Vectors a lane holds at most: 16 values of either type.
template <typename T, typename S, int VEC> constexpr int most_vectors() { return sizeof(T) < sizeof(S) && VEC > 1 ? 4 : 2; }
inline int most_vectors(const AddNormProblem& p, int vec) { return p.sum_fp32 && vec > 1 ? 4 : 2; }
// Whether a row fits in the registers of 16 waves.
inline bool in_registers(const AddNormProblem& p, int vec) { return p.C / vec <= 1024 * most_vectors(p, vec); }

// most: vectors of a lane where a row takes more than a wave.
inline RowMap row_map(const AddNormProblem& p, int vec, int most, unsigned most_blocks)
{
    RowMap m;
    m.nv = p.C / vec;
    m.L = 1;
    while (m.L < 64 && m.L < m.nv) m.L *= 2;
    while (m.L < 1024 && most * m.L < m.nv) m.L *= 2;
    m.threads = m.L > 256 ? m.L : 256;
    m.slots = m.threads / m.L;
    m.rows = (unsigned)p.B * (unsigned)p.T;
    const unsigned need = (m.rows + m.slots - 1) / m.slots;
    m.blocks = need < most_blocks ? need : most_blocks;
    return m;
}

// Elements of a vector: 16 bytes of the wider type where channels, addresses and strides allow, else 1.
inline int vec_of(const AddNormProblem& p, std::initializer_list<const Rows*> rows)
{
    const int v = p.bf16 && !p.sum_fp32 ? 8 : 4;
    bool ok = p.C % v == 0;
    for (const Rows* r : rows)
        ok = ok && (!r->p || ((uintptr_t)r->p % 16 == 0 && (p.B == 1 || r->batch % v == 0) && (p.T == 1 || r->row % v == 0)));
    return ok ? v : 1;
}

// Sums of N values over the L lanes of a row, in each of them.  Rows of several waves meet in LDS, in two halves of
// `red` used in turn, so one barrier a sum does.
template <int N> __device__ __forceinline__ void row_sums(float* v, int L, float (*red)[16][N], int turn)
{
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = norm::lane_sum(v[i], L < 64 ? L : 64);
    if (L <= 64) return;
    const int wave = threadIdx.x >> 6, per = L >> 6, first = wave / per * per;
    if ((threadIdx.x & 63) == 0)
#pragma unroll
        for (int i = 0; i < N; ++i) red[turn][wave][i] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = 0.0f;
    for (int w = 0; w < per; ++w)
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += red[turn][first + w][i];
}

}  // namespace addnorm
}  // namespace tfla
