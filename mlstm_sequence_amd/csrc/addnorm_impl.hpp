// addnorm_impl.hpp -- what the residual sum's kernels share.
//
// A row lives in the registers of L lanes, a few vectors each: part of a wave,
// a wave, or up to 16 waves.  A vector is 16 bytes of the wider type, so that
// each load of a wave covers whole lines (bf16 with a stream of fp32, [4, 4096,
// 4096] forward: 153 us; eight elements, 32 bytes of the stream, 164).  Where
// channels, addresses or strides leave them off 16 bytes, vectors are loaded as
// they lie and a row's last one is moved back to end with the row: C=1001, 32768
// rows of bf16 54 us forward and 63 backward, one element to a lane's load 93
// and 324.  Rows are walked with the next one's loads under way, so the weights
// stay in registers.
#pragma once

#include "norm_impl.hpp"

namespace tfla {
namespace addnorm {

// VEC elements as they lie in memory.  EDGE: wherever they lie; NT: loads past the caches.
template <typename T, int VEC, bool EDGE, bool NT> struct Pack {
    typedef T vec __attribute__((ext_vector_type(VEC)));
    typedef vec mem __attribute__((aligned(EDGE ? sizeof(T) : sizeof(vec))));
    vec v;
    __device__ __forceinline__ void load(const T* p)
    {
        if (NT) v = __builtin_nontemporal_load((const mem*)p);
        else v = *(const mem*)p;
    }
    __device__ __forceinline__ void store(T* p) const { *(mem*)p = v; }
    __device__ __forceinline__ float get(int i) const { return to_float((T)v[i]); }
    __device__ __forceinline__ void set(int i, float x) { v[i] = from_float<T>(x); }
};

// The first column of a row's vector.  EDGE: the last vector ends with the row; what it shares with the one before it
// is counted there, and written by both, the same.
template <int VEC, bool EDGE> __device__ __forceinline__ int column(int vector, int C)
{
    return EDGE ? min(vector * VEC, C - VEC) : vector * VEC;
}

// A lane's vectors.
template <int VEC, int NV, bool EDGE> struct Columns {
    int c[NV];          // first columns
    bool in[NV];        // whether the vector is one of the row
    int shared[NV];     // EDGE: elements that another vector counts, all where there is none
    __device__ __forceinline__ Columns(int lane, int L, int nv, int C)
    {
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int i = lane + k * L;
            in[k] = i < nv;
            c[k] = column<VEC, EDGE>(min(i, nv - 1), C);
            shared[k] = in[k] ? i * VEC - c[k] : VEC;
        }
    }
    __device__ __forceinline__ bool counts(int k, int v) const { return EDGE ? v >= shared[k] : in[k]; }
};

// L lanes to a row, slots rows to a workgroup of `threads`, `blocks` workgroups taking rows in turn.
struct RowMap {
    int L, nv, slots, threads;
    unsigned rows, blocks;
    bool only = false;   // backward: the one workgroup's sums are the weights' gradients
};

// Vectors a lane holds at most: 16 values of either type, 8 of fp32 alone.
template <typename T, typename S> constexpr int most_vectors() { return sizeof(T) < sizeof(S) ? 4 : 2; }
inline int most_vectors(const AddNormProblem& p) { return p.sum_fp32 ? 4 : 2; }
// Elements of a vector: 16 bytes of the wider type.
template <typename T, typename S> constexpr int vec_of() { return 16 / (sizeof(T) > sizeof(S) ? sizeof(T) : sizeof(S)); }
inline int vec_of(const AddNormProblem& p) { return p.bf16 && !p.sum_fp32 ? 8 : 4; }
// Vectors of a row, and whether it has one and fits in the registers of 16 waves; longer rows are read two and three
// times (bf16 [2, 4096, 16384], which still fits, backward at 2.2 TB/s, as the registers of 16 waves spill).
inline int vectors(const AddNormProblem& p) { return (p.C + vec_of(p) - 1) / vec_of(p); }
inline bool in_registers(const AddNormProblem& p) { return p.C >= vec_of(p) && vectors(p) <= 1024 * most_vectors(p); }

// most: vectors of a lane where a row takes more than a wave.  tight: beyond two waves a row takes as many as it needs,
// not a power of two (backward [4, 4096, 2560] with a stream of fp32 138 us, 198 by powers; forward equal to 4 % either
// way, so it keeps the powers).
inline RowMap row_map(const AddNormProblem& p, int most, unsigned most_blocks, bool tight)
{
    RowMap m;
    m.nv = vectors(p);
    m.L = 1;
    while (m.L < 64 && m.L < m.nv) m.L *= 2;
    while (m.L < 1024 && most * m.L < m.nv) m.L *= 2;
    if (tight && m.L > 128) m.L = (m.nv + 64 * most - 1) / (64 * most) * 64;
    m.threads = m.L > 128 ? m.L : 256;
    m.slots = m.threads / m.L;
    m.rows = (unsigned)p.B * (unsigned)p.T;
    const unsigned need = (m.rows + m.slots - 1) / m.slots;
    m.blocks = need < most_blocks ? need : most_blocks;
    return m;
}

// Whether channels, addresses or strides leave vectors off their alignment.
inline bool edged(const AddNormProblem& p, std::initializer_list<const Rows*> rows)
{
    const int v = vec_of(p);
    bool ok = p.C % v == 0;
    for (const Rows* r : rows)
        ok = ok && (!r->p || ((uintptr_t)r->p % 16 == 0 && (p.B == 1 || r->batch % v == 0) && (p.T == 1 || r->row % v == 0)));
    return !ok;
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
