// addnorm.hip -- residual sum with a layer or RMS norm, forward.
//
//   t = x + residual,  y = (t - mean) rstd weight + bias   (RMS: mean taken as 0)
//
// Bound by memory: x and the stream are read once, the stream and y written
// once (addnorm_impl.hpp).  Mean and variance take two passes over registers.
#include "gfx950.hpp"

#include "addnorm_impl.hpp"

namespace tfla {
namespace {

using namespace addnorm;

// Workgroups at most, their rows in turn (bf16 [4, 4096, 4096] 107 us, a workgroup to each row 179; [2, 1024, 4096] 18.5 us,
// 2048 of them 23.4; [8, 4096, 256] with a stream of fp32 18.1 us, 512 of them 20.3), twice as many where a stream of fp32
// gives each eight rows that take all of it ([4, 4096, 4096]: 153 us, 1024 of them 157).
unsigned most_blocks(const AddNormProblem& p)
{
    return p.sum_fp32 && p.C >= 1024 && (int64_t)p.B * p.T >= 8 * 2048 ? 2048 : 1024;
}

// T: activations, S: the stream.  NV vectors a lane.
template <typename T, typename S, int NV, bool EDGE>
__global__ __launch_bounds__(1024) void addnorm_fwd_kernel(AddNormProblem p, RowMap m)
{
    constexpr int VEC = vec_of<T, S>();
    __shared__ float red[2][16][1];
    const int slot = threadIdx.x / m.L, lv = threadIdx.x - slot * m.L;
    const bool sum = p.residual.p != nullptr, shift = !p.rms;
    const Columns<VEC, NV, EDGE> cols(lv, m.L, m.nv, p.C);
    const int* c = cols.c;
    float w[NV][VEC], bs[NV][VEC];
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            w[k][v] = p.weight ? p.weight[c[k] + v] : 1.0f;
            bs[k][v] = p.bias ? p.bias[c[k] + v] : 0.0f;
        }
    const float inv = 1.0f / (float)p.C;
    Pack<T, VEC, EDGE, false> rx[NV];
    Pack<S, VEC, EDGE, false> rr[NV];
    auto fetch = [&](unsigned i) {                    // behind the last row: the last
        i = min(i, m.rows - 1);
        const int64_t b = i / (unsigned)p.T, t = i % (unsigned)p.T;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            rx[k].load((const T*)p.x.p + b * p.x.batch + t * p.x.row + c[k]);
            if (sum) rr[k].load((const S*)p.residual.p + b * p.residual.batch + t * p.residual.row + c[k]);
        }
    };
    const unsigned step = gridDim.x * m.slots, first = blockIdx.x * m.slots;
    fetch(first + slot);
    int turn = 0;
    for (unsigned i0 = first; i0 < m.rows; i0 += step) {
        const unsigned i = i0 + slot;
        float x[NV][VEC], s = 0.0f, q = 0.0f, mean = 0.0f;
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                x[k][v] = rx[k].get(v);
                if (sum) x[k][v] += rr[k].get(v);
            }
        fetch(i + step);
        if (shift) {
#pragma unroll
            for (int k = 0; k < NV; ++k)
#pragma unroll
                for (int v = 0; v < VEC; ++v) s += cols.counts(k, v) ? x[k][v] : 0.0f;
            row_sums<1>(&s, m.L, red, turn);
            turn ^= 1;
            mean = s * inv;
        }
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                const float d = x[k][v] - mean;
                q += cols.counts(k, v) ? d * d : 0.0f;
            }
        row_sums<1>(&q, m.L, red, turn);
        turn ^= 1;
        const float rstd = 1.0f / sqrtf(q * inv + p.eps);
        if (i >= m.rows) continue;
        const int64_t b = i / (unsigned)p.T, t = i % (unsigned)p.T;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            if (!cols.in[k]) continue;
            Pack<T, VEC, EDGE, false> o;
            Pack<S, VEC, EDGE, false> ot;
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                o.set(v, (x[k][v] - mean) * rstd * w[k][v] + bs[k][v]);
                ot.set(v, x[k][v]);
            }
            o.store((T*)p.y.p + b * p.y.batch + t * p.y.row + c[k]);
            if (sum) ot.store((S*)p.total.p + b * p.total.batch + t * p.total.row + c[k]);
        }
    }
}

// A workgroup to a row of any length, walked from memory.
template <typename T, typename S>
__global__ __launch_bounds__(256) void addnorm_fwd_long_kernel(AddNormProblem p)
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

template <typename T, typename S, bool EDGE>
hipError_t fwd_e(const AddNormProblem& p, hipStream_t stream)
{
    const RowMap m = row_map(p, most_vectors(p), most_blocks(p), false);
    const int v = (m.nv + m.L - 1) / m.L;
    if (v == 1) addnorm_fwd_kernel<T, S, 1, EDGE><<<m.blocks, m.threads, 0, stream>>>(p, m);
    else if (v == 2) addnorm_fwd_kernel<T, S, 2, EDGE><<<m.blocks, m.threads, 0, stream>>>(p, m);
    else if constexpr (most_vectors<T, S>() == 4) addnorm_fwd_kernel<T, S, 4, EDGE><<<m.blocks, m.threads, 0, stream>>>(p, m);
    return hipGetLastError();
}

template <typename T, typename S>
hipError_t fwd_t(const AddNormProblem& p, hipStream_t stream)
{
    if (in_registers(p))
        return edged(p, {&p.x, &p.residual, &p.y, &p.total}) ? fwd_e<T, S, true>(p, stream) : fwd_e<T, S, false>(p, stream);
    addnorm_fwd_long_kernel<T, S><<<grid_of((int64_t)p.B * p.T), 256, 0, stream>>>(p);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_addnorm_fwd(const AddNormProblem& p, hipStream_t stream)
{
    if (!p.bf16) return fwd_t<float, float>(p, stream);
    return p.sum_fp32 ? fwd_t<bf16, float>(p, stream) : fwd_t<bf16, bf16>(p, stream);
}

}  // namespace tfla
