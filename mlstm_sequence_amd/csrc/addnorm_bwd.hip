// addnorm_bwd.hip -- residual sum with a layer or RMS norm, backward.
//
//   d = t - mean,  v = dy weight
//   dt = rstd (v - mean(v) - d rstd^2 mean(v d)) + dtotal,  dweight = sum dy d rstd,  dbias = sum dy
//
// The layout of the forward pass (addnorm_impl.hpp), the statistics formed
// again: two sums over a row, mean(t) and then three together.  The weights'
// gradients add up in registers over the rows that a workgroup takes and
// leave it once, to be added over the workgroups in a fixed order.  Bound by
// memory: the stream, its gradient and dy are read once, dt written once.
// [8, 4096, 4096] of bf16: 1.07 GB in 213 us (5.0 TB/s, as a copy).
#include "gfx950.hpp"

#include <algorithm>

#include "addnorm_impl.hpp"
#include "sums.hpp"

namespace tfla {
namespace {

using namespace addnorm;

// How the rows fall to workgroups, and the parts of the weights' gradients, which each writes once.
//
// bf16 rows of 512 to 1024 vectors take one vector a lane ([4, 4096, 5120] 188 us, two 218; [4, 4096, 8192] 226 and 253),
// not fp32 ones ([4, 4096, 2560]: 176 and 124) nor those of both types ([4, 4096, 4096]: 215, four 208).
//
// At most as many workgroups as the chip holds, by the registers of their variant: beyond 256 lanes to a row one on a CU,
// since a CU has 16 waves of bf16 (107 registers), whose rows take nine or more, and eight of both types (198), whose rows
// take five or more; a second or third for each CU only comes after the first and leaves sums of its own (bf16 [4, 4096,
// 5120]: 188 us, 198, 208).  With fp32 alone two up to 384 ([4, 4096, 2560]: 124 us, one 133; [4, 4096, 4096] 193 and 177);
// below three of bf16 or of a vector a lane ([4, 4096, 2560]: 90 us, two 104, four 112) and two else ([4, 4096, 2048] with
// a stream of fp32 96 us, three 113).  One on each CU, and more only where each has eight
// rows (bf16 [2, 1024, 8192] 49 us, twice as many 65).
//
// Up to eight rows, two for each that a workgroup holds, go to one, whose sums are the gradients: no workspace, no
// second launch (bf16 [1, 8, 1024] from Python 10.2 us, else 14.1; eight for each, [1, 8, 4096], 21 and 14.2).
RowMap map_of(const AddNormProblem& p)
{
    const int nv = vectors(p);
    const bool half = p.bf16 && !p.sum_fp32;
    RowMap m = row_map(p, half && nv > 512 && nv <= 1024 ? 1 : most_vectors(p), ~0u, true);
    const unsigned wide = !p.bf16 && m.L <= 384 ? 512 : 256;
    const unsigned cap = m.threads > 256 ? wide : half || nv <= m.L ? 768 : 512;
    m.only = m.rows <= (unsigned)std::min(8, 2 * m.slots);
    m.blocks = m.only ? 1 : std::min(m.blocks, std::min(cap, std::max(m.rows / 8, 256u)));
    return m;
}

// Whether a call moves more than the last-level cache holds (256 MB): its loads then go past it ([8, 4096, 4096] of bf16
// 209 us, through it 221; [1, 2048, 4096], 67 MB, 43 us past it and 39 through it).
bool streams(const AddNormProblem& p)
{
    const int64_t e = p.bf16 ? 2 : 4, es = p.sum_fp32 ? 4 : e;
    return (int64_t)p.B * p.T * p.C * (2 * e + (p.dtotal.p ? 2 : 1) * es) >= (int64_t(256) << 20);
}

// THREADS: the workgroup's size is at most that.  1024 leave a lane 128 registers: bf16 rows of more than 8192 channels
// keep 47 to 51 values in scratch, those with a stream of fp32 100; no other variant keeps any.
template <typename T, typename S, int NV, int THREADS, bool EDGE, bool NT>
__global__ __launch_bounds__(THREADS) void addnorm_bwd_kernel(AddNormProblem p, RowMap m)
{
    constexpr bool TWO = sizeof(T) != sizeof(S);
    constexpr int VEC = vec_of<T, S>();
    __shared__ float red1[2][16][1], red3[2][16][3];
    __shared__ float acc[THREADS > 256 ? 1 : 256 * NV * VEC];
    const int slot = threadIdx.x / m.L, lv = threadIdx.x - slot * m.L;
    const bool shift = !p.rms, behind = p.dtotal.p != nullptr;
    const Columns<VEC, NV, EDGE> cols(lv, m.L, m.nv, p.C);
    const int* c = cols.c;
    float w[NV][VEC], dw[NV][VEC], db[NV][VEC];
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            w[k][v] = p.weight ? p.weight[c[k] + v] : 1.0f;
            dw[k][v] = db[k][v] = 0.0f;
        }
    const float inv = 1.0f / (float)p.C;
    Pack<S, VEC, EDGE, NT> rt[NV], re[NV];
    Pack<T, VEC, EDGE, NT> rg[NV];
    auto fetch = [&](unsigned i) {                    // behind the last row: the last
        i = min(i, m.rows - 1);
        const int64_t b = i / (unsigned)p.T, t = i % (unsigned)p.T;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            rt[k].load((const S*)p.total.p + b * p.total.batch + t * p.total.row + c[k]);
            rg[k].load((const T*)p.dy.p + b * p.dy.batch + t * p.dy.row + c[k]);
            if (behind) re[k].load((const S*)p.dtotal.p + b * p.dtotal.batch + t * p.dtotal.row + c[k]);
        }
    };
    const unsigned step = gridDim.x * m.slots, first = blockIdx.x * m.slots;
    fetch(first + slot);
    int turn = 0;
    for (unsigned i0 = first; i0 < m.rows; i0 += step, turn ^= 1) {
        const unsigned i = i0 + slot;
        const bool live = i < m.rows;
        float d[NV][VEC], g[NV][VEC], s = 0.0f, mean = 0.0f;
        Pack<S, VEC, EDGE, NT> e[NV];
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            e[k] = re[k];
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                d[k][v] = rt[k].get(v);
                g[k][v] = rg[k].get(v);
            }
        }
        fetch(i + step);
        if (shift) {
#pragma unroll
            for (int k = 0; k < NV; ++k)
#pragma unroll
                for (int v = 0; v < VEC; ++v) s += cols.counts(k, v) ? d[k][v] : 0.0f;
            row_sums<1>(&s, m.L, red1, turn);
            mean = s * inv;
        }
        float q[3] = {0.0f, 0.0f, 0.0f};              // d^2, v, v d
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                d[k][v] -= mean;
                const float u = g[k][v] * w[k][v];
                q[0] += cols.counts(k, v) ? d[k][v] * d[k][v] : 0.0f;
                q[1] += cols.counts(k, v) ? u : 0.0f;
                q[2] += cols.counts(k, v) ? u * d[k][v] : 0.0f;
            }
        row_sums<3>(q, m.L, red3, turn);
        const float rstd = 1.0f / sqrtf(q[0] * inv + p.eps);
        if (!live) continue;
        const float m1 = shift ? q[1] * inv : 0.0f, m2 = q[2] * inv * rstd * rstd;
        const int64_t b = i / (unsigned)p.T, t = i % (unsigned)p.T;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            if (!cols.in[k]) continue;
            Pack<T, VEC, EDGE, false> o;
            Pack<S, VEC, EDGE, false> o2;
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                dw[k][v] += g[k][v] * (d[k][v] * rstd);
                db[k][v] += g[k][v];
                float x = rstd * (g[k][v] * w[k][v] - m1 - d[k][v] * m2);
                if (behind) x += e[k].get(v);
                o.set(v, x);
                if (TWO) o2.set(v, x);
            }
            o.store((T*)p.dx.p + b * p.dx.batch + t * p.dx.row + c[k]);
            if (TWO && p.dresidual.p) o2.store((S*)p.dresidual.p + b * p.dresidual.batch + t * p.dresidual.row + c[k]);
        }
    }
    if (!p.dweight && !p.dbias) return;
    float* part = (float*)p.ws + (int64_t)blockIdx.x * 2 * p.C;
    float *pw = m.only ? p.dweight : part, *pb = m.only ? p.dbias : part + p.C;
    if (m.slots == 1) {
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int v = 0; v < VEC; ++v)
                if (cols.in[k]) {
                    if (pw) pw[c[k] + v] = dw[k][v];
                    if (pb) pb[c[k] + v] = db[k][v];
                }
        return;
    }
    if constexpr (THREADS == 256) {
        // the slots' sums in order
        for (int which = 0; which < 2; ++which) {
            float* to = which ? pb : pw;
            if (!to) continue;
            __syncthreads();
#pragma unroll
            for (int k = 0; k < NV; ++k)
#pragma unroll
                for (int v = 0; v < VEC; ++v) acc[(k * 256 + threadIdx.x) * VEC + v] = which ? db[k][v] : dw[k][v];
            __syncthreads();
            const int n = m.L * VEC;
            for (int e = threadIdx.x; e < NV * n; e += 256) {
                const int k = e / n, at = e % n, i = k * m.L + at / VEC;
                float s = 0.0f;
                for (int j = 0; j < m.slots; ++j) s += acc[k * 256 * VEC + j * n + at];
                if (i < m.nv) to[column<VEC, EDGE>(i, p.C) + at % VEC] = s;
            }
        }
    }
}

// Rows of any length: dt by a workgroup to a row in two readings, the statistics left in the workspace, the weights'
// gradients by a thread to a column and a run of rows in a third.
constexpr int kRun = 64;

template <typename T, typename S>
__global__ __launch_bounds__(256) void addnorm_bwd_long_kernel(AddNormProblem p, f32x2* stats)
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
    if (threadIdx.x == 0 && (p.dweight || p.dbias)) stats[id] = f32x2{mean, rstd};
}

template <typename T, typename S>
__global__ __launch_bounds__(256) void addnorm_columns_kernel(AddNormProblem p, const f32x2* stats)
{
    const int nb = (p.C + 255) / 256;
    const int64_t run = block_id() / nb, rows = (int64_t)p.B * p.T;
    const int c = (int)(block_id() % nb) * 256 + threadIdx.x;
    if (c >= p.C || run * kRun >= rows) return;
    float dw = 0.0f, db = 0.0f;
    for (int64_t i = run * kRun; i < min(rows, (run + 1) * kRun); ++i) {
        const int64_t b = i / p.T, t = i % p.T;
        const f32x2 st = stats[i];
        const float g = to_float(((const T*)p.dy.p)[b * p.dy.batch + t * p.dy.row + c]);
        dw += g * ((to_float(((const S*)p.total.p)[b * p.total.batch + t * p.total.row + c]) - st[0]) * st[1]);
        db += g;
    }
    float* part = (float*)p.ws + run * 2 * p.C;
    part[c] = dw;
    part[p.C + c] = db;
}

// dweight and dbias from the workgroups' sums [parts][2][C]
__global__ __launch_bounds__(1024) void addnorm_params_kernel(AddNormProblem p, int64_t parts)
{
    __shared__ float red[16][64];
    const int64_t W = p.C, i = (int64_t)blockIdx.x * 64 + threadIdx.x;
    const float s = part_sum((const float*)p.ws, parts, 2 * W, 2 * W, blockIdx.x, red);
    if (threadIdx.x >= 64 || i >= 2 * W) return;
    if (i < W) {
        if (p.dweight) p.dweight[i] = s;
    } else if (p.dbias) {
        p.dbias[i - W] = s;
    }
}

hipError_t params(const AddNormProblem& p, int64_t parts, hipStream_t stream)
{
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || (!p.dweight && !p.dbias)) return e;
    addnorm_params_kernel<<<(unsigned)((2 * (int64_t)p.C + 63) / 64), 1024, 0, stream>>>(p, parts);
    return hipGetLastError();
}

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }
int64_t runs_of(const AddNormProblem& p) { return ((int64_t)p.B * p.T + kRun - 1) / kRun; }

template <typename T, typename S, bool EDGE, bool NT>
hipError_t bwd_n(const AddNormProblem& p, hipStream_t stream)
{
    const RowMap m = map_of(p);
    const int v = (m.nv + m.L - 1) / m.L;
    constexpr int most = most_vectors<T, S>();
    if constexpr (sizeof(T) == 2 && sizeof(S) == 2)
        if (m.threads > 256 && v == 1) {
            addnorm_bwd_kernel<T, S, 1, 1024, EDGE, NT><<<m.blocks, m.threads, 0, stream>>>(p, m);
            return m.only ? hipGetLastError() : params(p, m.blocks, stream);
        }
    if (m.threads > 512) addnorm_bwd_kernel<T, S, most, 1024, EDGE, NT><<<m.blocks, m.threads, 0, stream>>>(p, m);
    else if (m.threads > 256) addnorm_bwd_kernel<T, S, most, 512, EDGE, NT><<<m.blocks, m.threads, 0, stream>>>(p, m);
    else if (v == 1) addnorm_bwd_kernel<T, S, 1, 256, EDGE, NT><<<m.blocks, m.threads, 0, stream>>>(p, m);
    else if (v == 2) addnorm_bwd_kernel<T, S, 2, 256, EDGE, NT><<<m.blocks, m.threads, 0, stream>>>(p, m);
    else if constexpr (most == 4) addnorm_bwd_kernel<T, S, 4, 256, EDGE, NT><<<m.blocks, m.threads, 0, stream>>>(p, m);
    return m.only ? hipGetLastError() : params(p, m.blocks, stream);
}

template <typename T, typename S>
hipError_t bwd_long(const AddNormProblem& p, hipStream_t stream)
{
    f32x2* stats = (f32x2*)(p.ws + align256((size_t)runs_of(p) * 2 * p.C * sizeof(float)));
    addnorm_bwd_long_kernel<T, S><<<grid_of((int64_t)p.B * p.T), 256, 0, stream>>>(p, stats);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || (!p.dweight && !p.dbias)) return e;
    addnorm_columns_kernel<T, S><<<grid_of(runs_of(p) * ((p.C + 255) / 256)), 256, 0, stream>>>(p, stats);
    return params(p, runs_of(p), stream);
}

template <typename T, typename S>
hipError_t bwd_t(const AddNormProblem& p, hipStream_t stream)
{
    if (!in_registers(p)) return bwd_long<T, S>(p, stream);
    const bool edge = edged(p, {&p.total, &p.dy, &p.dtotal, &p.dx, &p.dresidual});
    if (streams(p)) return edge ? bwd_n<T, S, true, true>(p, stream) : bwd_n<T, S, false, true>(p, stream);
    return edge ? bwd_n<T, S, true, false>(p, stream) : bwd_n<T, S, false, false>(p, stream);
}

}  // namespace

size_t addnorm_bwd_workspace(const AddNormProblem& p)
{
    const size_t row = 2 * (size_t)p.C * sizeof(float);
    if (in_registers(p)) return map_of(p).only ? 0 : map_of(p).blocks * row;
    return align256((size_t)runs_of(p) * row) + (size_t)p.B * p.T * sizeof(f32x2);
}

hipError_t launch_addnorm_bwd(const AddNormProblem& p, hipStream_t stream)
{
    if (!p.bf16) return bwd_t<float, float>(p, stream);
    return p.sum_fp32 ? bwd_t<bf16, float>(p, stream) : bwd_t<bf16, bf16>(p, stream);
}

}  // namespace tfla
