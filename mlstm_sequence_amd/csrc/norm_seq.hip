// norm_seq.hip -- group norm over a sequence's rows (norm_impl.hpp): a
// feature map's places as rows, say.
//
// A lane owns VEC columns of the G x C, a workgroup 64 such lanes and a run
// of rows that its four waves share.  Forward: the columns' means and squared
// deviations of each run (groups of rows formed around their own mean and
// joined pairwise, so a large mean costs no digits), joined over columns and
// runs to one mean and rstd a set, then the values once more to normalise
// them.  Backward: the columns' sums of du and du xh of each run, which give
// the weights' gradients and, weighted, the set's two means; then the values
// once more.  Bound by memory: two readings and a writing (what fits the
// last-level cache is read from there the second time).  6 x 4096 x 512 fp32:
// forward and backward together, 400 MB with the second readings, in 84 us,
// 4.8 TB/s.
#include "norm_impl.hpp"

namespace tfla {
namespace {

using namespace norm;

constexpr int kRows = 4;   // rows loaded together

struct SeqMap {
    int nv, ncs;           // vectors of a row, workgroups across it
    int run, nrun;         // rows of a run, runs of a sequence
};

SeqMap seq_map(const NormProblem& p, int vec)
{
    SeqMap m;
    m.nv = p.G * p.C / vec;
    m.ncs = (m.nv + 63) / 64;
    m.run = 16;            // rows of each wave: a quarter
    while (m.run < 256 && (int64_t)p.B * m.ncs * ((p.T + 2 * m.run - 1) / (2 * m.run)) >= 384) m.run *= 2;
    m.nrun = (p.T + m.run - 1) / m.run;
    return m;
}

// The lane's columns: rows lie at base + t * row.
struct Cols {
    int b, run, cs, g, c, lane, wave, t0, t1;
    bool live;
    template <int VEC> __device__ __forceinline__ bool set(const NormProblem& p, const SeqMap& m)
    {
        int64_t i = block_id();
        cs = (int)(i % m.ncs);
        i /= m.ncs;
        run = (int)(i % m.nrun);
        if (i / m.nrun >= p.B) return false;
        b = (int)(i / m.nrun);
        lane = threadIdx.x & 63;
        wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        const int cv = cs * 64 + lane;
        live = cv < m.nv;
        const int col = min(cv, m.nv - 1) * VEC;
        g = col / p.C;
        c = col % p.C;
        // each wave a quarter of the run
        const int q = m.run / 4;
        t0 = min(run * m.run + wave * q, p.T);
        t1 = min(t0 + q, p.T);
        return true;
    }
};

__device__ __forceinline__ void join(float& n, float& mean, float& m2, float nb, float mb, float m2b)
{
    const float t = n + nb, d = mb - mean, f = nb / t;
    mean += d * f;
    m2 += m2b + d * d * n * f;
    n = t;
}

// means and squared deviations of the run's columns: part [B][nrun][2][G C]
template <typename T, int VEC>
__global__ __launch_bounds__(256) void seq_stats_kernel(NormProblem p, SeqMap m)
{
    __shared__ float red[4][2][64 * VEC];
    Cols q;
    if (!q.set<VEC>(p, m)) return;
    const T* x = (const T*)p.x.p + at(p.x, q.b, 0, q.g, q.c);
    float mean[VEC], m2[VEC], n = 0.0f;
#pragma unroll
    for (int v = 0; v < VEC; ++v) mean[v] = m2[v] = 0.0f;
    Pack<T, VEC> raw[kRows];
    auto fetch = [&](int t) {
#pragma unroll
        for (int k = 0; k < kRows; ++k) raw[k].load(x + min(t + k, p.T - 1) * p.x.row);
    };
    fetch(q.t0);
    for (int t = q.t0; t < q.t1; t += kRows) {
        const int cnt = min(kRows, q.t1 - t);
        float e[kRows][VEC];
#pragma unroll
        for (int k = 0; k < kRows; ++k)
#pragma unroll
            for (int v = 0; v < VEC; ++v) e[k][v] = raw[k].get(v);
        fetch(t + kRows);
        const float nb = (float)cnt, tot = n + nb, f = nb / tot, inv = 1.0f / nb;
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            float s = 0.0f, d2 = 0.0f;
#pragma unroll
            for (int k = 0; k < kRows; ++k) s += k < cnt ? e[k][v] : 0.0f;
            s *= inv;
#pragma unroll
            for (int k = 0; k < kRows; ++k) {
                const float d = k < cnt ? e[k][v] - s : 0.0f;
                d2 += d * d;
            }
            const float d = s - mean[v];
            mean[v] += d * f;
            m2[v] += d2 + d * d * n * f;
        }
        n = tot;
    }
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
        red[q.wave][0][v * 64 + q.lane] = mean[v];
        red[q.wave][1][v * 64 + q.lane] = m2[v];
    }
    __syncthreads();
    const int W = p.G * p.C, r0 = q.run * m.run, quarter = m.run / 4;
    float* part = (float*)p.ws + ((int64_t)q.b * m.nrun + q.run) * 2 * W;
    for (int i = threadIdx.x; i < 64 * VEC; i += 256) {
        const int cv = q.cs * 64 + (i & 63);
        float nn = (float)min(quarter, p.T - r0), a = red[0][0][i], s = red[0][1][i];
        for (int w = 1; w < 4; ++w) {
            const int rows = min(quarter, p.T - r0 - w * quarter);
            if (rows > 0) join(nn, a, s, (float)rows, red[w][0][i], red[w][1][i]);
        }
        if (cv < m.nv) {
            part[cv * VEC + (i >> 6)] = a;
            part[W + cv * VEC + (i >> 6)] = s;
        }
    }
}

// One workgroup to a set: mean and rstd, to the caller's arrays and stat [B][G][2].
__global__ __launch_bounds__(256) void seq_join_kernel(NormProblem p, SeqMap m, float* __restrict__ stat)
{
    __shared__ float red[3][256];
    const int b = (int)(blockIdx.x / p.G), g = (int)(blockIdx.x % p.G);
    const int64_t W = (int64_t)p.G * p.C;
    const float* part = (const float*)p.ws + (int64_t)b * m.nrun * 2 * W + (int64_t)g * p.C;
    float n = 0.0f, mean = 0.0f, m2 = 0.0f;
    for (unsigned i = threadIdx.x; i < (unsigned)m.nrun * p.C; i += 256) {
        const int run = (int)(i / p.C), c = (int)(i % p.C);
        const float* s = part + run * 2 * W + c;
        join(n, mean, m2, (float)min(m.run, p.T - run * m.run), s[0], s[W]);
    }
    red[0][threadIdx.x] = n;
    red[1][threadIdx.x] = mean;
    red[2][threadIdx.x] = m2;
    for (int k = 128; k; k >>= 1) {
        __syncthreads();
        if ((int)threadIdx.x < k && red[0][threadIdx.x + k] > 0.0f)
            join(red[0][threadIdx.x], red[1][threadIdx.x], red[2][threadIdx.x], red[0][threadIdx.x + k],
                 red[1][threadIdx.x + k], red[2][threadIdx.x + k]);
    }
    if (threadIdx.x == 0) {
        const float rstd = 1.0f / sqrtf(red[2][0] / red[0][0] + p.eps);
        const int64_t id = blockIdx.x;
        stat[2 * id] = red[1][0];
        stat[2 * id + 1] = rstd;
        if (p.mean) p.mean[id] = red[1][0];
        if (p.rstd) p.rstd[id] = rstd;
    }
}

template <typename T, int VEC, bool GATED, bool ACTIVE>
__global__ __launch_bounds__(256) void seq_apply_kernel(NormProblem p, SeqMap m, const float* __restrict__ stat)
{
    Cols q;
    if (!q.set<VEC>(p, m) || !q.live) return;
    const T* x = (const T*)p.x.p + at(p.x, q.b, 0, q.g, q.c);
    const T* z = GATED ? (const T*)p.gate.p + at(p.gate, q.b, 0, q.g, q.c) : nullptr;
    T* y = (T*)p.y.p + at(p.y, q.b, 0, q.g, q.c);
    const bool silu = p.act == kActSilu;
    const float mean = stat[2 * ((int64_t)q.b * p.G + q.g)], rstd = stat[2 * ((int64_t)q.b * p.G + q.g) + 1];
    float w[VEC], bs[VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
        w[v] = rstd * (p.weight ? p.weight[(int64_t)q.g * p.C + q.c + v] : 1.0f);
        bs[v] = p.bias ? p.bias[(int64_t)q.g * p.C + q.c + v] : 0.0f;
    }
    Pack<T, VEC> rx[kRows], rz[kRows];
    auto fetch = [&](int t) {
#pragma unroll
        for (int k = 0; k < kRows; ++k) {
            const int64_t s = min(t + k, p.T - 1);
            rx[k].load(x + s * p.x.row);
            if (GATED) rz[k].load(z + s * p.gate.row);
        }
    };
    fetch(q.t0);
    for (int t = q.t0; t < q.t1; t += kRows) {
        Pack<T, VEC> o[kRows];
#pragma unroll
        for (int k = 0; k < kRows; ++k)
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                const float u = (rx[k].get(v) - mean) * w[v] + bs[v];
                o[k].set(v, GATED ? u * act_f<T, ACTIVE>(rz[k].get(v), silu) : act_f<T, ACTIVE>(u, silu));
            }
        fetch(t + kRows);
#pragma unroll
        for (int k = 0; k < kRows; ++k)
            if (t + k < q.t1) o[k].store(y + (t + k) * p.y.row);
    }
}

// FINAL: dx and dgate, given the sets' two means in `means` [B][G][2]; else the columns' sums of du xh and du of
// the run: part [B][nrun][2][G C].
template <typename T, int VEC, bool GATED, bool ACTIVE, bool FINAL>
__global__ __launch_bounds__(256) void seq_grad_kernel(NormProblem p, SeqMap m, const float* __restrict__ means)
{
    __shared__ float red[FINAL ? 1 : 4][2][64 * VEC];
    Cols q;
    if (!q.set<VEC>(p, m)) return;
    const T* x = (const T*)p.x.p + at(p.x, q.b, 0, q.g, q.c);
    const T* dy = (const T*)p.dy.p + at(p.dy, q.b, 0, q.g, q.c);
    const T* z = GATED ? (const T*)p.gate.p + at(p.gate, q.b, 0, q.g, q.c) : nullptr;
    T* dx = FINAL ? (T*)p.dx.p + at(p.dx, q.b, 0, q.g, q.c) : nullptr;
    T* dz = FINAL && GATED ? (T*)p.dgate.p + at(p.dgate, q.b, 0, q.g, q.c) : nullptr;
    const bool silu = p.act == kActSilu;
    const int64_t id = (int64_t)q.b * p.G + q.g;
    const float mean = p.mean[id], rstd = p.rstd[id];
    const float c1 = FINAL ? means[2 * id] : 0.0f, c2 = FINAL ? means[2 * id + 1] : 0.0f;
    float w[VEC], bs[VEC], s1[VEC], s2[VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
        w[v] = p.weight ? p.weight[(int64_t)q.g * p.C + q.c + v] : 1.0f;
        bs[v] = p.bias ? p.bias[(int64_t)q.g * p.C + q.c + v] : 0.0f;
        s1[v] = s2[v] = 0.0f;
    }
    Pack<T, VEC> rx[kRows], rg[kRows], rz[kRows];
    auto fetch = [&](int t) {
#pragma unroll
        for (int k = 0; k < kRows; ++k) {
            const int64_t s = min(t + k, p.T - 1);
            rx[k].load(x + s * p.x.row);
            rg[k].load(dy + s * p.dy.row);
            if (GATED) rz[k].load(z + s * p.gate.row);
        }
    };
    fetch(q.t0);
    for (int t = q.t0; t < q.t1; t += kRows) {
        Pack<T, VEC> o[kRows], oz[kRows];
#pragma unroll
        for (int k = 0; k < kRows; ++k)
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                const float xh = (rx[k].get(v) - mean) * rstd, u = xh * w[v] + bs[v], g = rg[k].get(v);
                float f, slope;
                act_both<T, ACTIVE>(GATED ? rz[k].get(v) : u, silu, &f, &slope);
                const float du = g * (GATED ? f : slope);
                if (FINAL) {
                    o[k].set(v, rstd * (du * w[v] - c1 - xh * c2));
                    if (GATED) oz[k].set(v, g * u * slope);
                } else {
                    const bool own = t + k < q.t1;
                    s1[v] += own ? du * xh : 0.0f;
                    s2[v] += own ? du : 0.0f;
                }
            }
        fetch(t + kRows);
        if (FINAL && q.live) {
#pragma unroll
            for (int k = 0; k < kRows; ++k)
                if (t + k < q.t1) {
                    o[k].store(dx + (t + k) * p.dx.row);
                    if (GATED) oz[k].store(dz + (t + k) * p.dgate.row);
                }
        }
    }
    if (FINAL) return;
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
        red[FINAL ? 0 : q.wave][0][v * 64 + q.lane] = s1[v];
        red[FINAL ? 0 : q.wave][1][v * 64 + q.lane] = s2[v];
    }
    __syncthreads();
    const int64_t W = (int64_t)p.G * p.C;
    float* part = (float*)p.ws + ((int64_t)q.b * m.nrun + q.run) * 2 * W;
    for (int i = threadIdx.x; i < 2 * 64 * VEC; i += 256) {
        const int which = i / (64 * VEC), e = i % (64 * VEC), cv = q.cs * 64 + (e & 63);
        float s = 0.0f;
        for (int u = 0; u < (FINAL ? 1 : 4); ++u) s += red[u][which][e];
        if (cv < m.nv) part[which * W + cv * VEC + (e >> 6)] = s;
    }
}

// The first B G workgroups, one to a set: mean(v) and mean(v xh); the others, 64 columns each: dweight and dbias.
__global__ __launch_bounds__(1024) void seq_means_kernel(NormProblem p, SeqMap m, float* __restrict__ means)
{
    __shared__ float red[16][64];
    const int64_t W = (int64_t)p.G * p.C;
    const unsigned sets = (unsigned)p.B * p.G;
    if (blockIdx.x >= sets) {
        const int64_t i = (int64_t)(blockIdx.x - sets) * 64 + threadIdx.x;
        const float s = part_sum((const float*)p.ws, (int64_t)p.B * m.nrun, 2 * W, 2 * W, blockIdx.x - sets, red);
        if (threadIdx.x >= 64 || i >= 2 * W) return;
        if (i < W) {
            if (p.dweight) p.dweight[i] = s;
        } else if (p.dbias) {
            p.dbias[i - W] = s;
        }
        return;
    }
    const int b = (int)(blockIdx.x / p.G), g = (int)(blockIdx.x % p.G);
    const float* part = (const float*)p.ws + (int64_t)b * m.nrun * 2 * W + (int64_t)g * p.C;
    float s1 = 0.0f, s2 = 0.0f;
    for (int64_t i = threadIdx.x; i < (int64_t)m.nrun * p.C; i += 1024) {
        const int run = (int)(i / p.C), c = (int)(i % p.C);
        const float w = p.weight ? p.weight[(int64_t)g * p.C + c] : 1.0f;
        s1 += w * part[run * 2 * W + W + c];
        s2 += w * part[run * 2 * W + c];
    }
    s1 = lane_sum(s1, 64);
    s2 = lane_sum(s2, 64);
    if ((threadIdx.x & 63) == 0) {
        red[0][threadIdx.x >> 6] = s1;
        red[1][threadIdx.x >> 6] = s2;
    }
    __syncthreads();
    if (threadIdx.x < 2) {
        float s = 0.0f;
        for (int u = 0; u < 16; ++u) s += red[threadIdx.x][u];
        means[2 * (int64_t)blockIdx.x + threadIdx.x] = s / ((float)p.T * (float)p.C);
    }
}

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

size_t part_bytes(const NormProblem& p, const SeqMap& m)
{
    return align256((size_t)p.B * m.nrun * 2 * p.G * p.C * sizeof(float));
}

template <typename T, int VEC>
hipError_t fwd_vec(const NormProblem& p, hipStream_t stream)
{
    const SeqMap m = seq_map(p, VEC);
    const dim3 blocks = grid_of((int64_t)p.B * m.nrun * m.ncs);
    float* stat = (float*)(p.ws + part_bytes(p, m));
    seq_stats_kernel<T, VEC><<<blocks, 256, 0, stream>>>(p, m);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    seq_join_kernel<<<(unsigned)(p.B * p.G), 256, 0, stream>>>(p, m, stat);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    const bool a = p.act != kActNone;
    if (p.gate.p) {
        if (a) seq_apply_kernel<T, VEC, true, true><<<blocks, 256, 0, stream>>>(p, m, stat);
        else seq_apply_kernel<T, VEC, true, false><<<blocks, 256, 0, stream>>>(p, m, stat);
    } else {
        if (a) seq_apply_kernel<T, VEC, false, true><<<blocks, 256, 0, stream>>>(p, m, stat);
        else seq_apply_kernel<T, VEC, false, false><<<blocks, 256, 0, stream>>>(p, m, stat);
    }
    return hipGetLastError();
}

template <typename T, int VEC, bool GATED, bool ACTIVE>
hipError_t bwd_g(const NormProblem& p, hipStream_t stream)
{
    const SeqMap m = seq_map(p, VEC);
    const dim3 blocks = grid_of((int64_t)p.B * m.nrun * m.ncs);
    float* means = (float*)(p.ws + part_bytes(p, m));
    seq_grad_kernel<T, VEC, GATED, ACTIVE, false><<<blocks, 256, 0, stream>>>(p, m, nullptr);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int64_t W = (int64_t)p.G * p.C;
    const int64_t params = p.dweight || p.dbias ? (2 * W + 63) / 64 : 0;
    seq_means_kernel<<<(unsigned)((int64_t)p.B * p.G + params), 1024, 0, stream>>>(p, m, means);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    seq_grad_kernel<T, VEC, GATED, ACTIVE, true><<<blocks, 256, 0, stream>>>(p, m, means);
    return hipGetLastError();
}

template <typename T, int VEC>
hipError_t bwd_vec(const NormProblem& p, hipStream_t stream)
{
    const bool a = p.act != kActNone;
    if (p.gate.p) return a ? bwd_g<T, VEC, true, true>(p, stream) : bwd_g<T, VEC, true, false>(p, stream);
    return a ? bwd_g<T, VEC, false, true>(p, stream) : bwd_g<T, VEC, false, false>(p, stream);
}

template <typename T, bool BWD>
hipError_t seq_t(const NormProblem& p, hipStream_t stream)
{
    constexpr int wide = 16 / sizeof(T);
    const bool v = vec_of(p, BWD) == wide;
    if constexpr (BWD) return v ? bwd_vec<T, wide>(p, stream) : bwd_vec<T, 1>(p, stream);
    else return v ? fwd_vec<T, wide>(p, stream) : fwd_vec<T, 1>(p, stream);
}

}  // namespace

namespace norm {

// For whichever width the call's addresses allow; both passes keep the same.
size_t seq_workspace(const NormProblem& p)
{
    size_t most = 0;
    for (const int v : {1, p.bf16 ? 8 : 4}) {
        if (p.C % v) continue;
        const size_t n = part_bytes(p, seq_map(p, v));
        if (n > most) most = n;
    }
    return most + align256((size_t)p.B * p.G * 2 * sizeof(float));
}
size_t seq_bwd_workspace(const NormProblem& p) { return seq_workspace(p); }

hipError_t launch_seq_fwd(const NormProblem& p, hipStream_t stream)
{
    return p.bf16 ? seq_t<bf16, false>(p, stream) : seq_t<float, false>(p, stream);
}

hipError_t launch_seq_bwd(const NormProblem& p, hipStream_t stream)
{
    return p.bf16 ? seq_t<bf16, true>(p, stream) : seq_t<float, true>(p, stream);
}

}  // namespace norm
}  // namespace tfla
