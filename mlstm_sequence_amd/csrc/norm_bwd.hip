// norm_bwd.hip -- group norm per token, backward (norm_impl.hpp).
//
// The layout of the forward pass: a row in the registers of L lanes, weights
// kept, and with them the sums of their gradients over the tokens that a wave
// walks; the four waves of a workgroup walk different tokens of the same
// groups, add their sums in LDS and leave them in the workspace, to be added
// over the workgroups in a fixed order.  Bound by memory: x, dy and the gate
// are read once, dx and the gate's gradient written once: [8,4096,32,128] bf16,
// 1.35 GB in 278 us, 4.9 TB/s, where a copy moves 5.1.
#include "norm_impl.hpp"

namespace tfla {
namespace {

using namespace norm;

template <typename T, int VEC, int V, bool GATED, bool ACTIVE, bool BLOCK, bool NT>
__global__ __launch_bounds__(256) void norm_bwd_kernel(NormProblem p, TokenMap m)
{
    __shared__ float red[BLOCK ? 1 : 4][2][BLOCK ? 4 : 64 * VEC];
    const int lane = BLOCK ? threadIdx.x : threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const unsigned id = (unsigned)block_id(), group = id / (unsigned)m.ng, chunk = BLOCK ? group : group * 4 + wave;
    const int set = (int)(id % (unsigned)m.ng);
    if ((BLOCK ? group : group * 4) >= m.chunks) return;
    const unsigned i0 = min(chunk, m.chunks) * m.per * m.step;
    const unsigned i1 = chunk < m.chunks ? min(i0 + m.per * m.step, m.tokens) : i0;   // none behind the last chunk
    const int slot = lane / m.L, lv = lane & (m.L - 1);
    const int g = m.by_group ? set * m.slots + slot : set;
    const int off = m.by_group ? 0 : slot;
    const bool silu = p.act == kActSilu;
    const T* xp = (const T*)p.x.p + g * p.x.group;
    const T* gp = (const T*)p.dy.p + g * p.dy.group;
    const T* zp = GATED ? (const T*)p.gate.p + g * p.gate.group : nullptr;
    T* dxp = (T*)p.dx.p + g * p.dx.group;
    T* dzp = GATED ? (T*)p.dgate.p + g * p.dgate.group : nullptr;
    int c[V];
    bool in[V];
    float w[V][VEC], bs[V][VEC], dw[V][VEC], db[V][VEC];
#pragma unroll
    for (int k = 0; k < V; ++k) {
        in[k] = lv + k * m.L < m.nv;
        c[k] = min(lv + k * m.L, m.nv - 1) * VEC;
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            w[k][v] = p.weight ? p.weight[g * p.C + c[k] + v] : 1.0f;
            bs[k][v] = p.bias ? p.bias[g * p.C + c[k] + v] : 0.0f;
            dw[k][v] = db[k][v] = 0.0f;
        }
    }
    const float inv = 1.0f / (float)p.C;

    Pack<T, VEC> rx[V], rg[V], rz[V];
    float rm, rr;
    auto fetch = [&](unsigned i) {
        i = min(i + off, m.tokens - 1);
        const int b = (int)(i / (unsigned)p.T), t = (int)(i % (unsigned)p.T);
        rm = p.mean[(int64_t)i * p.G + g];
        rr = p.rstd[(int64_t)i * p.G + g];
#pragma unroll
        for (int k = 0; k < V; ++k) {
            rx[k].template load_t<NT>(xp + b * p.x.batch + t * p.x.row + c[k]);
            rg[k].template load_t<NT>(gp + b * p.dy.batch + t * p.dy.row + c[k]);
            if (GATED) rz[k].template load_t<NT>(zp + b * p.gate.batch + t * p.gate.row + c[k]);
        }
    };
    fetch(i0);
    for (unsigned i = i0; i < i1; i += m.step) {
        const float mean = rm, rstd = rr;
        float xh[V][VEC], du[V][VEC], dz[V][VEC], s1 = 0.0f, s2 = 0.0f;
        const unsigned tok = i + off;
        const bool live = tok < i1;
#pragma unroll
        for (int k = 0; k < V; ++k)
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                xh[k][v] = (rx[k].get(v) - mean) * rstd;
                du[k][v] = rg[k].get(v);
                if (GATED) dz[k][v] = rz[k].get(v);
            }
        fetch(i + m.step);
#pragma unroll
        for (int k = 0; k < V; ++k)
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                const float u = xh[k][v] * w[k][v] + bs[k][v], dy = du[k][v];
                float f, slope;
                act_both<T, ACTIVE>(GATED ? dz[k][v] : u, silu, &f, &slope);
                du[k][v] = dy * (GATED ? f : slope);
                if (GATED) dz[k][v] = dy * u * slope;
                const float d = live && in[k] ? du[k][v] : 0.0f;
                dw[k][v] += d * (live && in[k] ? xh[k][v] : 0.0f);
                db[k][v] += d;
                du[k][v] *= w[k][v];
                s1 += in[k] ? du[k][v] : 0.0f;
                s2 += in[k] ? du[k][v] * xh[k][v] : 0.0f;
            }
        s1 = row_sum<BLOCK>(s1, m.L, red[0][0]) * inv;
        s2 = row_sum<BLOCK>(s2, m.L, red[0][1]) * inv;
        if (!live) continue;                          // never for a workgroup's row
        const int b = (int)(tok / (unsigned)p.T), t = (int)(tok % (unsigned)p.T);
#pragma unroll
        for (int k = 0; k < V; ++k) {
            Pack<T, VEC> o, oz;
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                o.set(v, rstd * (du[k][v] - s1 - xh[k][v] * s2));
                if (GATED) oz.set(v, dz[k][v]);
            }
            if (in[k]) {
                o.template store_t<NT>(dxp + b * p.dx.batch + t * p.dx.row + c[k]);
                if (GATED) oz.template store_t<NT>(dzp + b * p.dgate.batch + t * p.dgate.row + c[k]);
            }
        }
    }
    if (!p.dweight && !p.dbias) return;
    const int64_t W = (int64_t)p.G * p.C;
    float* part = (float*)p.ws + group * 2 * W;
    if (BLOCK) {
#pragma unroll
        for (int k = 0; k < V; ++k)
#pragma unroll
            for (int v = 0; v < VEC; ++v)
                if (in[k]) {
                    part[(int64_t)g * p.C + c[k] + v] = dw[k][v];
                    part[W + (int64_t)g * p.C + c[k] + v] = db[k][v];
                }
        return;
    }
#pragma unroll
    for (int k = 0; k < V; ++k) {
        __syncthreads();
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            red[wave][0][lane * VEC + v] = dw[k][v];
            red[wave][1][lane * VEC + v] = db[k][v];
        }
        __syncthreads();
        // where slots are tokens they share their columns
        const int share = m.by_group ? 1 : m.slots, cols = 64 * VEC / share;
        for (int e = threadIdx.x; e < 2 * cols; e += 256) {
            const int which = e >= cols, q = which ? e - cols : e;
            float s = 0.0f;
            for (int a = 0; a < share; ++a)
                for (int u = 0; u < 4; ++u) s += red[u][which][a * cols + q];
            const int l = q / VEC, cv = (l & (m.L - 1)) + k * m.L;
            const int gg = m.by_group ? set * m.slots + l / m.L : set;
            if (cv < m.nv) part[which * W + (int64_t)gg * p.C + cv * VEC + q % VEC] = s;
        }
    }
}

// Rows of any length: dx and dgate by a workgroup to a row in two readings, the weights' gradients by a thread to a
// column and a run of tokens in a third.  Gated, bf16 [4092,8200] 332 us, where [4096,8192] takes 143 in registers
// (2.3 TB/s: four vectors a lane take all of them, one wave to a SIMD; [8192,4096] 95); fp32 [8184,4100] 454,
// [8192,4096] 159.
constexpr int kLongRun = 64;

template <typename T> struct Elem1 {
    float xh, du, dz;
};
template <typename T>
__device__ __forceinline__ Elem1<T> element(const NormProblem& p, float mean, float rstd, int b, int t, int g, int c)
{
    Elem1<T> e;
    const float w = p.weight ? p.weight[g * p.C + c] : 1.0f, bs = p.bias ? p.bias[g * p.C + c] : 0.0f;
    const bool active = p.act != kActNone, silu = p.act == kActSilu;
    e.xh = (to_float(((const T*)p.x.p)[at(p.x, b, t, g, c)]) - mean) * rstd;
    const float u = e.xh * w + bs, dy = to_float(((const T*)p.dy.p)[at(p.dy, b, t, g, c)]);
    const float a = p.gate.p ? to_float(((const T*)p.gate.p)[at(p.gate, b, t, g, c)]) : u;
    float f = a, slope = 1.0f;
    if (active) act_both<T, true>(a, silu, &f, &slope);
    e.du = dy * (p.gate.p ? f : slope);
    e.dz = dy * u * slope;
    return e;
}

template <typename T>
__global__ __launch_bounds__(256) void norm_bwd_long_kernel(NormProblem p)
{
    __shared__ float red[4];
    const int64_t id = block_id();
    if (id >= (int64_t)p.B * p.T * p.G) return;
    const int g = (int)(id % p.G);
    const int64_t tok = id / p.G;
    const int b = (int)(tok / p.T), t = (int)(tok % p.T);
    auto sum = [&](float v) { return row_sum<true>(v, 256, red); };
    const float mean = p.mean[id], rstd = p.rstd[id];
    float s1 = 0.0f, s2 = 0.0f;
    for (int c = threadIdx.x; c < p.C; c += 256) {
        const Elem1<T> e = element<T>(p, mean, rstd, b, t, g, c);
        const float v = e.du * (p.weight ? p.weight[g * p.C + c] : 1.0f);
        s1 += v;
        s2 += v * e.xh;
    }
    s1 = sum(s1) / (float)p.C;
    s2 = sum(s2) / (float)p.C;
    for (int c = threadIdx.x; c < p.C; c += 256) {
        const Elem1<T> e = element<T>(p, mean, rstd, b, t, g, c);
        const float v = e.du * (p.weight ? p.weight[g * p.C + c] : 1.0f);
        ((T*)p.dx.p)[at(p.dx, b, t, g, c)] = from_float<T>(rstd * (v - s1 - e.xh * s2));
        if (p.dgate.p) ((T*)p.dgate.p)[at(p.dgate, b, t, g, c)] = from_float<T>(e.dz);
    }
}

template <typename T>
__global__ __launch_bounds__(256) void norm_long_params_kernel(NormProblem p)
{
    const int W = p.G * p.C, nb = (W + 255) / 256;
    const int64_t part = block_id() / nb, rows = (int64_t)p.B * p.T;
    const int i = (int)(block_id() % nb) * 256 + threadIdx.x;
    if (i >= W || part * kLongRun >= rows) return;
    const int g = i / p.C, c = i % p.C;
    float s1 = 0.0f, s2 = 0.0f;
    const int64_t r1 = min((part + 1) * kLongRun, rows);
    for (int64_t r = part * kLongRun; r < r1; ++r) {
        const int64_t id = r * p.G + g;
        const Elem1<T> e = element<T>(p, p.mean[id], p.rstd[id], (int)(r / p.T), (int)(r % p.T), g, c);
        s1 += e.du * e.xh;
        s2 += e.du;
    }
    float* o = (float*)p.ws + part * 2 * W;
    o[i] = s1;
    o[W + i] = s2;
}

// dweight and dbias from the workgroups' sums [parts][2][G C]
__global__ __launch_bounds__(1024) void norm_params_kernel(NormProblem p, int64_t parts)
{
    __shared__ float red[16][64];
    const int64_t W = (int64_t)p.G * p.C, i = (int64_t)blockIdx.x * 64 + threadIdx.x;
    const float s = part_sum((const float*)p.ws, parts, 2 * W, 2 * W, blockIdx.x, red);
    if (threadIdx.x >= 64 || i >= 2 * W) return;
    if (i < W) {
        if (p.dweight) p.dweight[i] = s;
    } else if (p.dbias) {
        p.dbias[i - W] = s;
    }
}

hipError_t params(const NormProblem& p, int64_t parts, hipStream_t stream)
{
    const int64_t W = (int64_t)p.G * p.C;
    norm_params_kernel<<<(unsigned)((2 * W + 63) / 64), 1024, 0, stream>>>(p, parts);
    return hipGetLastError();
}

constexpr int64_t kWaves = 4096;
constexpr int kMostSteps = 32;

template <typename T, int VEC, int V, bool BLOCK, bool NT>
hipError_t bwd_v(const NormProblem& p, const TokenMap& m, hipStream_t stream)
{
    const int64_t groups = BLOCK ? m.chunks : (m.chunks + 3) / 4;
    const dim3 blocks = grid_of(groups * m.ng);
    const bool a = p.act != kActNone;
    if (p.gate.p) {
        if (a) norm_bwd_kernel<T, VEC, V, true, true, BLOCK, NT><<<blocks, BLOCK ? m.L : 256, 0, stream>>>(p, m);
        else norm_bwd_kernel<T, VEC, V, true, false, BLOCK, NT><<<blocks, BLOCK ? m.L : 256, 0, stream>>>(p, m);
    } else {
        if (a) norm_bwd_kernel<T, VEC, V, false, true, BLOCK, NT><<<blocks, BLOCK ? m.L : 256, 0, stream>>>(p, m);
        else norm_bwd_kernel<T, VEC, V, false, false, BLOCK, NT><<<blocks, BLOCK ? m.L : 256, 0, stream>>>(p, m);
    }
    hipError_t e = hipGetLastError();
    return e != hipSuccess || (!p.dweight && !p.dbias) ? e : params(p, groups, stream);
}

template <typename T, int VEC>
hipError_t bwd_vec(const NormProblem& p, hipStream_t stream)
{
    const TokenMap m = token_map(p, VEC, kWaves, kMostSteps);
    const bool nt = VEC > 1 && streams(p, p.gate.p ? 5 : 3);
    if (!m.block) return nt ? bwd_v<T, VEC, 1, false, (VEC > 1)>(p, m, stream) : bwd_v<T, VEC, 1, false, false>(p, m, stream);
    switch (lane_vectors(m)) {
    case 1: return bwd_v<T, VEC, 1, true, false>(p, m, stream);
    case 2: return bwd_v<T, VEC, 2, true, false>(p, m, stream);
    case 4: return bwd_v<T, VEC, 4, true, false>(p, m, stream);
    default: break;
    }
    norm_bwd_long_kernel<T><<<grid_of((int64_t)p.B * p.T * p.G), 256, 0, stream>>>(p);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || (!p.dweight && !p.dbias)) return e;
    const int64_t W = (int64_t)p.G * p.C, parts = ((int64_t)p.B * p.T + kLongRun - 1) / kLongRun;
    norm_long_params_kernel<T><<<grid_of(parts * ((W + 255) / 256)), 256, 0, stream>>>(p);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    return params(p, parts, stream);
}

template <typename T>
hipError_t bwd_t(const NormProblem& p, hipStream_t stream)
{
    constexpr int wide = 16 / sizeof(T);
    return vec_of(p, true) == wide ? bwd_vec<T, wide>(p, stream) : bwd_vec<T, 1>(p, stream);
}

}  // namespace

// For whichever width the call's addresses allow.
size_t norm_bwd_workspace(const NormProblem& p)
{
    if (p.sequence) return seq_bwd_workspace(p);
    int64_t most = ((int64_t)p.B * p.T + kLongRun - 1) / kLongRun;
    for (const int v : {1, p.bf16 ? 8 : 4}) {
        if (p.C % v) continue;
        const TokenMap m = token_map(p, v, kWaves, kMostSteps);
        const int64_t n = m.block ? m.chunks : (m.chunks + 3) / 4;
        if (n > most) most = n;
    }
    return (size_t)most * 2 * p.G * p.C * sizeof(float);
}

hipError_t launch_norm_bwd(const NormProblem& p, hipStream_t stream)
{
    if (p.sequence) return launch_seq_bwd(p, stream);
    return p.bf16 ? bwd_t<bf16>(p, stream) : bwd_t<float>(p, stream);
}

}  // namespace tfla
