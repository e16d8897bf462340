// norm.hip -- group norm per token, forward (norm_impl.hpp).
//
// Bound by memory: x and the gate are read once, y written once.  A row lives
// in the registers of L lanes, so mean and variance take two passes over
// registers and 2 log2 L lane steps; the next row's loads are under way
// meanwhile: [4,8192,8,512] bf16 with a gate, 807 MB in 171 us, 4.7 TB/s, where
// a copy moves 5.1.  Rows too long for that (above 1024 vectors: 8192 channels in bf16,
// 4096 in fp32, 1024 where they lie at odd addresses) are walked by a workgroup each, from
// memory, in single elements and three readings: gated, bf16 [4096,8192] 56 us (3.6 TB/s; [8192,4096] 44),
// [4092,8200] 95; fp32 [8192,4096] 80, [8184,4100] 161.
#include "norm_impl.hpp"

namespace tfla {
namespace {

using namespace norm;

template <typename T, int VEC, int V, bool GATED, bool ACTIVE, bool BLOCK, bool NT>
__global__ __launch_bounds__(256) void norm_fwd_kernel(NormProblem p, TokenMap m)
{
    __shared__ float red[4];
    const int lane = BLOCK ? threadIdx.x : threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const unsigned id = BLOCK ? (unsigned)block_id() : (unsigned)block_id() * 4 + wave;
    if (id >= m.chunks * (unsigned)m.ng) return;
    const int set = (int)(id % (unsigned)m.ng);
    const unsigned i0 = id / (unsigned)m.ng * m.per * m.step, i1 = min(i0 + m.per * m.step, m.tokens);
    const int slot = lane / m.L, lv = lane & (m.L - 1);
    const int g = m.by_group ? set * m.slots + slot : set;
    const int off = m.by_group ? 0 : slot;            // of the lane's token in a step
    const bool silu = p.act == kActSilu;
    const T* xp = (const T*)p.x.p + g * p.x.group;
    const T* zp = GATED ? (const T*)p.gate.p + g * p.gate.group : nullptr;
    T* yp = (T*)p.y.p + g * p.y.group;
    int c[V];
    bool in[V];
    float w[V][VEC], bs[V][VEC];
#pragma unroll
    for (int k = 0; k < V; ++k) {
        in[k] = lv + k * m.L < m.nv;
        c[k] = min(lv + k * m.L, m.nv - 1) * VEC;
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            w[k][v] = p.weight ? p.weight[g * p.C + c[k] + v] : 1.0f;
            bs[k][v] = p.bias ? p.bias[g * p.C + c[k] + v] : 0.0f;
        }
    }
    const float inv = 1.0f / (float)p.C;

    Pack<T, VEC> rx[V], rz[V];
    auto fetch = [&](unsigned i) {                    // behind the last token: the last
        i = min(i + off, m.tokens - 1);
        const int b = (int)(i / (unsigned)p.T), t = (int)(i % (unsigned)p.T);
#pragma unroll
        for (int k = 0; k < V; ++k) {
            rx[k].template load_t<NT>(xp + b * p.x.batch + t * p.x.row + c[k]);
            if (GATED) rz[k].template load_t<NT>(zp + b * p.gate.batch + t * p.gate.row + c[k]);
        }
    };
    fetch(i0);
    for (unsigned i = i0; i < i1; i += m.step) {
        float x[V][VEC], z[V][VEC], s = 0.0f, q = 0.0f;
#pragma unroll
        for (int k = 0; k < V; ++k)
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                x[k][v] = rx[k].get(v);
                if (GATED) z[k][v] = rz[k].get(v);
            }
        fetch(i + m.step);
#pragma unroll
        for (int k = 0; k < V; ++k)
#pragma unroll
            for (int v = 0; v < VEC; ++v) s += in[k] ? x[k][v] : 0.0f;
        const float mean = row_sum<BLOCK>(s, m.L, red) * inv;
#pragma unroll
        for (int k = 0; k < V; ++k)
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                x[k][v] -= mean;
                q += in[k] ? x[k][v] * x[k][v] : 0.0f;
            }
        const float rstd = 1.0f / sqrtf(row_sum<BLOCK>(q, m.L, red) * inv + p.eps);
        const unsigned tok = i + off;
        if (tok >= i1) continue;                      // never for a workgroup's row
        const int b = (int)(tok / (unsigned)p.T), t = (int)(tok % (unsigned)p.T);
        if (lv == 0) {
            if (p.mean) p.mean[(int64_t)tok * p.G + g] = mean;
            if (p.rstd) p.rstd[(int64_t)tok * p.G + g] = rstd;
        }
#pragma unroll
        for (int k = 0; k < V; ++k) {
            Pack<T, VEC> o;
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                const float u = x[k][v] * rstd * w[k][v] + bs[k][v];
                o.set(v, GATED ? u * act_f<T, ACTIVE>(z[k][v], silu) : act_f<T, ACTIVE>(u, silu));
            }
            if (in[k]) o.store(yp + b * p.y.batch + t * p.y.row + c[k]);
        }
    }
}

// A workgroup to a row of any length.
template <typename T>
__global__ __launch_bounds__(256) void norm_fwd_long_kernel(NormProblem p)
{
    __shared__ float red[4];
    const int64_t id = block_id();
    if (id >= (int64_t)p.B * p.T * p.G) return;
    const int g = (int)(id % p.G);
    const int64_t tok = id / p.G;
    const int b = (int)(tok / p.T), t = (int)(tok % p.T);
    auto sum = [&](float v) { return row_sum<true>(v, 256, red); };
    const T* x = (const T*)p.x.p + at(p.x, b, t, g, 0);
    const T* z = p.gate.p ? (const T*)p.gate.p + at(p.gate, b, t, g, 0) : nullptr;
    T* y = (T*)p.y.p + at(p.y, b, t, g, 0);
    const float* w = p.weight ? p.weight + (int64_t)g * p.C : nullptr;
    const float* bs = p.bias ? p.bias + (int64_t)g * p.C : nullptr;
    float s = 0.0f, q = 0.0f;
    for (int c = threadIdx.x; c < p.C; c += 256) s += to_float(x[c]);
    const float mean = sum(s) / (float)p.C;
    for (int c = threadIdx.x; c < p.C; c += 256) {
        const float d = to_float(x[c]) - mean;
        q += d * d;
    }
    const float rstd = 1.0f / sqrtf(sum(q) / (float)p.C + p.eps);
    if (threadIdx.x == 0) {
        if (p.mean) p.mean[id] = mean;
        if (p.rstd) p.rstd[id] = rstd;
    }
    const bool active = p.act != kActNone, silu = p.act == kActSilu;
    for (int c = threadIdx.x; c < p.C; c += 256) {
        const float u = (to_float(x[c]) - mean) * rstd * (w ? w[c] : 1.0f) + (bs ? bs[c] : 0.0f);
        const float in = z ? to_float(z[c]) : u;
        const float f = active ? act_f<T, true>(in, silu) : in;
        y[c] = from_float<T>(z ? u * f : f);
    }
}

template <typename T, int VEC, int V, bool BLOCK, bool NT>
hipError_t fwd_v(const NormProblem& p, const TokenMap& m, hipStream_t stream)
{
    const int64_t n = (int64_t)m.chunks * m.ng;
    const dim3 blocks = grid_of(BLOCK ? n : (n + 3) / 4);
    const bool a = p.act != kActNone;
    if (p.gate.p) {
        if (a) norm_fwd_kernel<T, VEC, V, true, true, BLOCK, NT><<<blocks, BLOCK ? m.L : 256, 0, stream>>>(p, m);
        else norm_fwd_kernel<T, VEC, V, true, false, BLOCK, NT><<<blocks, BLOCK ? m.L : 256, 0, stream>>>(p, m);
    } else {
        if (a) norm_fwd_kernel<T, VEC, V, false, true, BLOCK, NT><<<blocks, BLOCK ? m.L : 256, 0, stream>>>(p, m);
        else norm_fwd_kernel<T, VEC, V, false, false, BLOCK, NT><<<blocks, BLOCK ? m.L : 256, 0, stream>>>(p, m);
    }
    return hipGetLastError();
}

template <typename T, int VEC>
hipError_t fwd_vec(const NormProblem& p, hipStream_t stream)
{
    const TokenMap m = token_map(p, VEC, 4096, 32);
    const bool nt = VEC > 1 && streams(p, p.gate.p ? 3 : 2);
    if (!m.block) return nt ? fwd_v<T, VEC, 1, false, (VEC > 1)>(p, m, stream) : fwd_v<T, VEC, 1, false, false>(p, m, stream);
    switch (lane_vectors(m)) {
    case 1: return fwd_v<T, VEC, 1, true, false>(p, m, stream);
    case 2: return fwd_v<T, VEC, 2, true, false>(p, m, stream);
    case 4: return fwd_v<T, VEC, 4, true, false>(p, m, stream);
    default:
        norm_fwd_long_kernel<T><<<grid_of((int64_t)p.B * p.T * p.G), 256, 0, stream>>>(p);
        return hipGetLastError();
    }
}

template <typename T>
hipError_t fwd_t(const NormProblem& p, hipStream_t stream)
{
    constexpr int wide = 16 / sizeof(T);
    return vec_of(p, false) == wide ? fwd_vec<T, wide>(p, stream) : fwd_vec<T, 1>(p, stream);
}

}  // namespace

size_t norm_workspace(const NormProblem& p) { return p.sequence ? seq_workspace(p) : 0; }

hipError_t launch_norm_fwd(const NormProblem& p, hipStream_t stream)
{
    if (p.sequence) return launch_seq_fwd(p, stream);
    return p.bf16 ? fwd_t<bf16>(p, stream) : fwd_t<float>(p, stream);
}

}  // namespace tfla
