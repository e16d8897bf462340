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

// f alone.
template <typename T, int KIND> __device__ __forceinline__ float forget_of(float u, float decay)
{
    if (KIND == kCoupled) return __builtin_amdgcn_rcpf(1.0f + exp_t<T>(-u));
    const float r = sigmoid_t<T>(u);
    return KIND == kSigmoid ? r : exp_t<T>(-(decay * r));
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

// ---- tiles ---------------------------------------------------------------------------
//
// A workgroup owns 64 neighbouring channels of a sequence and walks their rows in
// tiles of 8 waves times PER rows; a lane holds V neighbouring channels and
// PER / V consecutive rows (64 / V lanes across a row).

constexpr int kWaves = 8;

template <int BYTES> struct RawOf;
template <> struct RawOf<2> { typedef unsigned short type; };
template <> struct RawOf<4> { typedef unsigned type; };
template <> struct RawOf<8> { typedef unsigned type __attribute__((ext_vector_type(2))); };

// V elements as they were loaded, and back.
template <typename T, int V> __device__ __forceinline__ void decode(typename RawOf<sizeof(T) * V>::type raw, float* o)
{
    typedef T vec __attribute__((ext_vector_type(V)));
    if constexpr (V == 1) {
        o[0] = to_float(__builtin_bit_cast(T, raw));
    } else {
        const vec v = __builtin_bit_cast(vec, raw);
#pragma unroll
        for (int k = 0; k < V; ++k) o[k] = to_float((T)v[k]);
    }
}
template <typename T, int V> __device__ __forceinline__ typename RawOf<sizeof(T) * V>::type encode(const float* x)
{
    typedef T vec __attribute__((ext_vector_type(V)));
    typedef typename RawOf<sizeof(T) * V>::type raw;
    if constexpr (V == 1) {
        return __builtin_bit_cast(raw, from_float<T>(x[0]));
    } else {
        vec v;
#pragma unroll
        for (int k = 0; k < V; ++k) v[k] = from_float<T>(x[k]);
        return __builtin_bit_cast(raw, v);
    }
}

// A lane's place in a tile.
struct Lane {
    int row;        // its first row
    int c;          // its first channel
    bool live;      // whether that is one
    int last;       // the last channel's vector, read in the place of those behind it
};

// A uniform value that the compiler takes for a new one in every tile: a lane's offsets of all rows of all tensors,
// kept in registers along the walk, would take more of them than the tile's values.
__device__ __forceinline__ unsigned hidden(unsigned x)
{
    asm volatile("" : "+s"(x));
    return x;
}

// The rows of a tensor that a workgroup walks.  BUF: by buffer instructions, whose bounds check makes rows behind the
// tile's last valid one, and channels behind the last, read as 0 and never written, at one 32-bit addition a row;
// else by 64-bit addresses held inside the tensor (rows further apart than a buffer spans, or sharing memory).
template <typename T, int V, bool BUF> struct Walk {
    typedef typename RawOf<sizeof(T) * V>::type raw;
    char* base;      // row 0 of the walk, channel 0
    int64_t row;     // bytes
    unsigned at;     // BUF: the lane's offset within a tile
    __device__ __forceinline__ void open(const Rows& m, int64_t b, int64_t first, const Lane& l)
    {
        row = m.row * (int64_t)sizeof(T);
        base = (char*)m.p + (b * m.batch + first * m.row) * (int64_t)sizeof(T);
        at = l.live ? (unsigned)(l.row * row) + (unsigned)l.c * (unsigned)sizeof(T) : 0x80000000u;
    }
    // N rows of the tile at t0, of which `rows` are valid (may be <= 0); end: rows of the walk
    template <int N> __device__ __forceinline__ void load(raw* o, int t0, int rows, int end, const Lane& l) const
    {
        if constexpr (BUF) {
            const auto rs = __builtin_amdgcn_make_buffer_rsrc(base + t0 * row, 0, (int)(max(rows, 0) * row), 0x27000);
            const unsigned step = hidden((unsigned)row);
            unsigned v = at;
#pragma unroll
            for (int r = 0; r < N; ++r, v += step) {
                if constexpr (sizeof(raw) == 2) o[r] = __builtin_amdgcn_raw_buffer_load_b16(rs, v, 0, 0);
                else if constexpr (sizeof(raw) == 4) o[r] = __builtin_amdgcn_raw_buffer_load_b32(rs, v, 0, 0);
                else o[r] = __builtin_bit_cast(raw, __builtin_amdgcn_raw_buffer_load_b64(rs, v, 0, 0));
            }
        } else {
            const char* p = base + (int64_t)min(l.c, l.last) * (int64_t)sizeof(T);
#pragma unroll
            for (int r = 0; r < N; ++r) o[r] = *(const raw*)(p + min(t0 + l.row + r, end - 1) * row);
        }
    }
    __device__ __forceinline__ void store(raw v, int r, int t0, int rows, const Lane& l) const
    {
        if constexpr (BUF) {
            const auto rs = __builtin_amdgcn_make_buffer_rsrc(base + t0 * row, 0, (int)(rows * row), 0x27000);
            const unsigned o = at + r * hidden((unsigned)row);
            if constexpr (sizeof(raw) == 2) __builtin_amdgcn_raw_buffer_store_b16(v, rs, o, 0, 0);
            else if constexpr (sizeof(raw) == 4) __builtin_amdgcn_raw_buffer_store_b32(v, rs, o, 0, 0);
            else {
                typedef int i32x2 __attribute__((ext_vector_type(2)));
                __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(i32x2, v), rs, o, 0, 0);
            }
        } else if (l.live && l.row + r < rows) {
            *(raw*)(base + (t0 + l.row + r) * row + (int64_t)l.c * (int64_t)sizeof(T)) = v;
        }
    }
    // Zeros in rows [from, to) of 64 channels from c0 on, by the whole workgroup.
    __device__ __forceinline__ void clear(int from, int to, int c0, int D) const
    {
        const int c = c0 + (threadIdx.x & 63);
        if (c >= D) return;
        for (int64_t t = from + (int)(threadIdx.x >> 6); t < to; t += kWaves) *(T*)(base + t * row + c * (int64_t)sizeof(T)) = from_float<T>(0.0f);
    }
};

// Whether a tensor's rows can be walked by buffer instructions in tiles of `tile` rows, and lie at multiples of `bytes`.
inline bool walks(const Rows& m, const DiagProblem& p, int tile)
{
    const int64_t row = m.row * (p.bf16 ? 2 : 4);
    return !m.p || (m.row >= p.D && row <= ((int64_t(1) << 31) - 1) / tile);
}
inline bool aligned(const Rows& m, const DiagProblem& p, size_t bytes)
{
    const size_t e = p.bf16 ? 2 : 4;
    return !m.p || ((uintptr_t)m.p % bytes == 0 && (p.B == 1 || m.batch * e % bytes == 0) && (p.T == 1 || m.row * e % bytes == 0));
}

// The value of the lower and of the upper half of the wave, in every lane.
__device__ __forceinline__ void halves(float v, float* low, float* high)
{
    const unsigned u = __builtin_bit_cast(unsigned, v);
    const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    const unsigned a = r[0], b = r[1];
    *low = __builtin_bit_cast(float, a);
    *high = __builtin_bit_cast(float, b);
}

// How a sequence is cut: nseg segments of len rows (whole chunks), walked by workgroups of their own.
struct Segments {
    int len, nseg, ncb;
};

struct Place {
    int seg, cb;
    int64_t b;
};
__device__ __forceinline__ bool place(const DiagProblem& p, const Segments& sg, Place* q)
{
    int64_t i = block_id();
    q->cb = (int)(i % sg.ncb);
    i /= sg.ncb;
    q->seg = (int)(i % sg.nseg);
    q->b = i / sg.nseg;
    return q->b < p.B;
}

template <int V, int PER> __device__ __forceinline__ Lane lane_of(const DiagProblem& p, const Place& q, int* half)
{
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    *half = lane / (64 / V);
    Lane l;
    l.row = wave * PER + *half * (PER / V);
    l.c = q.cb * 64 + lane % (64 / V) * V;
    l.live = l.c < p.D;
    l.last = p.D - V;
    return l;
}

inline Segments segments_of(const DiagProblem& p, int tile)
{
    Segments s;
    s.ncb = (p.D + 63) / 64;
    const int64_t blocks = (int64_t)p.B * s.ncb;
    const int tiles = (p.T + tile - 1) / tile;
    int64_t n = blocks >= 256 ? 1 : 512 / blocks;
    if (n > tiles) n = tiles;
    const int per = (int)((tiles + n - 1) / n);
    s.len = per * tile;
    s.nseg = (tiles + per - 1) / per;
    return s;
}

inline size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

// The segments' sums, [B][nseg][D] pairs, at the start of the workspace.
inline size_t ends_bytes(const DiagProblem& p, const Segments& s)
{
    return s.nseg > 1 ? align256((size_t)p.B * s.nseg * p.D * sizeof(f32x2)) : 0;
}

}  // namespace diag
}  // namespace tfla
