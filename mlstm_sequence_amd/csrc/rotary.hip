// rotary.hip -- rotary positions of queries and keys.
//
//   th = pos freq_j,  a' = scale (a cos th - b sin th),  b' = scale (b cos th + a sin th)
//
// Angles are formed and reduced in 64 bits: at position 10^6 and frequency 1
// an angle in fp32 is off by 0.03.  The remainder, at most an eighth of a
// turn, is small enough for the first terms of the series of sine and cosine
// in fp32.
//
// A token's angles serve all its heads: a workgroup forms those of its tokens
// once into LDS, and its threads then turn units of two vectors, a pair's two
// halves, of one head and token after another.  Bound by memory, each element
// read and written once: B=8 T=4096, 32 + 32 heads of 128 in bf16 into
// head-major outputs, 1.07 GB in 202 us (5.3 TB/s; a copy moves 5.0), backward
// B=1 T=65536 671 MB in 121 us (5.5).  Accesses past the caches gained nothing
// (210 to 216 us, when that case took 210; backward 139 to 189 for 128).
#include "gfx950.hpp"

#include "blocks.hpp"

namespace tfla {
namespace {

// scale cos(pos freq), scale sin(pos freq).  n quarter turns go from the angle in two parts of pi / 2; of the series
// the first term left out is below 2^-29 at pi / 4.
__device__ __forceinline__ f32x2 turn(double pos, double freq, float scale, bool inverse)
{
    const double a = pos * freq;
    const double n = rint(a * 0.63661977236758134308);                   // 2 / pi
    const double r = fma(-n, 6.123233995736766036e-17, fma(-n, 1.57079632679489661923, a));
    const float x = (float)r, y = x * x;
    const float s = x * fmaf(y, fmaf(y, fmaf(y, fmaf(y, 2.7557319e-6f, -1.9841270e-4f), 8.3333333e-3f), -1.6666667e-1f), 1.0f);
    const float c = fmaf(y, fmaf(y, fmaf(y, fmaf(y, fmaf(y, -2.7557319e-7f, 2.4801587e-5f), -1.3888889e-3f), 4.1666667e-2f), -0.5f), 1.0f);
    const int q = (int)(int64_t)n & 3;
    const float cs = q & 1 ? s : c, sn = q & 1 ? c : s;
    const float co = (q == 1 || q == 2) ? -cs : cs, si = q >= 2 ? -sn : sn;
    return f32x2{scale * co, scale * (inverse ? -si : si)};
}

__device__ __forceinline__ double position(const RotaryProblem& p, int b, int t)
{
    if (p.positions) return (double)p.positions[b * p.positions_batch + t];
    return (double)((int64_t)t + (p.start ? p.start[b] : 0));
}

// P elements as they lie in memory
template <typename T, int P> struct Pack {
    typedef T vec __attribute__((ext_vector_type(P)));
    vec v;
    __device__ __forceinline__ void load(const T* p) { v = *(const vec*)p; }
    __device__ __forceinline__ void store(T* p) const { *(vec*)p = v; }
    __device__ __forceinline__ float get(int i) const { return to_float((T)v[i]); }
    __device__ __forceinline__ void set(int i, float x) { v[i] = from_float<T>(x); }
};
template <typename T> struct Pack<T, 1> {
    T v;
    __device__ __forceinline__ void load(const T* p) { v = *p; }
    __device__ __forceinline__ void store(T* p) const { *p = v; }
    __device__ __forceinline__ float get(int) const { return to_float(v); }
    __device__ __forceinline__ void set(int, float x) { v = from_float<T>(x); }
};

// n / d for n below 2^31 (T. Granlund and P. Montgomery, "Division by invariant integers using multiplication", 1994)
struct Divisor {
    unsigned d, mul, shift;
};
Divisor divisor(unsigned d)
{
    unsigned s = 0;
    while ((uint64_t(1) << s) < d) ++s;
    return Divisor{d, (unsigned)(((uint64_t(1) << 32) * ((uint64_t(1) << s) - d)) / d + 1), s};
}
__device__ __forceinline__ unsigned quotient(unsigned n, const Divisor& v) { return (__umulhi(n, v.mul) + n) >> v.shift; }

// A head is cut into units of two vectors of P elements: the partners of P pairs, then what passes.
struct Geom {
    Divisor units, heads, kheads;
    int turned;           // units that turn
    int tok;              // tokens of a workgroup
    int tiles;            // of a sequence
};

constexpr int kEntries = 4096;   // angles of a workgroup's tokens, 32 KB
constexpr int kAhead = 2;        // units whose loads a thread has under way together (four: B=4 T=512 16 + 4 heads 8.4 us for 7.2)

template <typename T, int P, bool INTER>
__global__ __launch_bounds__(256) void rotary_kernel(RotaryProblem p, Geom gm)
{
    extern __shared__ f32x2 table[];                   // [tok][R / 2]: scale cos, scale sin
    const int64_t id = block_id();
    if (id >= (int64_t)p.B * gm.tiles) return;
    const int b = (int)(id / gm.tiles), t0 = (int)(id % gm.tiles) * gm.tok, nt = min(gm.tok, p.T - t0);
    const int len = p.lengths ? min(max(p.lengths[b] - t0, 0), nt) : nt;   // valid tokens here
    const int pairs = p.R / 2;
    for (int e = threadIdx.x; e < len * pairs; e += 256)
        table[e] = turn(position(p, b, t0 + e / pairs), p.freqs[e % pairs], p.scale, p.inverse);
    __syncthreads();
    auto tensor = [&](const Heads& in, const Heads& out, const Divisor& heads) {
        const T* x = (const T*)in.p + b * in.batch + t0 * in.row;
        T* y = (T*)out.p + b * out.batch + t0 * out.row;
        const unsigned n = (unsigned)nt * heads.d * gm.units.d;
        for (unsigned e0 = threadIdx.x; e0 < n; e0 += 256 * kAhead) {
            Pack<T, P> va[kAhead], vb[kAhead];
            int ca[kAhead], cb[kAhead], tk[kAhead], un[kAhead], hd[kAhead];
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                const unsigned e = min(e0 + 256 * i, n - 1), r = quotient(e, gm.units);
                un[i] = e - r * gm.units.d;
                tk[i] = quotient(r, heads);
                hd[i] = r - tk[i] * heads.d;
                const bool turned = un[i] < gm.turned;
                ca[i] = turned ? (INTER ? 2 * un[i] * P : un[i] * P) : p.R + (un[i] - gm.turned) * 2 * P;
                cb[i] = turned && !INTER ? ca[i] + pairs : ca[i] + P;
                const T* at = x + tk[i] * in.row + hd[i] * in.group;
                va[i].load(at + ca[i]);
                vb[i].load(at + min(cb[i], p.C - P));  // the last unit that passes may hold one vector
            }
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                if (un[i] < gm.turned) {
                    const f32x2* w = table + tk[i] * pairs + un[i] * P;
                    float oa[P], ob[P];
#pragma unroll
                    for (int k = 0; k < P; ++k) {
                        const f32x2 cs = w[k];
                        const float a = INTER && P > 1 ? (2 * k < P ? va[i].get(2 * k % P) : vb[i].get(2 * k % P)) : va[i].get(k);
                        const float c = INTER && P > 1 ? (2 * k < P ? va[i].get((2 * k + 1) % P) : vb[i].get((2 * k + 1) % P)) : vb[i].get(k);
                        oa[k] = a * cs[0] - c * cs[1];
                        ob[k] = c * cs[0] + a * cs[1];
                    }
#pragma unroll
                    for (int k = 0; k < P; ++k) {
                        if (INTER && P > 1) {
                            if (2 * k < P) {
                                va[i].set(2 * k % P, oa[k]);
                                va[i].set((2 * k + 1) % P, ob[k]);
                            } else {
                                vb[i].set(2 * k % P, oa[k]);
                                vb[i].set((2 * k + 1) % P, ob[k]);
                            }
                        } else {
                            va[i].set(k, oa[k]);
                            vb[i].set(k, ob[k]);
                        }
                    }
                }
                if (tk[i] >= len)
#pragma unroll
                    for (int k = 0; k < P; ++k) {
                        va[i].set(k, 0.0f);
                        vb[i].set(k, 0.0f);
                    }
                if (e0 + 256 * i < n) {
                    T* at = y + tk[i] * out.row + hd[i] * out.group;
                    va[i].store(at + ca[i]);
                    if (cb[i] < p.C) vb[i].store(at + cb[i]);
                }
            }
        }
    };
    tensor(p.q, p.q_out, gm.heads);
    if (p.Hk) tensor(p.k, p.k_out, gm.kheads);
}

template <typename T, int P>
hipError_t launch_p(const RotaryProblem& p, hipStream_t stream)
{
    Geom g;
    const int turned = p.R / 2 / P, passing = (p.C - p.R + 2 * P - 1) / (2 * P);
    g.units = divisor((unsigned)(turned + passing));
    g.heads = divisor((unsigned)p.H);
    g.kheads = divisor((unsigned)(p.Hk > 0 ? p.Hk : 1));
    g.turned = turned;
    // a workgroup's tokens: as many as two units to a thread take (eight: B=8 T=4096 32 + 32 heads of 128 bf16 210 us for
    // 202, backward B=1 T=65536 128 for 121), but 256 workgroups before that (B=1 T=4096 1 + 1 heads of 64: 4.4 us, without 6.4)
    const int64_t per = (int64_t)(turned + passing) * (p.H + p.Hk);
    int64_t tok = 512 / per;
    if (tok > (int64_t)p.B * p.T / 256) tok = (int64_t)p.B * p.T / 256;
    if (p.R && tok > kEntries / (p.R / 2)) tok = kEntries / (p.R / 2);
    if (tok > p.T) tok = p.T;
    if (tok < 1) tok = 1;
    g.tok = (int)tok;
    g.tiles = (p.T + g.tok - 1) / g.tok;
    const dim3 grid = grid_of((int64_t)p.B * g.tiles);
    const size_t lds = (size_t)g.tok * (p.R / 2) * sizeof(f32x2);
    if (p.interleaved) rotary_kernel<T, P, true><<<grid, 256, lds, stream>>>(p, g);
    else rotary_kernel<T, P, false><<<grid, 256, lds, stream>>>(p, g);
    return hipGetLastError();
}

bool fits(const Heads& h, const RotaryProblem& p, int n, size_t bytes)
{
    const int64_t e = p.bf16 ? 2 : 4, s = (int64_t)bytes;
    return !h.p || ((uintptr_t)h.p % bytes == 0 && (p.B == 1 || h.batch * e % s == 0) && (p.T == 1 || h.row * e % s == 0) &&
                    (n == 1 || h.group * e % s == 0));
}

// Elements of a vector: the most, up to 16 bytes, that divide the pairs and the channels and that addresses and
// strides allow (B=1 T=65536 16 + 2 heads of 128 bf16: 109 us, 8 bytes 152; 32 + 32 heads of B=8 T=4096 199 and 192).
int vector_of(const RotaryProblem& p)
{
    const int e = p.bf16 ? 2 : 4;
    for (int v = 16 / e; v > 1; v /= 2)
        if (p.R / 2 % v == 0 && p.C % v == 0 && fits(p.q, p, p.H, v * e) && fits(p.q_out, p, p.H, v * e) &&
            fits(p.k, p, p.Hk, v * e) && fits(p.k_out, p, p.Hk, v * e))
            return v;
    return 1;
}

template <typename T>
hipError_t launch_t(const RotaryProblem& p, hipStream_t stream)
{
    switch (vector_of(p)) {
    case 8: return launch_p<T, 16 / sizeof(T)>(p, stream);
    case 4: return launch_p<T, 4>(p, stream);
    case 2: return launch_p<T, 2>(p, stream);
    default: return launch_p<T, 1>(p, stream);
    }
}

}  // namespace

hipError_t launch_rotary(const RotaryProblem& p, hipStream_t stream)
{
    return p.bf16 ? launch_t<bf16>(p, stream) : launch_t<float>(p, stream);
}

}  // namespace tfla
