// rotary.hip -- rotary positions of queries and keys.
//
//   th = pos freq_j,  a' = scale (a cos th - b sin th),  b' = scale (b cos th + a sin th)
//
// Angles are formed and reduced in 64 bits: at position 10^6 and frequency 1
// an angle in fp32 is off by 0.03.  The remainder, at most an eighth of a
// turn, is small enough for the first terms of the series of sine and cosine
// in fp32.
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

// A thread to a pair, or to a channel behind R.
template <typename T>
__global__ __launch_bounds__(256) void rotary_kernel(RotaryProblem p)
{
    const int per = p.R / 2 + (p.C - p.R), heads = p.H + p.Hk;
    const int64_t i = block_id() * 256 + threadIdx.x;
    if (i >= (int64_t)p.B * p.T * heads * per) return;
    const int u = (int)(i % per);
    int64_t r = i / per;
    const int head = (int)(r % heads);
    r /= heads;
    const int b = (int)(r / p.T), t = (int)(r % p.T);
    const bool key = head >= p.H;
    const Heads &in = key ? p.k : p.q, &out = key ? p.k_out : p.q_out;
    const int g = key ? head - p.H : head;
    const T* x = (const T*)in.p + b * in.batch + t * in.row + g * in.group;
    T* y = (T*)out.p + b * out.batch + t * out.row + g * out.group;
    const bool live = !p.lengths || t < p.lengths[b];
    if (u >= p.R / 2) {
        const int c = p.R / 2 + u;
        y[c] = live ? x[c] : from_float<T>(0.0f);
        return;
    }
    const int ca = p.interleaved ? 2 * u : u, cb = p.interleaved ? 2 * u + 1 : u + p.R / 2;
    const f32x2 w = turn(position(p, b, t), p.freqs[u], p.scale, p.inverse);
    const float a = to_float(x[ca]), c = to_float(x[cb]);
    y[ca] = from_float<T>(live ? a * w[0] - c * w[1] : 0.0f);
    y[cb] = from_float<T>(live ? c * w[0] + a * w[1] : 0.0f);
}

template <typename T>
hipError_t launch_t(const RotaryProblem& p, hipStream_t stream)
{
    const int64_t n = (int64_t)p.B * p.T * (p.H + p.Hk) * (p.R / 2 + (p.C - p.R));
    rotary_kernel<T><<<grid_of((n + 255) / 256), 256, 0, stream>>>(p);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_rotary(const RotaryProblem& p, hipStream_t stream)
{
    return p.bf16 ? launch_t<bf16>(p, stream) : launch_t<float>(p, stream);
}

}  // namespace tfla
