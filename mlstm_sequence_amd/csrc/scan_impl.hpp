// scan_impl.hpp -- what the selective scan's forward and backward kernels
// share.
//
//   delta_t = softplus(dt_t + dt_bias),   a_t = exp(delta_t A[c,n])
//   h_t = a_t h_{t-1} + delta_t x_t B_t[n],   y_t = sum_n C_t[n] h_t + skip x_t
//
// Lanes are channels: a workgroup owns 64 channels of one group and a segment
// of one sequence, and its W waves split the N states, kStates to a wave, held
// in fp32 registers along the whole walk.  B_t and C_t are then the same for
// every lane of a wave: one LDS read of four values serves 64 x 4 states.
// What belongs to a channel and a step alone (softplus, the gate, their
// gradients) is done once, by the wave that owns the step in the tile, and
// handed to the others through LDS.
#pragma once

#include "act.hpp"
#include "blocks.hpp"

namespace tfla {
namespace scan {

constexpr int kStates = 4;    // states of a wave

typedef f32x4 f32x4u __attribute__((aligned(4)));   // four states of the caller's arrays

// ns <= kStates states of a channel, the rest 0 (ns <= 0: none).
__device__ __forceinline__ f32x4 load_states(const float* p, int ns)
{
    f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
    if (ns == kStates) v = *(const f32x4u*)p;
    else
        for (int n = 0; n < kStates - 1; ++n)
            if (n < ns) v[n] = p[n];
    return v;
}
__device__ __forceinline__ void store_states(float* p, int ns, f32x4 v)
{
    if (ns == kStates) *(f32x4u*)p = v;
    else
        for (int n = 0; n < kStates - 1; ++n)
            if (n < ns) p[n] = v[n];
}

__device__ __forceinline__ int clamp_len(const int* lengths, int b, int T)
{
    return lengths ? min(max(lengths[b], 0), T) : T;
}

// A lane's element of each tile's B or C, tile after tile: `at` its row of the tile fetched next, `last` the
// segment's last row, read in the place of rows behind it.  Stepping the pointer costs a quarter of the 64-bit
// product that a row number would need in every tile.
template <typename T> struct MatCursor {
    const T *at, *last;
    int64_t step;      // elements from tile to tile
    int s;             // the element's step within a tile
    // element (b, first + t0 + s, column): `first` the segment's first row, tiles from t0 on, `tile` steps apart
    __device__ __forceinline__ void set(const Rows& m, int b, int first, int column, int step_of, int t0, int tile, int len)
    {
        const T* base = (const T*)m.p + b * m.batch + first * m.row + column;
        s = step_of;
        at = base + (int64_t)(t0 + s) * m.row;
        last = base + (int64_t)max(len - 1, 0) * m.row;
        step = tile * m.row;
    }
    __device__ __forceinline__ T next(int t0, int len)
    {
        const T v = *(t0 + s < len ? at : last);
        at += step;
        return v;
    }
};

// How a sequence is cut: nseg segments of len steps (a multiple of the tile),
// walked by workgroups of their own.
struct Segments {
    int len, nseg;
};

// Where a workgroup stands: sequence, segment, channels, states.
struct Place {
    int b, seg, g, cb, lane, wave, c;   // c: the lane's channel (clamped to a valid one when !live)
    bool live;
    int blk;                            // block of channels within the sequence
};

__device__ __forceinline__ Place place(const ScanProblem& p, const Segments& sg)
{
    Place q;
    const int per = p.D / p.G;
    const int ncb = (per + 63) / 64;
    int i = blockIdx.x;
    q.blk = i % (ncb * p.G);
    i /= ncb * p.G;
    q.seg = i % sg.nseg;
    q.b = i / sg.nseg;
    q.cb = q.blk % ncb;
    q.g = q.blk / ncb;
    q.lane = threadIdx.x & 63;
    q.wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int k = q.cb * 64 + q.lane;
    q.live = k < per;
    q.c = q.g * per + min(k, per - 1);
    return q;
}

inline int waves_of(int N)
{
    const int w = (N + kStates - 1) / kStates;
    return w <= 1 ? 1 : w <= 2 ? 2 : w <= 4 ? 4 : w <= 8 ? 8 : 16;
}

inline int channel_blocks(const ScanProblem& p) { return p.G * ((p.D / p.G + 63) / 64); }

}  // namespace scan
}  // namespace tfla
