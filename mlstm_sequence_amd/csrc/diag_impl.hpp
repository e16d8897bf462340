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

// 1 - f^2 = 1 - e^{-z}, z = 2 w: below 0.4, where the difference would cancel, z times a polynomial of degree 4 fitted
// to (1 - e^{-z}) / z on [0, 0.4] (Chebyshev nodes).  The fit is off by 0.9 half steps at most, its value in fp32 by 1.6
// and the product by 2.4 (the worst of five million z).
__device__ __forceinline__ float one_minus_square(float z, float f)
{
    float s = fmaf(z, 7.0668478e-3f, -4.1237194e-2f);
    s = fmaf(z, s, 1.6660628e-1f);
    s = fmaf(z, s, -4.9999702e-1f);
    s = fmaf(z, s, 1.0f);
    return z < 0.4f ? z * s : fmaf(-f, f, 1.0f);
}

// A channel's decay and what the steps need of it.
struct Rate {
    float decay, twice, log2;
    __device__ __forceinline__ explicit Rate(float d = 0.0f) : decay(d), twice(2.0f * d), log2(-d * kLog2e) {}
};

template <typename T> __device__ __forceinline__ float decayed(float r, const Rate& d)
{
    return sizeof(T) == 2 ? exp2_fast(d.log2 * r) : exp_f(-(d.decay * r));
}

// The gates of a step; r = s(u), s = s(v) and m where the kind has them.
struct Gate {
    float f, i, r, s, m;
};

template <typename T, int KIND> __device__ __forceinline__ Gate gate_of(float u, float v, const Rate& d)
{
    Gate g;
    if (KIND == kCoupled) {
        const float e = exp_t<T>(-u);
        g.f = __builtin_amdgcn_rcpf(1.0f + e);
        // 1 - f without its cancellation; from e = 2^25 on it rounds to 1, and above 2^126, where the reciprocal is below
        // the smallest normal number, v_rcp_f32 gives f = 0, of which e f would make 0 (of an infinite e NaN)
        g.i = e >= 0x1p60f ? 1.0f : e * g.f;
    } else {
        g.s = sigmoid_t<T>(v);
        g.r = sigmoid_t<T>(u);
        if (KIND == kSigmoid) {
            g.f = g.r;
            g.i = g.s;
        } else {
            g.f = decayed<T>(g.r, d);
            g.m = __builtin_amdgcn_sqrtf(one_minus_square(d.twice * g.r, g.f));
            g.i = g.m * g.s;
        }
    }
    return g;
}

// f alone.
template <typename T, int KIND> __device__ __forceinline__ float forget_of(float u, const Rate& d)
{
    if (KIND == kCoupled) return __builtin_amdgcn_rcpf(1.0f + exp_t<T>(-u));
    const float r = sigmoid_t<T>(u);
    return KIND == kSigmoid ? r : decayed<T>(r, d);
}

struct GateGrads {
    float dx, du, dv, dd;
};

// Gradients of a step from its gates, x, the state before it and g.
template <int KIND> __device__ __forceinline__ GateGrads grads_of(const Gate& k, float x, float before, float g, const Rate& d)
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
        o.du = o.dd * d.decay * (1.0f - k.r);
        o.dv = di * k.i * (1.0f - k.s);
    }
    return o;
}

// ---- tiles ---------------------------------------------------------------------------
//
// A workgroup owns CH neighbouring channels of a sequence and walks their rows in
// tiles; a lane holds 16 consecutive rows of a channel, CH lanes side by side make
// a row group, the wave's groups and the eight waves follow each other in time.
// CH is 64, or 32 or 16 for more workgroups (cut_of), whose neighbours share lines:
// they are put on one XCD, whose L2 reads a line once for them.  (Two channels and
// eight rows to a lane: 3 to 7 % slower backward, whose registers they take, equal
// forward; 16 waves to a tile instead of eight 7 %.)
//
// Rows that begin off the lines (D=4097) make all neighbours share them: eight of
// 64 channels then go to an XCD, through the caches (B=4 T=4096 D=4097 bf16 with a
// decay: forward 204 us, backward 356, as rows on lines 253 and 643; fp32 coupled
// 241 and 398, 258 and 535).

constexpr int kWaves = 8;
constexpr int kRows = 16;                                 // of a lane
constexpr int kGroup = 2;                                 // rows whose gates a lane forms together
constexpr int kStreamed = 2;                              // of a buffer access: past the caches (nt)

template <int CH> struct Shape {
    static constexpr int groups = 64 / CH;                // row groups of a wave
    static constexpr int rows = groups * kRows;           // of a wave
    static constexpr int tile = kWaves * rows;
};
static_assert(Shape<64>::tile == kChunk && Shape<16>::tile == 4 * kChunk, "a tile starts where the forward pass leaves a state");

// A lane's place in a tile.
struct Lane {
    int row;        // its first row
    int c;          // its channel
    bool live;      // whether that is one
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
// AUX: the buffer accesses' cache policy.
template <typename T, bool BUF, int AUX> struct Walk {
    char* base = nullptr;   // row 0 of the walk, channel 0
    int64_t row = 0;        // bytes
    unsigned at = 0;        // BUF: the lane's offset within a tile
    int c = 0;              // else the channel, one inside the tensor
    __device__ __forceinline__ void open(const Rows& m, int64_t b, int64_t first, const Lane& l, int D)
    {
        row = m.row * (int64_t)sizeof(T);
        base = (char*)m.p + (b * m.batch + first * m.row) * (int64_t)sizeof(T);
        at = l.live ? (unsigned)(l.row * row) + (unsigned)l.c * (unsigned)sizeof(T) : 0x80000000u;
        c = min(l.c, D - 1);
    }
    // A tile of the walk: the rows from t0 on, of which `rows` are valid (may be <= 0); end: rows of the walk, >= 1
    // where anything is loaded.
    struct Tile {
        decltype(__builtin_amdgcn_make_buffer_rsrc((void*)nullptr, 0, 0, 0)) rs;
        unsigned step;
        int t0, rows, end;
    };
    __device__ __forceinline__ Tile tile(int t0, int rows, int end) const
    {
        Tile o;
        if constexpr (BUF) {
            // the clamp of a uniform value is done by a vector instruction; a descriptor in vector registers would make
            // every load a loop over its lanes' descriptors
            const int valid = __builtin_amdgcn_readfirstlane(max(rows, 0));
            o.rs = __builtin_amdgcn_make_buffer_rsrc(base + t0 * row, 0, (int)(valid * row), 0x27000);
            o.step = hidden((unsigned)row);
        }
        o.t0 = t0;
        o.rows = rows;
        o.end = end;
        return o;
    }
    __device__ __forceinline__ T load(const Tile& t, int r, const Lane& l) const
    {
        if constexpr (BUF) {
            const int o = (int)(at + r * t.step);
            if constexpr (sizeof(T) == 2) return __builtin_bit_cast(T, __builtin_amdgcn_raw_buffer_load_b16(t.rs, o, 0, AUX));
            else return __builtin_bit_cast(T, __builtin_amdgcn_raw_buffer_load_b32(t.rs, o, 0, AUX));
        } else {
            return *(const T*)(base + c * (int64_t)sizeof(T) + min(t.t0 + l.row + r, t.end - 1) * row);
        }
    }
    __device__ __forceinline__ void store(const Tile& t, float x, int r, const Lane& l) const
    {
        const T v = from_float<T>(x);
        if constexpr (BUF) {
            const int o = (int)(at + r * t.step);
            if constexpr (sizeof(T) == 2) __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(unsigned short, v), t.rs, o, 0, AUX);
            else __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(unsigned, v), t.rs, o, 0, AUX);
        } else if (l.live && l.row + r < t.rows) {
            *(T*)(base + c * (int64_t)sizeof(T) + (t.t0 + l.row + r) * row) = v;
        }
    }
    // Zeros in rows [from, to) of CH channels from c0 on, by the whole workgroup.
    template <int CH> __device__ __forceinline__ void clear(int from, int to, int c0, int D) const
    {
        const int k = c0 + (int)(threadIdx.x % CH);
        if (k >= D) return;
        for (int64_t t = from + (int)(threadIdx.x / CH); t < to; t += 64 * kWaves / CH)
            *(T*)(base + t * row + k * (int64_t)sizeof(T)) = from_float<T>(0.0f);
    }
};

// Whether a tensor's rows can be walked by buffer instructions: apart from each other, the longest tile below 2^31 bytes.
inline bool walks(const Rows& m, const DiagProblem& p)
{
    const int64_t row = m.row * (p.bf16 ? 2 : 4);
    return !m.p || (m.row >= p.D && row <= ((int64_t(1) << 31) - 1) / Shape<16>::tile);
}

// Whether a tensor's rows begin on lines of 128 bytes.
inline bool on_lines(const Rows& m, const DiagProblem& p)
{
    const int64_t e = p.bf16 ? 2 : 4;
    return !m.p || ((uintptr_t)m.p % 128 == 0 && (p.T == 1 || m.row * e % 128 == 0) && (p.B == 1 || m.batch * e % 128 == 0));
}

// The value of the lower and of the upper of the two lanes D apart (the one with bit D clear, and set), in both.
template <int D> __device__ __forceinline__ void pair_of(float v, float* low, float* high)
{
    const unsigned u = __builtin_bit_cast(unsigned, v);
    const auto r = D == 16 ? __builtin_amdgcn_permlane16_swap(u, u, false, false)
                           : __builtin_amdgcn_permlane32_swap(u, u, false, false);
    const unsigned x = r[0], y = r[1];
    *low = __builtin_bit_cast(float, x);
    *high = __builtin_bit_cast(float, y);
}

// Joins the row groups of a wave, D lanes apart and more: F, H go from the map of a lane's group to the wave's, pf, ph
// (1, 0 before) to the map of the groups before it.
template <int D> __device__ __forceinline__ void join(int lane, float* F, float* H, float* pf, float* ph)
{
    if constexpr (D < 64) {
        float lf, uf, lh, uh;
        pair_of<D>(*F, &lf, &uf);
        pair_of<D>(*H, &lh, &uh);
        const bool upper = lane & D;
        *ph += *pf * (upper ? lh : 0.0f);
        *pf *= upper ? lf : 1.0f;
        *F = lf * uf;
        *H = uf * lh + uh;
        join<2 * D>(lane, F, H, pf, ph);
    }
}
// The same with the adjoint's map a -> F a + A, qf, qa the map of the groups behind.
template <int D>
__device__ __forceinline__ void join_both(int lane, float* F, float* H, float* A, float* pf, float* ph, float* qf, float* qa)
{
    if constexpr (D < 64) {
        float lf, uf, lh, uh, la, ua;
        pair_of<D>(*F, &lf, &uf);
        pair_of<D>(*H, &lh, &uh);
        pair_of<D>(*A, &la, &ua);
        const bool upper = lane & D;
        *ph += *pf * (upper ? lh : 0.0f);
        *pf *= upper ? lf : 1.0f;
        *qa += *qf * (upper ? 0.0f : ua);
        *qf *= upper ? 1.0f : uf;
        *F = lf * uf;
        *H = uf * lh + uh;
        *A = lf * ua + la;
        join_both<2 * D>(lane, F, H, A, pf, ph, qf, qa);
    }
}

// F and A alone.
template <int D> __device__ __forceinline__ void join_behind(float* F, float* A)
{
    if constexpr (D < 64) {
        float lf, uf, la, ua;
        pair_of<D>(*F, &lf, &uf);
        pair_of<D>(*A, &la, &ua);
        *F = lf * uf;
        *A = lf * ua + la;
        join_behind<2 * D>(F, A);
    }
}
// The sum over the row groups.
template <int D> __device__ __forceinline__ float sum_groups(float v)
{
    if constexpr (D < 64) {
        float a, b;
        pair_of<D>(v, &a, &b);
        return sum_groups<2 * D>(a + b);
    }
    return v;
}

constexpr int kNear = 8;   // 16: within 4 %, but long few channels (B=12 T=15822 D=158 fp32 backward 364, 378 us)

// How the work is cut: ncb blocks of ch channels, nseg segments of len rows (whole tiles), each walked by a workgroup
// of its own; `near` blocks share lines.
struct Cut {
    int ch, ncb, nseg, len, near;
    int64_t blocks;
};

struct Place {
    int seg, cb;
    int64_t b;
};
// Workgroups go to the eight XCDs in turn; neighbouring channels go to one of them.
__device__ __forceinline__ bool place(const DiagProblem& p, const Cut& cut, Place* q)
{
    const int64_t id = block_id(), k = id / 8;
    int64_t i = (k / cut.near * 8 + id % 8) * cut.near + k % cut.near;
    q->cb = (int)(i % cut.ncb);
    i /= cut.ncb;
    q->seg = (int)(i % cut.nseg);
    q->b = i / cut.nseg;
    return q->b < p.B;
}

template <int CH> __device__ __forceinline__ Lane lane_of(const DiagProblem& p, const Place& q)
{
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    Lane l;
    l.row = wave * Shape<CH>::rows + lane / CH * kRows;
    l.c = q.cb * CH + lane % CH;
    l.live = l.c < p.D;
    return l;
}

inline int64_t blocks_of(const DiagProblem& p, int ch) { return (int64_t)p.B * ((p.D + ch - 1) / ch); }

// The cut of a call whose tensors are walked by buffer instructions (buf), else by segments of 64 channels always.
//
// A CU holds one workgroup (two of the forward pass's coupled gates), so time goes with the rounds of 256 workgroups: 64
// channels to one where that gives more than 128 (B=5 T=3000 D=2048 bf16, coupled, forward and backward: 53 and 89 us,
// of 32 channels 75 and 126), 32 where it gives more than 64 (B=4 T=1000 D=2048: 14.6 and 20.6 us, two segments of 64
// channels 22.4 and 27.7) unless the backward pass is long and in bf16 (T=8000, a decay: 271 us, segments 240).  With
// fewer 16 where the axis is short (T=1000 D=2048: 8.1 and 14.1 us, segments 11.1 and 13.7; T=3000 20.6 and 30.1, 19.7
// and 22.4) or, forward in fp32, where they give 256 (B=2 T=8000 D=2048: 105 us, segments 120); else segments of 64, as
// many as one round takes (B=3 T=10825 D=722: 59 and 88 us, one more to each sequence, which opens a second round, 83 and
// 119).  A segmented walk reads the inputs twice, narrow blocks read lines that they share.
inline Cut cut_of(const DiagProblem& p, bool buf, bool bwd, bool lines = true)
{
    Cut c;
    c.ch = 64;
    const int64_t full = blocks_of(p, 64);
    if (buf && full <= 128) {
        if (full > 64) c.ch = bwd && p.bf16 && p.T > 2048 ? 64 : 32;
        else if (p.T <= (bwd ? 768 : 2048) || (!bwd && !p.bf16 && blocks_of(p, 16) >= 256)) c.ch = 16;
    }
    const bool narrow = c.ch != 64;
    c.ncb = (p.D + c.ch - 1) / c.ch;
    c.near = lines ? 64 / c.ch : kNear;
    const int tile = kWaves * kRows * 64 / c.ch;
    const int tiles = (p.T + tile - 1) / tile;
    const int64_t blocks = (int64_t)p.B * c.ncb;
    int64_t n = narrow || blocks > 128 ? 1 : 256 / blocks;
    if (n > 64) n = 64;                                // a segment's start folds the maps of those before it
    if (n > tiles) n = tiles;
    const int per = (int)((tiles + n - 1) / n);
    c.len = per * tile;
    c.nseg = (tiles + per - 1) / per;
    const int64_t g = 8 * c.near, all = blocks * c.nseg;
    c.blocks = (all + g - 1) / g * g;
    return c;
}

inline size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

// The segments' maps, [B][nseg][D] pairs, at the start of the workspace.
inline size_t ends_bytes(const DiagProblem& p, const Cut& c)
{
    return c.nseg > 1 ? align256((size_t)p.B * c.nseg * p.D * sizeof(f32x2)) : 0;
}

}  // namespace diag
}  // namespace tfla
