// scan_bwd.hip -- backward pass of the selective scan (scan_impl.hpp).
//
// With g_t the gradient of h_t and dy_t that of o_t (after the gate):
//
//   g_t = C_t dy_t + a_{t+1} g_{t+1}       w_t = g_t a_t h_{t-1}
//   dC_t[n] = sum_c dy_t h_t               dB_t[n] = sum_c g_t delta_t x_t
//   dx_t = delta_t sum_n g_t B_t + skip dy_t
//   ddelta_t = x_t sum_n g_t B_t + sum_n w_t A         dA = sum_t w_t delta_t
//
// Pass 1 walks every segment forward from a zero state and keeps the state
// and the sum of the steps at the start of each tile of kTile steps; with
// more than one segment it also forms, with the running product P of the
// decays, the adjoint that the segment hands to the one before it when it is
// handed none itself, sum_t P_t C_t dy_t.  Pass 2 (a thread a state) turns
// the segments' ends into their true start states and incoming adjoints.
// Pass 3 walks the tiles from the last to the first: it recomputes a tile's
// states and decays into registers (a state from a zero start needs
// exp(A sum delta) times the segment's true start added), then runs the
// adjoint back over them.  Sums over a wave's channels (dB, dC) go through
// lane swaps and adds, about two a value; each block of 64 channels writes
// its own sums, and pass 4 adds blocks, segments and sequences in a fixed
// order.
//
// The arithmetic bounds pass 3: of 106 issue slots that a wave spends on a
// step of its four states, about 20 recompute, 32 run the adjoint and 18 sum
// over the channels.  B=4 T=2048 D=4096 N=16 bf16 with a gate: 611 to 616 us
// for the call; profiled apart pass 1 takes 186 us with 88 % of the issue
// slots taken, pass 3 498 with 82 %.  Segments cost it next to nothing, so there are enough of
// them to fill the chip.  N above 32 takes 16 waves, which leaves each 128
// registers, 64 of them for a tile's states and decays: 44 to 53 values go to
// scratch within the walk, and the call takes 1.87 ps a state and step (B=2
// T=1024 D=1024 N=64: 251 us) where it takes 1.17 at N=32 (B=2 T=2048 D=2048:
// 315) and 1.14 at N=16.
#include "scan_impl.hpp"
#include "sums.hpp"

#include <type_traits>

namespace tfla {
namespace {

using namespace scan;

constexpr float kLn2 = 0.6931471805599453f;
constexpr int kVm0 = 0x0f70;   // s_waitcnt: no vector load outstanding
// Tiles whose inputs are under way: two, but one where the registers are short (16 waves: 128 each; one wave: a whole
// tile's steps to prepare), N=64 (B=2 T=1024 D=1024) 287 us with two against 253, N=4 (B=4 T=1024
// D=2048) 121 against 88.
constexpr int ahead(int W) { return W == 1 || W == 16 ? 1 : 2; }
constexpr int kTile = 8;       // steps of a tile: its states and decays take 16 registers a step pair

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

struct Ws {
    f32x4* tiles;        // [B][blocks][tiles][W][64]: states at the tiles' starts (from the segment's zero start)
    float* cums;         // [B][blocks][tiles][64]: sum of the segment's steps before the tile
    float *ends, *adj;   // [B][nseg][D][N]: end states and handed adjoints, then start states and incoming adjoints
    float* sums;         // [B][nseg][D]: sum of the segment's steps
    float *pb, *pc;      // [ncb][B][T][G][N]: dB, dC of one block of channels
    float* pa;           // [B][nseg][D][N]
    float *pskip, *pbias;   // [B][nseg][D]
    size_t bytes;
};

// Segments of whole tiles, 32 steps at least (B=3 T=619 D=1000 G=2 N=8: 51 us; 64 at least: 67, 16 at least: 47, but
// B=1 T=512 D=2048 N=16 52 for 47).  Two waves of pass 3 fit a SIMD (registers): from there on (2048) one segment,
// which saves pass 1 its adjoint (B=8 T=2048 D=4096 N=16: 1164 us against 1172 with four), below it enough for 4096
// waves (B=1 T=2048 D=2048 N=16: 107 us, for 8192 116, though B=4 T=2048 D=4096 gains, 608 for 617); 2048 where a
// wave is alone in its workgroup and fills a SIMD's registers (B=4 T=1024 D=2048 N=4: 88 us, with 4096 waves 93).
Segments segments_of(const ScanProblem& p)
{
    const int64_t waves = (int64_t)p.B * channel_blocks(p) * waves_of(p.N);
    const int tiles = (p.T + kTile - 1) / kTile;
    int64_t n = waves >= 2048 ? 1 : (waves_of(p.N) == 1 ? 2048 : 4096) / waves;
    if (n > p.T / 32) n = p.T / 32;
    if (n < 1) n = 1;
    const int per = (int)((tiles + n - 1) / n);
    return Segments{per * kTile, (tiles + per - 1) / per};
}

Ws layout(const ScanProblem& p, const Segments& sg, char* base)
{
    const int W = waves_of(p.N);
    const size_t blocks = (size_t)p.B * channel_blocks(p), nt = (p.T + kTile - 1) / kTile;
    const int ncb = (p.D / p.G + 63) / 64;
    const size_t bn = (size_t)p.B * sg.nseg * p.D;
    Ws w;
    size_t off = 0;
    auto take = [&](size_t bytes) {
        char* r = base + off;
        off += align256(bytes);
        return r;
    };
    w.tiles = (f32x4*)take(blocks * nt * W * 64 * 16);
    w.cums = (float*)take(blocks * nt * 64 * 4);
    w.ends = (float*)take(bn * p.N * 4);
    w.adj = (float*)take(bn * p.N * 4);
    w.sums = (float*)take(bn * 4);
    const size_t bc = (size_t)ncb * p.B * p.T * p.G * p.N * 4;
    w.pb = (float*)take(bc);
    w.pc = (float*)take(bc);
    w.pa = (float*)take(bn * p.N * 4);
    w.pskip = (float*)take(bn * 4);
    w.pbias = (float*)take(bn * 4);
    w.bytes = off;
    return w;
}

// What passes 1 and 3 share of a workgroup's setting.  A wave's own steps of
// a tile are own .. own + OWN - 1; with more waves than steps the waves behind
// the last step own none (and read along with the last).
template <typename T, int W> struct Walk {
    static constexpr int TS = kTile, OWN = TS >= W ? TS / W : 1, NP = W * kStates;
    static_assert(TS * 2 * NP == 64 * W, "one element of B and C to a thread and tile");
    Place q;
    int s0, s1, len, own, n0, ns;
    bool mine;                       // this wave owns steps
    int64_t nt;
    const T *xp, *dp, *zp, *gp, *mp;
    int64_t mr;
    int ms;
    bool mv;

    __device__ __forceinline__ Walk(const ScanProblem& p, const Segments& sg, bool with_dy) : q(place(p, sg))
    {
        const int all = clamp_len(p.lengths, q.b, p.T);
        s0 = q.seg * sg.len;
        s1 = min(s0 + sg.len, p.T);
        len = max(0, min(all, s1) - s0);
        mine = q.wave * OWN < TS;
        own = min(q.wave * OWN, TS - 1);
        n0 = q.wave * kStates;
        ns = min(kStates, p.N - n0);
        nt = (p.T + TS - 1) / TS;
        xp = (const T*)p.x.p + q.b * p.x.batch + s0 * p.x.row;
        dp = (const T*)p.dt.p + q.b * p.dt.batch + s0 * p.dt.row;
        zp = p.z.p ? (const T*)p.z.p + q.b * p.z.batch + s0 * p.z.row : nullptr;
        gp = with_dy ? (const T*)p.dy.p + q.b * p.dy.batch + s0 * p.dy.row : nullptr;
        // this thread's element of a tile's B and C: step, matrix, state in that order
        const int e = threadIdx.x, n = e % NP;
        const Rows& m = e / NP % 2 ? p.cmat : p.bmat;
        mv = n < p.N;
        ms = e / NP / 2;
        mr = m.row;
        mp = (const T*)m.p + q.b * m.batch + s0 * m.row + q.g * p.N + min(n, p.N - 1);
    }
    // the same, for tiles from t0 on, `tile` steps apart
    __device__ __forceinline__ MatCursor<T> matrices(const ScanProblem& p, int t0, int tile) const
    {
        const int e = threadIdx.x, n = e % NP;
        MatCursor<T> c;
        c.set(e / NP % 2 ? p.cmat : p.bmat, q.b, s0, q.g * p.N + min(n, p.N - 1), e / NP / 2, t0, tile, len);
        return c;
    }
    // row t of the segment, the last one for rows behind the end: no branch stands around a load
    __device__ __forceinline__ int64_t row(int t) const { return min(t, len - 1); }
    __device__ __forceinline__ size_t tile0() const   // first tile of the segment among the sequence's, per block
    {
        return (size_t)s0 / TS;
    }
};

// Pass 1.  ADJ: also the adjoint handed on (more than one segment).
template <typename T, int W, bool ADJ, bool GATED>
__global__ __launch_bounds__(64 * W) void scan_tiles_kernel(ScanProblem p, Segments sg, Ws ws, int nblk)
{
    typedef Walk<T, W> K;
    constexpr int TS = K::TS, OWN = K::OWN;
    __shared__ f32x2 du[TS][64];
    __shared__ float gy[ADJ ? TS : 1][64];
    __shared__ f32x4 bc[TS][2][W];
    const K k(p, sg, ADJ);
    const Place& q = k.q;
    const unsigned c = q.c;
    const float bias = p.dt_bias ? p.dt_bias[c] : 0.0f;
    const size_t blk = (size_t)q.b * nblk + q.blk;
    f32x4* tiles = ws.tiles + ((blk * k.nt + k.tile0()) * W + q.wave) * 64 + q.lane;
    float* cums = ws.cums + (blk * k.nt + k.tile0()) * 64 + q.lane;
    float A[kStates], h[kStates], P[kStates], G[kStates], cum = 0.0f;
    {
        const f32x4 av = load_states(p.a + (size_t)c * p.N + k.n0, k.ns);
        const f32x4 hv = sg.nseg == 1 && p.state ? load_states(p.state + ((size_t)q.b * p.D + c) * p.N + k.n0, k.ns)
                                                 : f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int n = 0; n < kStates; ++n) {
            A[n] = av[n] * kLog2e;
            h[n] = hv[n];
            P[n] = 1.0f;
            G[n] = 0.0f;
        }
    }
    struct Raw {
        T x[OWN], dt[OWN], z[OWN], dy[OWN], m;
    };
    constexpr int AHEAD = ahead(W);
    Raw raw[AHEAD];
    MatCursor<T> mat = k.matrices(p, 0, TS);
    const int softplus = __builtin_amdgcn_readfirstlane(p.softplus);
    auto fetch = [&](Raw& r, int t0) {
#pragma unroll
        for (int i = 0; i < OWN; ++i) {
            const int64_t t = k.row(t0 + k.own + i);
            r.x[i] = (k.xp + t * p.x.row)[c];
            r.dt[i] = (k.dp + t * p.dt.row)[c];
            if (ADJ) r.dy[i] = (k.gp + t * p.dy.row)[c];
            if (ADJ && GATED) r.z[i] = (k.zp + t * p.z.row)[c];
        }
        r.m = mat.next(t0, k.len);
    };
    auto publish = [&](const Raw& r) {
        if (k.mine) {
#pragma unroll
            for (int i = 0; i < OWN; ++i) {
                const float u = to_float(r.dt[i]) + bias;
                const float d = softplus ? softplus_t<T>(u) : u;
                du[k.own + i][q.lane] = f32x2{d, d * to_float(r.x[i])};
                if (ADJ) {
                    float g = to_float(r.dy[i]);
                    if (GATED) {
                        const float z = to_float(r.z[i]);
                        g *= z * sigmoid_t<T>(z);
                    }
                    gy[k.own + i][q.lane] = g;
                }
            }
        }
        ((float*)bc)[threadIdx.x] = k.mv ? to_float(r.m) : 0.0f;
    };
    auto step = [&](int s) {
        const f32x2 v = du[s][q.lane];
        const f32x4 Bv = bc[s][0][q.wave], Cv = bc[s][1][q.wave];
        const float g = ADJ ? gy[s][q.lane] : 0.0f;
        cum += v[0];
#pragma unroll
        for (int n = 0; n < kStates; ++n) {
            const float a = exp2_fast(v[0] * A[n]);
            h[n] = a * h[n] + v[1] * Bv[n];
            if (ADJ) {
                P[n] *= a;
                G[n] += P[n] * (Cv[n] * g);
            }
        }
    };
    __builtin_amdgcn_s_waitcnt(kVm0);   // see scan.hip
    __builtin_amdgcn_sched_barrier(0);
    if (k.len > 0) {
#pragma unroll
        for (int a = 0; a < AHEAD; ++a) fetch(raw[a], a * TS);
        publish(raw[0]);
    }
    auto tile = [&](int t0, Raw& r, const Raw& next) {
        const int cnt = min(TS, k.len - t0);
        fetch(r, t0 + AHEAD * TS);
        tiles[(size_t)(t0 / TS) * W * 64] = f32x4{h[0], h[1], h[2], h[3]};
        if (ADJ && q.wave == 0) cums[(size_t)(t0 / TS) * 64] = cum;
        __syncthreads();
        if (cnt == TS) {
#pragma unroll
            for (int s = 0; s < TS; ++s) {
                step(s);
                if (s & 1) __builtin_amdgcn_sched_barrier(0);
            }
        } else {
            for (int s = 0; s < cnt; ++s) step(s);
        }
        __syncthreads();
        publish(next);
    };
    for (int t0 = 0; t0 < k.len; t0 += AHEAD * TS) {
#pragma unroll
        for (int a = 0; a < AHEAD; ++a)
            if (t0 + a * TS < k.len) tile(t0 + a * TS, raw[a], raw[(a + 1) % AHEAD]);
    }
    if (ADJ && q.live) {
        const size_t e = ((size_t)q.b * sg.nseg + q.seg) * p.D + c;
        store_states(ws.ends + e * p.N + k.n0, k.ns, f32x4{h[0], h[1], h[2], h[3]});
        store_states(ws.adj + e * p.N + k.n0, k.ns, f32x4{G[0], G[1], G[2], G[3]});
        if (q.wave == 0) ws.sums[e] = cum;
    }
}

// Pass 2.
__global__ __launch_bounds__(256) void scan_links_kernel(ScanProblem p, Segments sg, Ws ws)
{
    const int64_t DN = (int64_t)p.D * p.N;
    const int64_t i = block_id() * 256 + threadIdx.x;
    if (i >= p.B * DN) return;
    const int64_t b = i / DN, k = i % DN;
    const float A = p.a[k] * kLog2e;
    float* e = ws.ends + b * sg.nseg * DN + k;
    float* g = ws.adj + b * sg.nseg * DN + k;
    const float* s = ws.sums + b * sg.nseg * p.D + k / p.N;
    // in batches, whose loads are under way together
    constexpr int LINKS = 8;
    float h = p.state ? p.state[i] : 0.0f;
    for (int j0 = 0; j0 < sg.nseg; j0 += LINKS) {
        float a[LINKS], v[LINKS];
#pragma unroll
        for (int k = 0; k < LINKS; ++k) {
            const int64_t j = min(j0 + k, sg.nseg - 1);
            a[k] = s[j * p.D];
            v[k] = e[j * DN];
        }
#pragma unroll
        for (int k = 0; k < LINKS; ++k) {
            if (j0 + k < sg.nseg) e[(j0 + k) * DN] = h;
            h = exp2_fast(a[k] * A) * h + v[k];
        }
    }
    float in = p.dstate_out ? p.dstate_out[i] : 0.0f;
    for (int j0 = sg.nseg - 1; j0 >= 0; j0 -= LINKS) {
        float a[LINKS], v[LINKS];
#pragma unroll
        for (int k = 0; k < LINKS; ++k) {
            const int64_t j = max(j0 - k, 0);
            a[k] = s[j * p.D];
            v[k] = g[j * DN];
        }
#pragma unroll
        for (int k = 0; k < LINKS; ++k) {
            if (j0 - k >= 0) g[(j0 - k) * DN] = in;
            in = exp2_fast(a[k] * A) * in + v[k];
        }
    }
}

__device__ __forceinline__ float ror8(float v)
{
    return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), 0x128, 0xf, 0xf, true));
}
template <int CTRL>
__device__ __forceinline__ float dpp_add(float v)
{
    return v + __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), CTRL, 0xf, 0xf, true));
}

// Two values' sums over pairs of lanes 32 (16) apart: the lower half (even
// rows) of the result belongs to a, the upper half (odd rows) to b.
__device__ __forceinline__ float fold32(float a, float b)
{
    const auto r = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(unsigned, a), __builtin_bit_cast(unsigned, b), false, false);
    const unsigned lo = r[0], hi = r[1];   // a bit cast of a vector's element itself would take element 0
    return __builtin_bit_cast(float, lo) + __builtin_bit_cast(float, hi);
}
__device__ __forceinline__ float fold16(float a, float b)
{
    const auto r = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(unsigned, a), __builtin_bit_cast(unsigned, b), false, false);
    const unsigned lo = r[0], hi = r[1];
    return __builtin_bit_cast(float, lo) + __builtin_bit_cast(float, hi);
}

// Sums of eight values over the 64 lanes: lane l returns the sum of
// v[4 ((l >> 3) & 1) + 2 ((l >> 4) & 1) + (l >> 5)].
__device__ __forceinline__ float sum8(const float (&v)[8], int lane)
{
    const float a0 = fold32(v[0], v[1]), a1 = fold32(v[2], v[3]), a2 = fold32(v[4], v[5]), a3 = fold32(v[6], v[7]);
    const float b0 = fold16(a0, a1), b1 = fold16(a2, a3);
    const float c0 = b0 + ror8(b0), c1 = b1 + ror8(b1);
    float c = (lane & 8) ? c1 : c0;
    c = dpp_add<0x141>(c);   // lane ^ 7
    c = dpp_add<0x4e>(c);    // lane ^ 2
    c = dpp_add<0xb1>(c);    // lane ^ 1
    return c;
}

// Pass 3.
template <typename T, int W, bool GATED>
__global__ __launch_bounds__(64 * W) void scan_bwd_kernel(ScanProblem p, Segments sg, Ws ws, int nblk)
{
    typedef Walk<T, W> K;
    constexpr int TS = K::TS, OWN = K::OWN, NS = GATED ? 3 : 2;
    static_assert(TS == 8, "the sums of eight steps leave together");
    __shared__ f32x2 du[TS][64];              // delta, delta x
    __shared__ float gy[TS][64];              // dy after the gate
    __shared__ f32x4 bc[TS][2][W];
    __shared__ float part[W][NS][TS][64];     // sum_n g B, sum_n w A, sum_n C h
    const K k(p, sg, true);
    const Place& q = k.q;
    const unsigned c = q.c;
    T* dxp = (T*)p.dx.p + q.b * p.dx.batch + k.s0 * p.dx.row;
    T* ddp = (T*)p.ddt.p + q.b * p.ddt.batch + k.s0 * p.ddt.row;
    T* dzp = GATED ? (T*)p.dz.p + q.b * p.dz.batch + k.s0 * p.dz.row : nullptr;
    const float skip = p.skip ? p.skip[c] : 0.0f;
    const float bias = p.dt_bias ? p.dt_bias[c] : 0.0f;
    const size_t blk = (size_t)q.b * nblk + q.blk;
    const f32x4* tiles = ws.tiles + ((blk * k.nt + k.tile0()) * W + q.wave) * 64 + q.lane;
    const float* cums = ws.cums + (blk * k.nt + k.tile0()) * 64 + q.lane;
    const size_t erow = (((size_t)q.b * sg.nseg + q.seg) * p.D + c) * p.N + k.n0;
    const size_t srow = ((size_t)q.b * p.D + c) * p.N + k.n0;
    const bool linked = sg.nseg > 1;
    // which of a step's eight sums this lane stores, and for which of the tile's steps
    const int vi = 4 * ((q.lane >> 3) & 1) + 2 * ((q.lane >> 4) & 1) + (q.lane >> 5), vs = q.lane & 7;
    const bool stores = (vi & 3) < k.ns;
    float* sums = (vi >= 4 ? ws.pc : ws.pb) +
                  ((((size_t)q.cb * p.B + q.b) * p.T + k.s0 + vs) * p.G + q.g) * p.N + k.n0 + (vi & 3);

    float A[kStates], ag[kStates], dA[kStates], hs[kStates];
    {
        const f32x4 av = load_states(p.a + (size_t)c * p.N + k.n0, k.ns);
        f32x4 gv = {0.0f, 0.0f, 0.0f, 0.0f}, sv = {0.0f, 0.0f, 0.0f, 0.0f};
        if (linked) {
            gv = load_states(ws.adj + erow, k.ns);
            sv = load_states(ws.ends + erow, k.ns);
        } else if (p.dstate_out) {
            gv = load_states(p.dstate_out + srow, k.ns);
        }
#pragma unroll
        for (int n = 0; n < kStates; ++n) {
            A[n] = av[n] * kLog2e;
            ag[n] = q.live ? gv[n] : 0.0f;
            hs[n] = sv[n];
            dA[n] = 0.0f;
        }
    }
    float dskip = 0.0f, dbias = 0.0f;
    struct Raw {
        T x[OWN], dt[OWN], z[OWN], dy[OWN], m;
        f32x4 h0;
        float cum;
    };
    constexpr int AHEAD = ahead(W);
    Raw raw[AHEAD];
    float xv[OWN], dv[OWN], sl[OWN], ge[OWN], zf[OWN];   // the current tile's own steps, for their finish
    auto fetch = [&](Raw& r, int t0) {                   // behind the first tile: the first
        t0 = max(t0, 0);
#pragma unroll
        for (int i = 0; i < OWN; ++i) {
            const int64_t t = k.row(t0 + k.own + i);
            r.x[i] = (k.xp + t * p.x.row)[c];
            r.dt[i] = (k.dp + t * p.dt.row)[c];
            r.dy[i] = (k.gp + t * p.dy.row)[c];
            if (GATED) r.z[i] = (k.zp + t * p.z.row)[c];
        }
        r.m = k.mp[k.row(t0 + k.ms) * k.mr];   // a product a tile: the cursor steps forwards only
        r.h0 = tiles[(size_t)(t0 / TS) * W * 64];
        r.cum = linked ? cums[(size_t)(t0 / TS) * 64] : 0.0f;
    };
    auto publish = [&](const Raw& r) {
#pragma unroll
        for (int i = 0; i < OWN; ++i) {
            // a lane without a channel adds nothing to the sums over channels
            xv[i] = q.live ? to_float(r.x[i]) : 0.0f;
            const float u = to_float(r.dt[i]) + bias;
            dv[i] = u;
            sl[i] = 1.0f;
            if (p.softplus) {   // and its slope, sigmoid(u), from the same e^{-|u|}
                const float y = sizeof(T) == 2 ? exp2_fast(fabsf(u) * -kLog2e) : exp_f(-fabsf(u));
                dv[i] = softplus_of(u, y);
                sl[i] = __builtin_amdgcn_rcpf(1.0f + y) * (u < 0.0f ? y : 1.0f);
            }
            float g = q.live ? to_float(r.dy[i]) : 0.0f;
            if (GATED) {
                const float z = to_float(r.z[i]), sg = sigmoid_t<T>(z), zs = z * sg;
                zf[i] = g * (sg + zs * (1.0f - sg));
                g = q.live ? g * zs : 0.0f;
            }
            ge[i] = g;
            if (k.mine) {
                du[k.own + i][q.lane] = f32x2{dv[i], dv[i] * xv[i]};
                gy[k.own + i][q.lane] = g;
            }
        }
        ((float*)bc)[threadIdx.x] = k.mv ? to_float(r.m) : 0.0f;
    };
    auto finish = [&](int t0) {
        const int n = k.mine ? k.len - t0 - k.own : 0;
#pragma unroll
        for (int i = 0; i < OWN; ++i) {
            if (i < n) {
                const int s = k.own + i;
                float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
                for (int w = 0; w < W; ++w) {
                    s1 += part[w][0][s][q.lane];
                    s2 += part[w][1][s][q.lane];
                }
                const float dd = (xv[i] * s1 + s2 * kLn2) * sl[i];
                dskip += ge[i] * xv[i];
                dbias += dd;
                const int64_t t = t0 + s;
                float o = skip * xv[i];
                if (GATED) {
#pragma unroll
                    for (int w = 0; w < W; ++w) o += part[w][NS - 1][s][q.lane];
                }
                if (q.live) {
                    (dxp + t * p.dx.row)[c] = from_float<T>(dv[i] * s1 + skip * ge[i]);
                    (ddp + t * p.ddt.row)[c] = from_float<T>(dd);
                    if (GATED) (dzp + t * p.dz.row)[c] = from_float<T>(zf[i] * o);
                }
            }
        }
    };
    // cnt steps of the tile (ALL: all of them, known when compiled)
    auto walk = [&](auto ALL, int cnt, int t0, f32x4 h0, float cum) {
        constexpr bool all = decltype(ALL)::value;
        if (linked) {
#pragma unroll
            for (int n = 0; n < kStates; ++n) h0[n] += exp2_fast(cum * A[n]) * hs[n];
        }
        // The published values of the next step are read while the current one is computed; the scheduler is
        // kept from reading further ahead, which costs registers and with them waves on a SIMD.
        struct In {
            f32x2 v;
            f32x4 B, C;
            float g;
        } in[2];
        auto load = [&](In& r, int s, bool c4, bool g1) {
            r.v = du[s][q.lane];
            r.B = bc[s][0][q.wave];
            if (c4) r.C = bc[s][1][q.wave];
            if (g1) r.g = gy[s][q.lane];
        };
        float h[TS][kStates], a[TS][kStates];
        load(in[0], 0, GATED, false);
#pragma unroll
        for (int s = 0; s < TS; ++s) {
            if (s + 1 < TS) load(in[(s + 1) & 1], s + 1, GATED, false);
            __builtin_amdgcn_sched_barrier(0);
            if (all || s < cnt) {
                const In& r = in[s & 1];
#pragma unroll
                for (int n = 0; n < kStates; ++n) {
                    a[s][n] = exp2_fast(r.v[0] * A[n]);
                    h[s][n] = a[s][n] * (s ? h[s ? s - 1 : 0][n] : h0[n]) + r.v[1] * r.B[n];
                }
                if (GATED) {
                    float o = 0.0f;
#pragma unroll
                    for (int n = 0; n < kStates; ++n) o += r.C[n] * h[s][n];
                    part[q.wave][NS - 1][s][q.lane] = o;
                }
            }
        }
        float mine = 0.0f;
        load(in[(TS - 1) & 1], TS - 1, true, true);
#pragma unroll
        for (int s = TS - 1; s >= 0; --s) {
            if (s > 0) load(in[(s - 1) & 1], s - 1, true, true);
            __builtin_amdgcn_sched_barrier(0);
            if (all || s < cnt) {
                const In& r = in[s & 1];
                float s1 = 0.0f, s2 = 0.0f, sum[8];
#pragma unroll
                for (int n = 0; n < kStates; ++n) {
                    const float gn = r.C[n] * r.g + ag[n];
                    sum[n] = gn * r.v[1];
                    sum[4 + n] = r.g * h[s][n];
                    s1 += gn * r.B[n];
                    ag[n] = gn * a[s][n];
                    const float wn = ag[n] * (s ? h[s ? s - 1 : 0][n] : h0[n]);
                    s2 += wn * A[n];
                    dA[n] += wn * r.v[0];
                }
                part[q.wave][0][s][q.lane] = s1;
                part[q.wave][1][s][q.lane] = s2;
                const float t = sum8(sum, q.lane);
                mine = vs == s ? t : mine;
            }
        }
        if (stores && vs < cnt) sums[(size_t)t0 * p.G * p.N] = mine;
    };
    const int last = (k.len - 1) / TS * TS;
    __builtin_amdgcn_s_waitcnt(kVm0);   // see scan.hip
    __builtin_amdgcn_sched_barrier(0);
    if (k.len > 0) {
#pragma unroll
        for (int a = 0; a < AHEAD; ++a) fetch(raw[a], last - a * TS);
        publish(raw[0]);
    }
    auto tile = [&](int t0, Raw& r, const Raw& next) {
        const int cnt = min(TS, k.len - t0);
        const f32x4 h0 = r.h0;
        const float cum = r.cum;
        fetch(r, t0 - AHEAD * TS);
        __syncthreads();
        if (cnt == TS) walk(std::true_type{}, TS, t0, h0, cum);
        else walk(std::false_type{}, cnt, t0, h0, cum);
        __syncthreads();
        finish(t0);
        publish(next);
    };
    for (int t0 = last; t0 >= 0 && k.len > 0; t0 -= AHEAD * TS) {
#pragma unroll
        for (int a = 0; a < AHEAD; ++a)
            if (t0 - a * TS >= 0) tile(t0 - a * TS, raw[a], raw[(a + 1) % AHEAD]);
    }
    for (int t = k.len + q.wave; t < k.s1 - k.s0; t += W)
        if (q.live) {
            (dxp + t * p.dx.row)[c] = from_float<T>(0.0f);
            (ddp + t * p.ddt.row)[c] = from_float<T>(0.0f);
            if (GATED) (dzp + t * p.dz.row)[c] = from_float<T>(0.0f);
        }
    if (q.live) {
        if (p.dstate && q.seg == 0) store_states(p.dstate + srow, k.ns, f32x4{ag[0], ag[1], ag[2], ag[3]});
        store_states(ws.pa + erow, k.ns, f32x4{dA[0], dA[1], dA[2], dA[3]});
    }
    __syncthreads();
    part[q.wave][0][0][q.lane] = dskip;
    part[q.wave][1][0][q.lane] = dbias;
    __syncthreads();
    if (q.wave == 0 && q.live) {
        float s1 = 0.0f, s2 = 0.0f;
        for (int w = 0; w < W; ++w) {
            s1 += part[w][0][0][q.lane];
            s2 += part[w][1][0][q.lane];
        }
        const size_t e = ((size_t)q.b * sg.nseg + q.seg) * p.D + c;
        ws.pskip[e] = s1;
        ws.pbias[e] = s2;
    }
}

// Pass 4: dB and dC over the blocks of channels (rows behind a sequence are
// 0), a thread an element; dA, dskip and ddt_bias over segments and
// sequences, 64 columns to a workgroup.  I: the type that counts dB's and dC's
// elements (a division in 64 bits costs more than the sum).
template <typename T, typename I>
__global__ __launch_bounds__(1024) void scan_sums_kernel(ScanProblem p, Ws ws, int ncb, int parts)
{
    __shared__ float red[16][64];
    const I GN = (I)(p.G * p.N), nbc = (I)p.B * (I)p.T * GN;
    const int64_t na = (int64_t)p.D * p.N, first = (2 * (int64_t)nbc + 1023) / 1024, da = (na + 63) / 64, dd = (p.D + 63) / 64;
    int64_t blk = block_id();
    if (blk < first) {
        I i = (I)blk * 1024 + threadIdx.x;
        if (i >= 2 * nbc) return;
        const bool isc = i >= nbc;
        if (isc) i -= nbc;
        const I r = i / GN;
        const int k = (int)(i % GN), b = (int)(r / (I)p.T), t = (int)(r % (I)p.T);
        float s = 0.0f;
        if (t < clamp_len(p.lengths, b, p.T)) {
            const float* src = (isc ? ws.pc : ws.pb) + i;
#pragma unroll 8
            for (int cb = 0; cb < ncb; ++cb) s += src[(size_t)cb * nbc];
        }
        const Rows& o = isc ? p.dcmat : p.dbmat;
        ((T*)o.p)[b * o.batch + t * o.row + k] = from_float<T>(s);
        return;
    }
    blk -= first;
    const float* part = ws.pa;
    float* out = p.da;
    int64_t n = na;
    if (blk >= da) {
        blk -= da;
        n = p.D;
        part = blk < dd ? ws.pskip : ws.pbias;
        out = blk < dd ? p.dskip : p.ddt_bias;
        if (blk >= dd) blk -= dd;
        if (blk >= dd) return;   // behind the last workgroup
    }
    const float s = part_sum(part, parts, n, n, blk, red);
    if (threadIdx.x < 64 && out && blk * 64 + threadIdx.x < n) out[blk * 64 + threadIdx.x] = s;
}

template <typename T, int W>
hipError_t bwd_w(const ScanProblem& p, hipStream_t stream)
{
    const Segments sg = segments_of(p);
    const int nblk = channel_blocks(p);
    const unsigned blocks = (unsigned)p.B * sg.nseg * nblk;
    const Ws ws = layout(p, sg, p.ws);
    hipError_t e;
    if (sg.nseg > 1) {
        if (p.z.p) scan_tiles_kernel<T, W, true, true><<<blocks, 64 * W, 0, stream>>>(p, sg, ws, nblk);
        else scan_tiles_kernel<T, W, true, false><<<blocks, 64 * W, 0, stream>>>(p, sg, ws, nblk);
        if ((e = hipGetLastError()) != hipSuccess) return e;
        const int64_t n = (int64_t)p.B * p.D * p.N;
        scan_links_kernel<<<grid_of((n + 255) / 256), 256, 0, stream>>>(p, sg, ws);
    } else {
        scan_tiles_kernel<T, W, false, false><<<blocks, 64 * W, 0, stream>>>(p, sg, ws, nblk);
    }
    if ((e = hipGetLastError()) != hipSuccess) return e;
    if (p.z.p) scan_bwd_kernel<T, W, true><<<blocks, 64 * W, 0, stream>>>(p, sg, ws, nblk);
    else scan_bwd_kernel<T, W, false><<<blocks, 64 * W, 0, stream>>>(p, sg, ws, nblk);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    const int64_t nbc = (int64_t)p.B * p.T * p.G * p.N;
    const dim3 grid = grid_of((2 * nbc + 1023) / 1024 + ((int64_t)p.D * p.N + 63) / 64 + 2 * ((p.D + 63) / 64));
    const int ncb = (p.D / p.G + 63) / 64, parts = p.B * sg.nseg;
    if (nbc < (int64_t(1) << 30)) scan_sums_kernel<T, uint32_t><<<grid, 1024, 0, stream>>>(p, ws, ncb, parts);
    else scan_sums_kernel<T, uint64_t><<<grid, 1024, 0, stream>>>(p, ws, ncb, parts);
    return hipGetLastError();
}

template <typename T>
hipError_t bwd_t(const ScanProblem& p, hipStream_t stream)
{
    switch (waves_of(p.N)) {
    case 1: return bwd_w<T, 1>(p, stream);
    case 2: return bwd_w<T, 2>(p, stream);
    case 4: return bwd_w<T, 4>(p, stream);
    case 8: return bwd_w<T, 8>(p, stream);
    default: return bwd_w<T, 16>(p, stream);
    }
}

}  // namespace

size_t scan_bwd_workspace(const ScanProblem& p) { return layout(p, segments_of(p), nullptr).bytes; }

hipError_t launch_scan_bwd(const ScanProblem& p, hipStream_t stream)
{
    return p.bf16 ? bwd_t<bf16>(p, stream) : bwd_t<float>(p, stream);
}

}  // namespace tfla
