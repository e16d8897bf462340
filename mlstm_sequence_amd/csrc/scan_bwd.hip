// scan_bwd.hip -- backward pass of the selective scan (scan_impl.hpp).
//
// With g_t the gradient of h_t and dy_t that of o_t (after the gate):
//
//   g_t = C_t dy_t + a_{t+1} g_{t+1}       w_t = g_t a_t h_{t-1}
//   dC_t[n] = sum_c dy_t h_t               dB_t[n] = sum_c g_t delta_t x_t
//   dx_t = delta_t sum_n g_t B_t + skip dy_t
//   ddelta_t = x_t sum_n g_t B_t + sum_n w_t A         dA = sum_t w_t delta_t
//
// Pass 1 walks forward and keeps the state at the start of every tile of
// steps.  Pass 2 walks the tiles from the last to the first: it recomputes
// the tile's states and decays into registers, then runs the adjoint back
// over them.  Sums over a wave's channels (dB, dC) go through lane swaps and
// adds; each 64-channel block writes its own sums, and pass 3 adds the blocks
// and sequences up in a fixed order.
#include "scan_impl.hpp"

namespace tfla {
namespace {

using namespace scan;

constexpr float kLn2 = 0.6931471805599453f;

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

// steps of a tile: 16 waves leave half the registers to each
constexpr int tile_steps(int w) { return w > 8 ? 8 : 16; }

struct Ws {
    f32x4* tiles;        // [blocks][tiles][W][64]: states at the tiles' starts
    float *pb, *pc;      // [ncb][B][T][G][N]: dB, dC of one block of channels
    float* pa;           // [B][D][N]
    float *pskip, *pbias;   // [B][D]
    size_t bytes;
};

Ws layout(const ScanProblem& p, char* base)
{
    const int W = waves_of(p.N), ts = tile_steps(W);
    const int per = p.D / p.G, ncb = (per + 63) / 64;
    const size_t blocks = (size_t)p.B * p.G * ncb, nt = (p.T + ts - 1) / ts;
    Ws w;
    size_t off = 0;
    auto take = [&](size_t bytes) {
        char* r = base + off;
        off += align256(bytes);
        return r;
    };
    w.tiles = (f32x4*)take(blocks * nt * W * 64 * 16);
    const size_t bc = (size_t)ncb * p.B * p.T * p.G * p.N * 4;
    w.pb = (float*)take(bc);
    w.pc = (float*)take(bc);
    w.pa = (float*)take((size_t)p.B * p.D * p.N * 4);
    w.pskip = (float*)take((size_t)p.B * p.D * 4);
    w.pbias = (float*)take((size_t)p.B * p.D * 4);
    w.bytes = off;
    return w;
}

// Pass 1.
template <typename T, int W>
__global__ __launch_bounds__(64 * W) void scan_tiles_kernel(ScanProblem p, f32x4* __restrict__ tiles)
{
    constexpr int TS = tile_steps(W);
    __shared__ f32x2 du[TS][64];
    const Place q = place(p, Segments{p.T, 1});
    const int len = clamp_len(p.lengths, q.b, p.T);
    const int n0 = q.wave * kStates;
    const bool has = n0 < p.N;
    const int nn = has ? n0 : 0;
    const T* xp = (const T*)p.x.p + q.b * p.x.batch + q.c;
    const T* dp = (const T*)p.dt.p + q.b * p.dt.batch + q.c;
    const T* Bp = (const T*)p.bmat.p + q.b * p.bmat.batch + q.g * p.N + nn;
    const float bias = p.dt_bias ? p.dt_bias[q.c] : 0.0f;
    const size_t srow = ((size_t)q.b * p.D + q.c) * p.N + nn;
    const size_t nt = (p.T + TS - 1) / TS;
    f32x4* out = tiles + ((size_t)blockIdx.x * nt * W + q.wave) * 64 + q.lane;
    float A[kStates], h[kStates];
#pragma unroll
    for (int n = 0; n < kStates; ++n) {
        A[n] = p.a[(size_t)q.c * p.N + nn + n] * kLog2e;
        h[n] = p.state ? p.state[srow + n] : 0.0f;
    }
    for (int t0 = 0; t0 < len; t0 += TS) {
        const int cnt = min(TS, len - t0);
        out[(size_t)(t0 / TS) * W * 64] = f32x4{h[0], h[1], h[2], h[3]};
        __syncthreads();
        for (int s = q.wave; s < cnt; s += W) {
            const float xv = to_float(xp[(t0 + s) * p.x.row]);
            const float u = to_float(dp[(t0 + s) * p.dt.row]) + bias;
            const float d = p.softplus ? softplus_t<T>(u) : u;
            du[s][q.lane] = f32x2{d, d * xv};
        }
        __syncthreads();
        for (int s = 0; s < cnt; ++s) {
            const f32x2 v = du[s][q.lane];
            Uniform4<T> Bv;
            Bv.load(Bp + (t0 + s) * p.bmat.row);
#pragma unroll
            for (int n = 0; n < kStates; ++n) h[n] = exp2_fast(v[0] * A[n]) * h[n] + v[1] * Bv.get(n);
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

// v0 + v1 where each half (rows, lane pairs ...) afterwards holds one of the
// two values' partial sums: 32 lanes apart, 16 lanes apart.
__device__ __forceinline__ float fold32(float a, float b)
{
    const auto r = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(unsigned, a), __builtin_bit_cast(unsigned, b), false, false);
    const unsigned lo = r[0], hi = r[1];   // a bit cast of a vector's element itself would take element 0
    return __builtin_bit_cast(float, lo) + __builtin_bit_cast(float, hi);
}
__device__ __forceinline__ float fold16(float a, float b)
{
    const auto r = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(unsigned, a), __builtin_bit_cast(unsigned, b), false, false);
    const unsigned lo = r[0], hi = r[1];   // a bit cast of a vector's element itself would take element 0
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

// Pass 2.
template <typename T, int W>
__global__ __launch_bounds__(64 * W) void scan_bwd_kernel(ScanProblem p, Ws ws)
{
    constexpr int TS = tile_steps(W);
    constexpr int OWN = TS / W > 0 ? TS / W : 1;
    __shared__ f32x4 in[TS][64];              // delta, delta x, dy after the gate
    __shared__ float part[W][3][TS][64];      // sum_n g B, sum_n w A, sum_n C h
    const Place q = place(p, Segments{p.T, 1});
    const int len = clamp_len(p.lengths, q.b, p.T);
    const int n0 = q.wave * kStates;
    const bool has = n0 < p.N;
    const int nn = has ? n0 : 0;
    const T* xp = (const T*)p.x.p + q.b * p.x.batch + q.c;
    const T* dp = (const T*)p.dt.p + q.b * p.dt.batch + q.c;
    const T* zp = p.z.p ? (const T*)p.z.p + q.b * p.z.batch + q.c : nullptr;
    const T* gp = (const T*)p.dy.p + q.b * p.dy.batch + q.c;
    T* dxp = (T*)p.dx.p + q.b * p.dx.batch + q.c;
    T* ddp = (T*)p.ddt.p + q.b * p.ddt.batch + q.c;
    T* dzp = p.z.p ? (T*)p.dz.p + q.b * p.dz.batch + q.c : nullptr;
    const T* Bp = (const T*)p.bmat.p + q.b * p.bmat.batch + q.g * p.N + nn;
    const T* Cp = (const T*)p.cmat.p + q.b * p.cmat.batch + q.g * p.N + nn;
    const float skip = p.skip ? p.skip[q.c] : 0.0f;
    const float bias = p.dt_bias ? p.dt_bias[q.c] : 0.0f;
    const size_t srow = ((size_t)q.b * p.D + q.c) * p.N + nn;
    const size_t nt = (p.T + TS - 1) / TS;
    const f32x4* starts = ws.tiles + ((size_t)blockIdx.x * nt * W + q.wave) * 64 + q.lane;
    // which of a step's eight sums this lane stores, and for which of eight steps
    const int vi = 4 * ((q.lane >> 3) & 1) + 2 * ((q.lane >> 4) & 1) + (q.lane >> 5), vs = q.lane & 7;
    float* sums = (vi >= 4 ? ws.pc : ws.pb) +
                  (((size_t)q.cb * p.B + q.b) * p.T * p.G + q.g) * p.N + nn + (vi & 3);

    float A[kStates], ag[kStates], dA[kStates];
#pragma unroll
    for (int n = 0; n < kStates; ++n) {
        A[n] = p.a[(size_t)q.c * p.N + nn + n] * kLog2e;
        ag[n] = p.dstate_out ? p.dstate_out[srow + n] : 0.0f;
        dA[n] = 0.0f;
    }
    float dskip = 0.0f, dbias = 0.0f;
    for (int t0 = (len - 1) / TS * TS; t0 >= 0 && len > 0; t0 -= TS) {
        const int cnt = min(TS, len - t0);
        float xv[OWN], dv[OWN], sl[OWN], gv[OWN], dzv[OWN], ge[OWN];
#pragma unroll
        for (int i = 0; i < OWN; ++i) {
            const int s = q.wave + i * W;
            if (s < cnt) {
                xv[i] = q.live ? to_float(xp[(t0 + s) * p.x.row]) : 0.0f;
                const float u = to_float(dp[(t0 + s) * p.dt.row]) + bias;
                dv[i] = p.softplus ? softplus_t<T>(u) : u;
                sl[i] = p.softplus ? sigmoid_t<T>(u) : 1.0f;
                gv[i] = q.live ? to_float(gp[(t0 + s) * p.dy.row]) : 0.0f;
                ge[i] = gv[i];
                if (zp) {
                    const float z = to_float(zp[(t0 + s) * p.z.row]);
                    const float sg = sigmoid_t<T>(z);
                    ge[i] = gv[i] * z * sg;
                    dzv[i] = gv[i] * sg * (1.0f + z * (1.0f - sg));
                }
                in[s][q.lane] = f32x4{dv[i], dv[i] * xv[i], ge[i], 0.0f};
            }
        }
        __syncthreads();
        if (has) {
            const f32x4 h0 = starts[(size_t)(t0 / TS) * W * 64];
            float h[TS][kStates], a[TS][kStates];
#pragma unroll
            for (int s = 0; s < TS; ++s) {
                if (s < cnt) {
                    const f32x4 v = in[s][q.lane];
                    Uniform4<T> Bv, Cv;
                    Bv.load(Bp + (t0 + s) * p.bmat.row);
                    Cv.load(Cp + (t0 + s) * p.cmat.row);
                    float o = 0.0f;
#pragma unroll
                    for (int n = 0; n < kStates; ++n) {
                        a[s][n] = exp2_fast(v[0] * A[n]);
                        h[s][n] = a[s][n] * (s ? h[s ? s - 1 : 0][n] : h0[n]) + v[1] * Bv.get(n);
                        o += Cv.get(n) * h[s][n];
                    }
                    if (zp) part[q.wave][2][s][q.lane] = o;
                }
            }
            float mine = 0.0f;
#pragma unroll
            for (int s = TS - 1; s >= 0; --s) {
                if (s < cnt) {
                    const f32x4 v = in[s][q.lane];
                    Uniform4<T> Bv, Cv;
                    Bv.load(Bp + (t0 + s) * p.bmat.row);
                    Cv.load(Cp + (t0 + s) * p.cmat.row);
                    float s1 = 0.0f, s2 = 0.0f, sum[8];
#pragma unroll
                    for (int n = 0; n < kStates; ++n) {
                        const float gn = Cv.get(n) * v[2] + ag[n];
                        sum[n] = gn * v[1];
                        sum[4 + n] = v[2] * h[s][n];
                        s1 += gn * Bv.get(n);
                        ag[n] = gn * a[s][n];
                        const float wn = ag[n] * (s ? h[s ? s - 1 : 0][n] : h0[n]);
                        s2 += wn * A[n];
                        dA[n] += wn * v[0];
                    }
                    part[q.wave][0][s][q.lane] = s1;
                    part[q.wave][1][s][q.lane] = s2;
                    const float r = sum8(sum, q.lane);
                    mine = vs == (s & 7) ? r : mine;
                }
                if ((s & 7) == 0 && s < cnt && s + vs < cnt) sums[(size_t)(t0 + s + vs) * p.G * p.N] = mine;
            }
        } else {
            for (int s = 0; s < cnt; ++s)
                for (int k = 0; k < 3; ++k) part[q.wave][k][s][q.lane] = 0.0f;
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < OWN; ++i) {
            const int s = q.wave + i * W;
            if (s < cnt) {
                float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
                for (int w = 0; w < W; ++w) {
                    s1 += part[w][0][s][q.lane];
                    s2 += part[w][1][s][q.lane];
                }
                const float dd = (xv[i] * s1 + s2 * kLn2) * sl[i];
                dskip += ge[i] * xv[i];
                dbias += dd;
                if (q.live) {
                    dxp[(t0 + s) * p.dx.row] = from_float<T>(dv[i] * s1 + skip * ge[i]);
                    ddp[(t0 + s) * p.ddt.row] = from_float<T>(dd);
                }
                if (zp) {
                    float o = skip * xv[i];
#pragma unroll
                    for (int w = 0; w < W; ++w) o += part[w][2][s][q.lane];
                    if (q.live) dzp[(t0 + s) * p.dz.row] = from_float<T>(dzv[i] * o);
                }
            }
        }
    }
    for (int t = len + q.wave; t < p.T; t += W)
        if (q.live) {
            dxp[t * p.dx.row] = from_float<T>(0.0f);
            ddp[t * p.ddt.row] = from_float<T>(0.0f);
            if (zp) dzp[t * p.dz.row] = from_float<T>(0.0f);
        }
    if (has && q.live) {
#pragma unroll
        for (int n = 0; n < kStates; ++n) {
            if (p.dstate) p.dstate[srow + n] = ag[n];
            ws.pa[srow + n] = dA[n];
        }
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
        ws.pskip[(size_t)q.b * p.D + q.c] = s1;
        ws.pbias[(size_t)q.b * p.D + q.c] = s2;
    }
}

// Pass 3: dB and dC over the blocks of channels (rows behind a sequence are
// 0), dA, dskip and ddt_bias over the sequences.
template <typename T>
__global__ __launch_bounds__(256) void scan_sums_kernel(ScanProblem p, Ws ws, int ncb)
{
    const int64_t GN = (int64_t)p.G * p.N, rows = (int64_t)p.B * p.T;
    const int64_t nbc = rows * GN, na = (int64_t)p.D * p.N;
    int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i < 2 * nbc) {
        const bool isc = i >= nbc;
        if (isc) i -= nbc;
        const int64_t r = i / GN, k = i % GN;
        const int b = (int)(r / p.T), t = (int)(r % p.T);
        float s = 0.0f;
        if (t < clamp_len(p.lengths, b, p.T)) {
            const float* src = (isc ? ws.pc : ws.pb) + i;
            for (int cb = 0; cb < ncb; ++cb) s += src[cb * nbc];
        }
        const Rows& o = isc ? p.dcmat : p.dbmat;
        ((T*)o.p)[b * o.batch + t * o.row + k] = from_float<T>(s);
        return;
    }
    i -= 2 * nbc;
    if (i < na) {
        float s = 0.0f;
        for (int b = 0; b < p.B; ++b) s += ws.pa[b * na + i];
        p.da[i] = s;
        return;
    }
    i -= na;
    if (i < p.D) {
        float s = 0.0f, r = 0.0f;
        for (int b = 0; b < p.B; ++b) {
            s += ws.pskip[(int64_t)b * p.D + i];
            r += ws.pbias[(int64_t)b * p.D + i];
        }
        if (p.dskip) p.dskip[i] = s;
        if (p.ddt_bias) p.ddt_bias[i] = r;
    }
}

template <typename T, int W>
hipError_t bwd_w(const ScanProblem& p, hipStream_t stream)
{
    const int ncb = (p.D / p.G + 63) / 64;
    const unsigned blocks = (unsigned)p.B * p.G * ncb;
    const Ws ws = layout(p, p.ws);
    scan_tiles_kernel<T, W><<<blocks, 64 * W, 0, stream>>>(p, ws.tiles);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    scan_bwd_kernel<T, W><<<blocks, 64 * W, 0, stream>>>(p, ws);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    const int64_t n = 2 * (int64_t)p.B * p.T * p.G * p.N + (int64_t)p.D * p.N + p.D;
    scan_sums_kernel<T><<<(unsigned)((n + 255) / 256), 256, 0, stream>>>(p, ws, ncb);
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

size_t scan_bwd_workspace(const ScanProblem& p) { return layout(p, nullptr).bytes; }

hipError_t launch_scan_bwd(const ScanProblem& p, hipStream_t stream)
{
    return p.bf16 ? bwd_t<bf16>(p, stream) : bwd_t<float>(p, stream);
}

}  // namespace tfla
