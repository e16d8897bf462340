// diag_bwd.hip -- gated linear recurrence of channels, backward (diag_impl.hpp).
#include "diag_impl.hpp"
#include "sums.hpp"

namespace tfla {
namespace {

using namespace diag;

// A thread walks a channel of a sequence, chunk after chunk from the end: the states of a chunk again from its start,
// then the adjoint back over them.
template <typename T, int KIND>
__global__ __launch_bounds__(64) void diag_bwd_kernel(DiagProblem p)
{
    __shared__ float hs[kChunk][64];
    const int nb = (p.D + 63) / 64, lane = threadIdx.x, c = (int)(block_id() % nb) * 64 + lane;
    const int64_t b = block_id() / nb;
    if (b >= p.B || c >= p.D) return;
    const int len = clamp_len(p.lengths, (int)b, p.T), chunks = (p.T + kChunk - 1) / kChunk;
    const T* x = (const T*)p.x.p + b * p.x.batch + c;
    const T* u = (const T*)p.fgate.p + b * p.fgate.batch + c;
    const T* v = KIND != kCoupled ? (const T*)p.igate.p + b * p.igate.batch + c : nullptr;
    const T* dy = (const T*)p.dy.p + b * p.dy.batch + c;
    T* dx = (T*)p.dx.p + b * p.dx.batch + c;
    T* du = (T*)p.dfgate.p + b * p.dfgate.batch + c;
    T* dv = KIND != kCoupled ? (T*)p.digate.p + b * p.digate.batch + c : nullptr;
    const float decay = KIND == kDecay ? p.decay[c] : 0.0f;
    for (int64_t t = len; t < p.T; ++t) {
        dx[t * p.dx.row] = du[t * p.dfgate.row] = from_float<T>(0.0f);
        if (dv) dv[t * p.digate.row] = from_float<T>(0.0f);
    }
    auto gates = [&](int64_t t) {
        return gate_of<T, KIND>(to_float(u[t * p.fgate.row]), v ? to_float(v[t * p.igate.row]) : 0.0f, decay);
    };
    float a = p.dstate_out ? p.dstate_out[b * p.D + c] : 0.0f, dd = 0.0f;   // a = f_{t+1} g_{t+1}
    for (int64_t t0 = (len - 1) / kChunk * kChunk; len > 0 && t0 >= 0; t0 -= kChunk) {
        const int n = (int)min<int64_t>(kChunk, len - t0);
        float h = p.starts[(b * chunks + t0 / kChunk) * p.D + c];
        for (int k = 0; k < n; ++k) {
            hs[k][lane] = h;
            const Gate g = gates(t0 + k);
            h = g.f * h + g.i * to_float(x[(t0 + k) * p.x.row]);
        }
        for (int k = n - 1; k >= 0; --k) {
            const int64_t t = t0 + k;
            const Gate k_ = gates(t);
            const float g = to_float(dy[t * p.dy.row]) + a;
            const GateGrads o = grads_of<KIND>(k_, to_float(x[t * p.x.row]), hs[k][lane], g, decay);
            a = k_.f * g;
            dd += o.dd;
            dx[t * p.dx.row] = from_float<T>(o.dx);
            du[t * p.dfgate.row] = from_float<T>(o.du);
            if (dv) dv[t * p.digate.row] = from_float<T>(o.dv);
        }
    }
    if (p.dstate) p.dstate[b * p.D + c] = a;
    if (KIND == kDecay) ((float*)p.ws)[b * p.D + c] = dd;
}

__global__ __launch_bounds__(1024) void diag_params_kernel(DiagProblem p, int64_t parts)
{
    __shared__ float red[16][64];
    const int64_t i = (int64_t)blockIdx.x * 64 + threadIdx.x;
    const float s = part_sum((const float*)p.ws, parts, p.D, p.D, blockIdx.x, red);
    if (threadIdx.x < 64 && i < p.D) p.ddecay[i] = s;
}

template <typename T>
hipError_t bwd_t(const DiagProblem& p, hipStream_t stream)
{
    const dim3 grid = grid_of((int64_t)p.B * ((p.D + 63) / 64));
    switch (p.kind) {
    case kCoupled: diag_bwd_kernel<T, kCoupled><<<grid, 64, 0, stream>>>(p); break;
    case kSigmoid: diag_bwd_kernel<T, kSigmoid><<<grid, 64, 0, stream>>>(p); break;
    default: diag_bwd_kernel<T, kDecay><<<grid, 64, 0, stream>>>(p); break;
    }
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || p.kind != kDecay) return e;
    diag_params_kernel<<<(unsigned)((p.D + 63) / 64), 1024, 0, stream>>>(p, p.B);
    return hipGetLastError();
}

}  // namespace

size_t diag_bwd_workspace(const DiagProblem& p) { return p.kind == kDecay ? (size_t)p.B * p.D * sizeof(float) : 0; }

hipError_t launch_diag_bwd(const DiagProblem& p, hipStream_t stream)
{
    return p.bf16 ? bwd_t<bf16>(p, stream) : bwd_t<float>(p, stream);
}

}  // namespace tfla
