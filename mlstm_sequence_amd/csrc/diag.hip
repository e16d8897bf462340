// diag.hip -- gated linear recurrence of channels, forward (diag_impl.hpp).
#include "diag_impl.hpp"

namespace tfla {
namespace {

using namespace diag;

// A thread walks a channel of a sequence.
template <typename T, int KIND>
__global__ __launch_bounds__(64) void diag_fwd_kernel(DiagProblem p)
{
    const int nb = (p.D + 63) / 64, c = (int)(block_id() % nb) * 64 + threadIdx.x;
    const int64_t b = block_id() / nb;
    if (b >= p.B || c >= p.D) return;
    const int len = clamp_len(p.lengths, (int)b, p.T), chunks = (p.T + kChunk - 1) / kChunk;
    const T* x = (const T*)p.x.p + b * p.x.batch + c;
    const T* u = (const T*)p.fgate.p + b * p.fgate.batch + c;
    const T* v = KIND != kCoupled ? (const T*)p.igate.p + b * p.igate.batch + c : nullptr;
    T* y = (T*)p.y.p + b * p.y.batch + c;
    const float decay = KIND == kDecay ? p.decay[c] : 0.0f;
    float h = p.state ? p.state[b * p.D + c] : 0.0f;
    for (int64_t t = 0; t < p.T; ++t) {
        if (p.starts && t % kChunk == 0) p.starts[(b * chunks + t / kChunk) * p.D + c] = h;
        if (t < len) {
            const Gate g = gate_of<T, KIND>(to_float(u[t * p.fgate.row]), v ? to_float(v[t * p.igate.row]) : 0.0f, decay);
            h = g.f * h + g.i * to_float(x[t * p.x.row]);
        }
        y[t * p.y.row] = from_float<T>(t < len ? h : 0.0f);
    }
    if (p.state_out) p.state_out[b * p.D + c] = h;
}

template <typename T>
hipError_t fwd_t(const DiagProblem& p, hipStream_t stream)
{
    const dim3 grid = grid_of((int64_t)p.B * ((p.D + 63) / 64));
    switch (p.kind) {
    case kCoupled: diag_fwd_kernel<T, kCoupled><<<grid, 64, 0, stream>>>(p); break;
    case kSigmoid: diag_fwd_kernel<T, kSigmoid><<<grid, 64, 0, stream>>>(p); break;
    default: diag_fwd_kernel<T, kDecay><<<grid, 64, 0, stream>>>(p); break;
    }
    return hipGetLastError();
}

}  // namespace

size_t diag_workspace(const DiagProblem&) { return 0; }

hipError_t launch_diag_fwd(const DiagProblem& p, hipStream_t stream)
{
    return p.bf16 ? fwd_t<bf16>(p, stream) : fwd_t<float>(p, stream);
}

}  // namespace tfla
