// blocks.hpp -- the operators around the recurrences (internal): problem
// descriptions and launchers of the causal convolution, the selective scan,
// the group norm, rotary positions, the gated linear recurrence of channels
// and the residual sum with a norm.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <string>

namespace tfla {

// Records the thread's error message and returns `code` (tfla_api.cpp).
int fail(int code, const std::string& msg);
// Whether a test asked the library's own allocations to fail.
bool inject_alloc_fault();

// A grid of `blocks` workgroups in two dimensions (one holds fewer than 2^32
// threads); a kernel takes its number from block_id() and leaves when that
// is behind the last.
inline dim3 grid_of(int64_t blocks)
{
    const int64_t x = blocks < (1 << 21) ? blocks : (1 << 21);
    return dim3((unsigned)x, (unsigned)((blocks + x - 1) / x));
}

__device__ __forceinline__ int64_t block_id() { return (int64_t)blockIdx.y * gridDim.x + blockIdx.x; }

// Rows of a [B,T,width] tensor: element (b,t,c) at p[b * batch + t * row + c].
struct Rows {
    void* p = nullptr;
    int64_t batch = 0, row = 0;
};

// ---- causal depthwise convolution (conv.hip) ------------------------------------
struct ConvProblem {
    int B, T, D, K;
    bool bf16, silu;
    Rows x, y, dy, dx;
    const float *weight, *bias;
    const int* lengths;
    const void *state, *dstate_out;
    void *state_out, *dstate;
    float *dweight, *dbias;
    float* part;      // backward workspace [parts][K+1][D]: weight and bias gradients of runs of rows
};

size_t conv_bwd_workspace(int B, int T, int D, int K, bool bf16);
hipError_t launch_conv_fwd(const ConvProblem& p, hipStream_t stream);
hipError_t launch_conv_bwd(const ConvProblem& p, hipStream_t stream);

// ---- selective state space scan (scan.hip, scan_bwd.hip) ----------------------------
struct ScanProblem {
    int B, T, D, N, G;
    bool bf16, softplus;
    Rows x, dt, z, bmat, cmat;              // z.p NULL: no gate; bmat, cmat rows of [G][N]
    const float *a, *skip, *dt_bias;        // [D,N], [D] or NULL, [D] or NULL
    const float* state;                     // [B,D,N] or NULL
    const int* lengths;
    Rows y;
    float* state_out;
    // backward
    Rows dy, dx, ddt, dz, dbmat, dcmat;
    const float* dstate_out;
    float *da, *dskip, *ddt_bias, *dstate;
    char* ws;
};

size_t scan_workspace(const ScanProblem& p);
hipError_t launch_scan_fwd(const ScanProblem& p, hipStream_t stream);
size_t scan_bwd_workspace(const ScanProblem& p);
hipError_t launch_scan_bwd(const ScanProblem& p, hipStream_t stream);

// ---- group norm with an activation or a gate (norm.hip) -------------------------------
// Element (b,t,g,c) at p[b * batch + t * row + g * group + c].
struct Heads {
    void* p = nullptr;
    int64_t batch = 0, row = 0, group = 0;
};

enum NormAct { kActNone = 0, kActSilu = 1, kActSigmoid = 2 };

struct NormProblem {
    int B, T, G, C, act;
    bool bf16, sequence;                    // sequence: statistics over T and C, else over C
    float eps;
    Heads x, gate, y;                       // gate.p NULL: y = act(u), else u act(gate)
    const float *weight, *bias;             // [G,C] or NULL
    float *mean, *rstd;                     // forward outputs (NULL: not wanted), backward inputs
    Heads dy, dx, dgate;
    float *dweight, *dbias;
    char* ws;
};

size_t norm_workspace(const NormProblem& p);
hipError_t launch_norm_fwd(const NormProblem& p, hipStream_t stream);
size_t norm_bwd_workspace(const NormProblem& p);
hipError_t launch_norm_bwd(const NormProblem& p, hipStream_t stream);

// ---- rotary positions (rotary.hip) -------------------------------------------------------
struct RotaryProblem {
    int B, T, H, Hk, C, R;
    bool bf16, interleaved, inverse;        // inverse: the turn by minus the angle (backward)
    float scale;
    const double* freqs;                    // [R/2]
    const int* positions;                   // row b at positions + b * positions_batch, or NULL
    int64_t positions_batch;
    const int *start, *lengths;             // [B] or NULL
    Heads q, k, q_out, k_out;
};

hipError_t launch_rotary(const RotaryProblem& p, hipStream_t stream);

// ---- gated linear recurrence of channels (diag.hip, diag_bwd.hip) ------------------------
enum DiagKind { kCoupled = 0, kSigmoid = 1, kDecay = 2 };

struct DiagProblem {
    int B, T, D, kind;
    bool bf16;
    Rows x, fgate, igate;                   // igate.p NULL: coupled
    const float* decay;                     // [D], kDecay only
    const int* lengths;
    const float* state;                     // [B,D] or NULL
    Rows y;
    float *state_out, *starts;              // [B,D], [B,chunks,D] or NULL
    // backward
    Rows dy, dx, dfgate, digate;
    const float* dstate_out;
    float *ddecay, *dstate;
    char* ws;
};

size_t diag_workspace(const DiagProblem& p);
hipError_t launch_diag_fwd(const DiagProblem& p, hipStream_t stream);
size_t diag_bwd_workspace(const DiagProblem& p);
hipError_t launch_diag_bwd(const DiagProblem& p, hipStream_t stream);

// ---- residual sum with a norm (addnorm.hip, addnorm_bwd.hip) -------------------------------
struct AddNormProblem {
    int B, T, C;
    bool bf16, sum_fp32, rms;               // sum_fp32: the stream is fp32 beside bf16 activations
    float eps;
    Rows x, residual, y, total;             // residual.p, total.p NULL: no residual
    const float *weight, *bias;             // [C] or NULL
    // backward
    Rows dy, dtotal, dx, dresidual;
    float *dweight, *dbias;
    char* ws;
};

hipError_t launch_addnorm_fwd(const AddNormProblem& p, hipStream_t stream);
size_t addnorm_bwd_workspace(const AddNormProblem& p);
hipError_t launch_addnorm_bwd(const AddNormProblem& p, hipStream_t stream);

}  // namespace tfla
