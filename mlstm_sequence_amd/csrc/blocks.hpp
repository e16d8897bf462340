// blocks.hpp -- the operators around the recurrences (internal): problem
// descriptions and launchers of the causal convolution, the selective scan
// and the group norm.
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

}  // namespace tfla
