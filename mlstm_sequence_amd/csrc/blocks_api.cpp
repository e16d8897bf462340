// blocks_api.cpp -- C entry points of the operators around the recurrences
// (include/tfla.h): argument checks (no HIP call before they pass), workspace
// and launches.  No exception leaves an entry point.
#include "checks.hpp"

namespace {

using namespace tfla::checks;
using tfla::fail;

// ---- causal convolution ---------------------------------------------------------------

int check_conv_sizes(int B, int T, int D, int K, int flags)
{
    int rc = check_flags(flags);
    if (rc) return rc;
    if (B < 1 || T < 1 || D < 1 || K < 1) return fail(TFLA_ERR_INVALID_ARG, "B, T, D and K must be >= 1");
    if (K > 8) return fail(TFLA_ERR_UNSUPPORTED, "K must be 1 to 8, got " + std::to_string(K));
    if ((int64_t)B * T > kMaxRows) return fail(TFLA_ERR_UNSUPPORTED, "B*T must be <= 2^30");
    if (D > (1 << 24)) return fail(TFLA_ERR_UNSUPPORTED, "D must be <= 2^24");
    return TFLA_OK;
}

int check_conv(const tfla_conv_args* a, bool bwd, tfla::ConvProblem* p, View* views, size_t* nv)
{
    if (!a) return fail(TFLA_ERR_INVALID_ARG, "args is NULL");
    int rc = check_conv_sizes(a->B, a->T, a->D, a->K, a->flags);
    if (rc) return rc;
    if (a->act != TFLA_ACT_NONE && a->act != TFLA_ACT_SILU)
        return fail(TFLA_ERR_INVALID_ARG, "act must be TFLA_ACT_NONE or TFLA_ACT_SILU");
    const bool bf16 = (a->flags & TFLA_IO_BF16) != 0;
    const size_t e = bf16 ? 2 : 4;
    const int64_t D = a->D, K = a->K, B = a->B;
    const void* state = K > 1 ? a->state : nullptr;
    void* state_out = K > 1 && !bwd ? a->state_out : nullptr;
    const void* dso = K > 1 && bwd ? a->dstate_out : nullptr;
    void* dstate = K > 1 && bwd ? a->dstate : nullptr;
    if ((rc = check_aligned("x", a->x.data, e, true)) || (rc = check_aligned("weight", a->weight, 4, true)) ||
        (rc = check_aligned("bias", a->bias, 4, false)) || (rc = check_aligned("state", state, e, false)) ||
        (rc = check_aligned("lengths", a->lengths, 4, false)))
        return rc;
    const int64_t sb = B * (K - 1) * D * (int64_t)e;
    size_t n = 0;
    views[n++] = rows("x", a->x, a->B, a->T, D, e);
    views[n++] = flat("weight", a->weight, D * K * 4);
    views[n++] = flat("bias", a->bias, D * 4);
    views[n++] = flat("state", state, sb);
    views[n++] = flat("lengths", a->lengths, B * 4);
    size_t no = 0;
    if (!bwd) {
        if ((rc = check_aligned("y", a->y.data, e, true)) || (rc = check_aligned("state_out", state_out, e, false)))
            return rc;
        views[n + no++] = rows("y", a->y, a->B, a->T, D, e);
        views[n + no++] = flat("state_out", state_out, sb);
    } else {
        if ((rc = check_aligned("dy", a->dy.data, e, true)) || (rc = check_aligned("dstate_out", dso, e, false)) ||
            (rc = check_aligned("dx", a->dx.data, e, true)) || (rc = check_aligned("dweight", a->dweight, 4, true)) ||
            (rc = check_aligned("dbias", a->dbias, 4, false)) || (rc = check_aligned("dstate", dstate, e, false)))
            return rc;
        if ((a->bias == nullptr) != (a->dbias == nullptr))
            return fail(TFLA_ERR_INVALID_ARG, "dbias must be given exactly when bias is");
        views[n++] = rows("dy", a->dy, a->B, a->T, D, e);
        views[n++] = flat("dstate_out", dso, sb);
        views[n + no++] = rows("dx", a->dx, a->B, a->T, D, e);
        views[n + no++] = flat("dweight", a->dweight, D * K * 4);
        views[n + no++] = flat("dbias", a->dbias, D * 4);
        views[n + no++] = flat("dstate", dstate, sb);
    }
    const int twin[2] = {-1, 3};   // state_out may be state
    if ((rc = check_views(views, n, views + n, no, bwd ? nullptr : twin))) return rc;
    *nv = n + no;
    *p = tfla::ConvProblem{};
    p->B = a->B;
    p->T = a->T;
    p->D = a->D;
    p->K = a->K;
    p->bf16 = bf16;
    p->silu = a->act == TFLA_ACT_SILU;
    p->x = dev(a->x);
    p->weight = a->weight;
    p->bias = a->bias;
    p->lengths = a->lengths;
    p->state = state;
    p->state_out = state_out;
    p->dstate_out = dso;
    p->dstate = dstate;
    if (bwd) {
        p->dy = dev(a->dy);
        p->dx = dev(a->dx);
        p->dweight = a->dweight;
        p->dbias = a->dbias;
    } else {
        p->y = dev(a->y);
    }
    return TFLA_OK;
}

// ---- selective scan ---------------------------------------------------------------------

int check_scan_sizes(int B, int T, int D, int N, int G, int flags, tfla::ScanProblem* p)
{
    if (flags & ~(TFLA_IO_BF16 | TFLA_SCAN_SOFTPLUS))
        return fail(TFLA_ERR_INVALID_ARG, "unknown flags " + std::to_string(flags));
    if (B < 1 || T < 1 || D < 1 || N < 1 || G < 1)
        return fail(TFLA_ERR_INVALID_ARG, "B, T, D, N and G must be >= 1");
    if (D % G) return fail(TFLA_ERR_INVALID_ARG, "G must divide D");
    if (N > 64) return fail(TFLA_ERR_UNSUPPORTED, "N must be 1 to 64, got " + std::to_string(N));
    if ((int64_t)B * T > kMaxRows) return fail(TFLA_ERR_UNSUPPORTED, "B*T must be <= 2^30");
    if (D > (1 << 24)) return fail(TFLA_ERR_UNSUPPORTED, "D must be <= 2^24");
    // workgroups of up to 1024 threads, a grid below 2^32 of them
    if ((int64_t)B * G * ((D / G + 63) / 64) >= (1 << 21))
        return fail(TFLA_ERR_UNSUPPORTED, "B*D too large: blocks of 64 channels of a group must be below 2^21");
    *p = tfla::ScanProblem{};
    p->B = B;
    p->T = T;
    p->D = D;
    p->N = N;
    p->G = G;
    p->bf16 = (flags & TFLA_IO_BF16) != 0;
    p->softplus = (flags & TFLA_SCAN_SOFTPLUS) != 0;
    return TFLA_OK;
}

int check_scan(const tfla_scan_args* a, bool bwd, tfla::ScanProblem* p, View* views, size_t* nv)
{
    if (!a) return fail(TFLA_ERR_INVALID_ARG, "args is NULL");
    const int B = a->B, T = a->T;
    int rc = check_scan_sizes(B, T, a->D, a->N, a->G, a->flags, p);
    if (rc) return rc;
    const int64_t D = a->D, GN = (int64_t)a->G * a->N, e = p->bf16 ? 2 : 4;
    const int64_t sb = (int64_t)B * D * a->N * 4, ab = D * a->N * 4;
    size_t n = 0;
    auto in_rows = [&](const char* name, const tfla_rows& r, int64_t w, bool required) {
        views[n++] = rows(name, r, B, T, w, e);
        return check_aligned(name, r.data, e, required);
    };
    auto in_flat = [&](const char* name, const void* q, int64_t bytes, bool required) {
        views[n++] = flat(name, q, bytes);
        return check_aligned(name, q, 4, required);
    };
    if ((rc = in_rows("x", a->x, D, true)) || (rc = in_rows("dt", a->dt, D, true)) ||
        (rc = in_rows("z", a->z, D, false)) || (rc = in_rows("bmat", a->bmat, GN, true)) ||
        (rc = in_rows("cmat", a->cmat, GN, true)) || (rc = in_flat("a", a->a, ab, true)) ||
        (rc = in_flat("skip", a->skip, D * 4, false)) || (rc = in_flat("dt_bias", a->dt_bias, D * 4, false)) ||
        (rc = in_flat("state", a->state, sb, false)) || (rc = in_flat("lengths", a->lengths, (int64_t)B * 4, false)))
        return rc;
    if (bwd && ((rc = in_rows("dy", a->dy, D, true)) || (rc = in_flat("dstate_out", a->dstate_out, sb, false))))
        return rc;
    const size_t ni = n;
    if (!bwd) {
        if ((rc = in_rows("y", a->y, D, true)) || (rc = in_flat("state_out", a->state_out, sb, false))) return rc;
    } else {
        if ((rc = in_rows("dx", a->dx, D, true)) || (rc = in_rows("ddt", a->ddt, D, true)) ||
            (rc = in_rows("dz", a->dz, D, false)) || (rc = in_rows("dbmat", a->dbmat, GN, true)) ||
            (rc = in_rows("dcmat", a->dcmat, GN, true)) || (rc = in_flat("da", a->da, ab, true)) ||
            (rc = in_flat("dskip", a->dskip, D * 4, false)) || (rc = in_flat("ddt_bias", a->ddt_bias, D * 4, false)) ||
            (rc = in_flat("dstate", a->dstate, sb, false)))
            return rc;
        if (!a->z.data != !a->dz.data || !a->skip != !a->dskip || !a->dt_bias != !a->ddt_bias)
            return fail(TFLA_ERR_INVALID_ARG, "dz, dskip and ddt_bias must be given exactly when z, skip and dt_bias are");
    }
    const int twin[2] = {-1, 8};   // state_out may be state
    if ((rc = check_views(views, ni, views + ni, n - ni, bwd ? nullptr : twin))) return rc;
    *nv = n;
    p->x = dev(a->x);
    p->dt = dev(a->dt);
    p->z = dev(a->z);
    p->bmat = dev(a->bmat);
    p->cmat = dev(a->cmat);
    p->a = a->a;
    p->skip = a->skip;
    p->dt_bias = a->dt_bias;
    p->state = a->state;
    p->lengths = a->lengths;
    if (!bwd) {
        p->y = dev(a->y);
        p->state_out = a->state_out;
        return TFLA_OK;
    }
    p->dy = dev(a->dy);
    p->dstate_out = a->dstate_out;
    p->dx = dev(a->dx);
    p->ddt = dev(a->ddt);
    p->dz = dev(a->dz);
    p->dbmat = dev(a->dbmat);
    p->dcmat = dev(a->dcmat);
    p->da = a->da;
    p->dskip = a->dskip;
    p->ddt_bias = a->ddt_bias;
    p->dstate = a->dstate;
    return TFLA_OK;
}

int run_scan(const tfla_scan_args* args, bool bwd, void* workspace, size_t workspace_bytes, void* stream)
{
    tfla::ScanProblem p;
    View views[32];
    size_t nv;
    int rc = check_scan(args, bwd, &p, views, &nv);
    if (rc) return rc;
    hipStream_t s = static_cast<hipStream_t>(stream);
    const size_t need = bwd ? tfla::scan_bwd_workspace(p) : tfla::scan_workspace(p);
    return with_workspace(workspace, workspace_bytes, need, views, nv, s, [&](char* base) {
        p.ws = base;
        return bwd ? hip_status(tfla::launch_scan_bwd(p, s), "scan gradient kernel launch")
                   : hip_status(tfla::launch_scan_fwd(p, s), "scan kernel launch");
    });
}

// ---- group norm -----------------------------------------------------------------------

int check_norm_sizes(int B, int T, int G, int C, int flags, tfla::NormProblem* p)
{
    if (flags & ~(TFLA_IO_BF16 | TFLA_NORM_SEQUENCE))
        return fail(TFLA_ERR_INVALID_ARG, "unknown flags " + std::to_string(flags));
    if (B < 1 || T < 1 || G < 1 || C < 1) return fail(TFLA_ERR_INVALID_ARG, "B, T, G and C must be >= 1");
    if ((int64_t)B * T > kMaxRows) return fail(TFLA_ERR_UNSUPPORTED, "B*T must be <= 2^30");
    if ((int64_t)G * C > (1 << 24)) return fail(TFLA_ERR_UNSUPPORTED, "G*C must be <= 2^24");
    if ((int64_t)B * T * G >= (int64_t(1) << 31)) return fail(TFLA_ERR_UNSUPPORTED, "B*T*G must be below 2^31");
    // the sequence's statistics: a workgroup to a set, partial sums counted in 32 bits
    if ((flags & TFLA_NORM_SEQUENCE) && ((int64_t)B * G > (1 << 20) || (int64_t)(T / 16 + 1) * C >= (int64_t(1) << 31)))
        return fail(TFLA_ERR_UNSUPPORTED, "TFLA_NORM_SEQUENCE: B*G must be <= 2^20 and T*C/16 below 2^31");
    *p = tfla::NormProblem{};
    p->B = B;
    p->T = T;
    p->G = G;
    p->C = C;
    p->bf16 = (flags & TFLA_IO_BF16) != 0;
    p->sequence = (flags & TFLA_NORM_SEQUENCE) != 0;
    return TFLA_OK;
}

int check_norm(const tfla_norm_args* a, bool bwd, tfla::NormProblem* p, View* views, size_t* nv)
{
    if (!a) return fail(TFLA_ERR_INVALID_ARG, "args is NULL");
    int rc = check_norm_sizes(a->B, a->T, a->G, a->C, a->flags, p);
    if (rc) return rc;
    if (a->act != TFLA_ACT_NONE && a->act != TFLA_ACT_SILU && a->act != TFLA_ACT_SIGMOID)
        return fail(TFLA_ERR_INVALID_ARG, "unknown act " + std::to_string(a->act));
    if (!bwd && !(a->eps > 0.0f)) return fail(TFLA_ERR_INVALID_ARG, "eps must be > 0");
    const int64_t e = p->bf16 ? 2 : 4, wb = (int64_t)a->G * a->C * 4;
    const int64_t sb = (int64_t)a->B * (p->sequence ? 1 : a->T) * a->G * 4;
    size_t n = 0;
    auto strided = [&](const char* name, const tfla_heads& r, bool required) {
        views[n++] = heads(name, r, a->B, a->T, a->G, a->C, e);
        return check_aligned(name, r.data, e, required);
    };
    auto plain = [&](const char* name, const void* q, int64_t bytes, bool required) {
        views[n++] = flat(name, q, bytes);
        return check_aligned(name, q, 4, required);
    };
    if ((rc = strided("x", a->x, true)) || (rc = strided("gate", a->gate, false)) ||
        (rc = plain("weight", a->weight, wb, false)) || (rc = plain("bias", a->bias, wb, false)))
        return rc;
    if (bwd && ((rc = strided("dy", a->dy, true)) || (rc = plain("mean", a->mean, sb, true)) ||
                (rc = plain("rstd", a->rstd, sb, true))))
        return rc;
    const size_t ni = n;
    if (!bwd) {
        if ((rc = strided("y", a->y, true)) || (rc = plain("mean", a->mean, sb, false)) ||
            (rc = plain("rstd", a->rstd, sb, false)))
            return rc;
    } else {
        if ((rc = strided("dx", a->dx, true)) || (rc = strided("dgate", a->dgate, false)) ||
            (rc = plain("dweight", a->dweight, wb, false)) || (rc = plain("dbias", a->dbias, wb, false)))
            return rc;
        if (!a->gate.data != !a->dgate.data || !a->weight != !a->dweight || !a->bias != !a->dbias)
            return fail(TFLA_ERR_INVALID_ARG, "dgate, dweight and dbias must be given exactly when gate, weight and bias are");
    }
    if ((rc = check_views(views, ni, views + ni, n - ni))) return rc;
    *nv = n;
    p->act = a->act;
    p->eps = a->eps;
    p->x = dev(a->x);
    p->gate = dev(a->gate);
    p->weight = a->weight;
    p->bias = a->bias;
    p->mean = a->mean;
    p->rstd = a->rstd;
    if (!bwd) {
        p->y = dev(a->y);
        return TFLA_OK;
    }
    p->dy = dev(a->dy);
    p->dx = dev(a->dx);
    p->dgate = dev(a->dgate);
    p->dweight = a->dweight;
    p->dbias = a->dbias;
    return TFLA_OK;
}

int run_norm(const tfla_norm_args* args, bool bwd, void* workspace, size_t workspace_bytes, void* stream)
{
    tfla::NormProblem p;
    View views[16];
    size_t nv;
    int rc = check_norm(args, bwd, &p, views, &nv);
    if (rc) return rc;
    hipStream_t s = static_cast<hipStream_t>(stream);
    const size_t need = bwd ? tfla::norm_bwd_workspace(p) : tfla::norm_workspace(p);
    return with_workspace(workspace, workspace_bytes, need, views, nv, s, [&](char* base) {
        p.ws = base;
        return bwd ? hip_status(tfla::launch_norm_bwd(p, s), "norm gradient kernel launch")
                   : hip_status(tfla::launch_norm_fwd(p, s), "norm kernel launch");
    });
}

}  // namespace

extern "C" {

size_t tfla_norm_workspace_bytes(int B, int T, int G, int C, int flags)
{
    tfla::NormProblem p;
    const int rc = guarded([&]() -> int { return check_norm_sizes(B, T, G, C, flags, &p); });
    return rc == TFLA_OK ? tfla::norm_workspace(p) : 0;
}

int tfla_norm_fwd(const tfla_norm_args* args, void* workspace, size_t workspace_bytes, void* stream)
{
    return guarded([&]() -> int { return run_norm(args, false, workspace, workspace_bytes, stream); });
}

size_t tfla_norm_bwd_workspace_bytes(int B, int T, int G, int C, int flags)
{
    tfla::NormProblem p;
    const int rc = guarded([&]() -> int { return check_norm_sizes(B, T, G, C, flags, &p); });
    return rc == TFLA_OK ? tfla::norm_bwd_workspace(p) : 0;
}

int tfla_norm_bwd(const tfla_norm_args* args, void* workspace, size_t workspace_bytes, void* stream)
{
    return guarded([&]() -> int { return run_norm(args, true, workspace, workspace_bytes, stream); });
}

size_t tfla_scan_workspace_bytes(int B, int T, int D, int N, int G, int flags)
{
    tfla::ScanProblem p;
    const int rc = guarded([&]() -> int { return check_scan_sizes(B, T, D, N, G, flags, &p); });
    return rc == TFLA_OK ? tfla::scan_workspace(p) : 0;
}

int tfla_scan_fwd(const tfla_scan_args* args, void* workspace, size_t workspace_bytes, void* stream)
{
    return guarded([&]() -> int { return run_scan(args, false, workspace, workspace_bytes, stream); });
}

size_t tfla_scan_bwd_workspace_bytes(int B, int T, int D, int N, int G, int flags)
{
    tfla::ScanProblem p;
    const int rc = guarded([&]() -> int { return check_scan_sizes(B, T, D, N, G, flags, &p); });
    return rc == TFLA_OK ? tfla::scan_bwd_workspace(p) : 0;
}

int tfla_scan_bwd(const tfla_scan_args* args, void* workspace, size_t workspace_bytes, void* stream)
{
    return guarded([&]() -> int { return run_scan(args, true, workspace, workspace_bytes, stream); });
}

int tfla_conv_fwd(const tfla_conv_args* args, void* stream)
{
    return guarded([&]() -> int {
        tfla::ConvProblem p;
        View views[16];
        size_t nv;
        int rc = check_conv(args, false, &p, views, &nv);
        if (rc) return rc;
        return hip_status(tfla::launch_conv_fwd(p, static_cast<hipStream_t>(stream)), "convolution kernel launch");
    });
}

size_t tfla_conv_bwd_workspace_bytes(int B, int T, int D, int K, int flags)
{
    size_t n = 0;
    if (guarded([&]() -> int { return check_conv_sizes(B, T, D, K, flags); }) == TFLA_OK)
        n = tfla::conv_bwd_workspace(B, T, D, K, (flags & TFLA_IO_BF16) != 0);
    return n;
}

int tfla_conv_bwd(const tfla_conv_args* args, void* workspace, size_t workspace_bytes, void* stream)
{
    return guarded([&]() -> int {
        tfla::ConvProblem p;
        View views[16];
        size_t nv;
        int rc = check_conv(args, true, &p, views, &nv);
        if (rc) return rc;
        hipStream_t s = static_cast<hipStream_t>(stream);
        const size_t need = tfla::conv_bwd_workspace(p.B, p.T, p.D, p.K, p.bf16);
        return with_workspace(workspace, workspace_bytes, need, views, nv, s, [&](char* base) {
            p.part = reinterpret_cast<float*>(base);
            return hip_status(tfla::launch_conv_bwd(p, s), "convolution gradient kernel launch");
        });
    });
}

}  // extern "C"
