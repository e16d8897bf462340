// edges_api.cpp -- C entry points of rotary positions, the gated linear
// recurrence of channels and the residual sum with a norm (include/tfla.h):
// argument checks (no HIP call before they pass), workspace and launches.
// No exception leaves an entry point.
#include "checks.hpp"

namespace {

using namespace tfla::checks;
using tfla::fail;

// Views of a call's tensors, inputs first.
struct Views {
    View v[16];
    size_t n = 0, ni = 0;   // all, inputs
    int add(const View& view, const void* p, size_t align, bool required)
    {
        v[n++] = view;
        return check_aligned(view.name, p, align, required);
    }
    int check(const int* twin = nullptr) const { return check_views(v, ni, v + ni, n - ni, twin); }
};

// ---- rotary positions -----------------------------------------------------------------

int check_rotary(const tfla_rotary_args* a, bool bwd, tfla::RotaryProblem* p)
{
    if (!a) return fail(TFLA_ERR_INVALID_ARG, "args is NULL");
    if (a->flags & ~(TFLA_IO_BF16 | TFLA_ROTARY_INTERLEAVED))
        return fail(TFLA_ERR_INVALID_ARG, "unknown flags " + std::to_string(a->flags));
    const int B = a->B, T = a->T, H = a->H, Hk = a->Hk, C = a->C, R = a->R;
    if (B < 1 || T < 1 || H < 1 || C < 1) return fail(TFLA_ERR_INVALID_ARG, "B, T, H and C must be >= 1");
    if (Hk < 0) return fail(TFLA_ERR_INVALID_ARG, "Hk must be >= 0");
    if (R < 0 || R > C || R % 2) return fail(TFLA_ERR_INVALID_ARG, "R must be even, 0 to C");
    if (C > 1024) return fail(TFLA_ERR_UNSUPPORTED, "C must be <= 1024, got " + std::to_string(C));
    if ((int64_t)B * T > kMaxRows) return fail(TFLA_ERR_UNSUPPORTED, "B*T must be <= 2^30");
    if (((int64_t)H + Hk) * C > (1 << 24)) return fail(TFLA_ERR_UNSUPPORTED, "(H+Hk)*C must be <= 2^24");
    if (a->positions && a->start) return fail(TFLA_ERR_INVALID_ARG, "positions and start must not both be given");
    const int64_t e = a->flags & TFLA_IO_BF16 ? 2 : 4;
    Views w;
    int rc;
    const tfla_heads none{nullptr, 0, 0, 0};
    const tfla_heads &k = Hk ? a->k : none, &k_out = Hk ? a->k_out : none;
    const tfla_rows pos{const_cast<int*>(a->positions), a->positions_batch, 0};
    if ((rc = w.add(heads("q", a->q, B, T, H, C, e), a->q.data, e, true)) ||
        (rc = w.add(heads("k", k, B, T, Hk, C, e), k.data, e, Hk > 0)) ||
        (rc = w.add(flat("freqs", a->freqs, (int64_t)(R / 2) * 8), a->freqs, 8, R > 0)) ||
        (rc = w.add(rows("positions", pos, B, 1, T, 4), a->positions, 4, false)) ||
        (rc = w.add(flat("start", a->start, (int64_t)B * 4), a->start, 4, false)) ||
        (rc = w.add(flat("lengths", a->lengths, (int64_t)B * 4), a->lengths, 4, false)))
        return rc;
    w.ni = w.n;
    if ((rc = w.add(heads("q_out", a->q_out, B, T, H, C, e), a->q_out.data, e, true)) ||
        (rc = w.add(heads("k_out", k_out, B, T, Hk, C, e), k_out.data, e, Hk > 0)))
        return rc;
    const int twin[2] = {0, 1};   // q_out may be q, k_out k
    if ((rc = w.check(twin))) return rc;
    *p = tfla::RotaryProblem{};
    p->B = B;
    p->T = T;
    p->H = H;
    p->Hk = Hk;
    p->C = C;
    p->R = R;
    p->bf16 = (a->flags & TFLA_IO_BF16) != 0;
    p->interleaved = (a->flags & TFLA_ROTARY_INTERLEAVED) != 0;
    p->inverse = bwd;
    p->scale = a->scale;
    p->freqs = a->freqs;
    p->positions = a->positions;
    p->positions_batch = a->positions_batch;
    p->start = a->start;
    p->lengths = a->lengths;
    p->q = dev(a->q);
    p->k = dev(k);
    p->q_out = dev(a->q_out);
    p->k_out = dev(k_out);
    return TFLA_OK;
}

int run_rotary(const tfla_rotary_args* args, bool bwd, void* stream)
{
    tfla::RotaryProblem p;
    int rc = check_rotary(args, bwd, &p);
    if (rc) return rc;
    return hip_status(tfla::launch_rotary(p, static_cast<hipStream_t>(stream)), "rotary kernel launch");
}

// ---- gated linear recurrence of channels --------------------------------------------------

int check_diag_sizes(int B, int T, int D, int kind, int flags, tfla::DiagProblem* p)
{
    int rc = check_flags(flags);
    if (rc) return rc;
    if (B < 1 || T < 1 || D < 1) return fail(TFLA_ERR_INVALID_ARG, "B, T and D must be >= 1");
    if (kind != TFLA_DIAG_COUPLED && kind != TFLA_DIAG_SIGMOID && kind != TFLA_DIAG_DECAY)
        return fail(TFLA_ERR_INVALID_ARG, "unknown kind " + std::to_string(kind));
    if ((int64_t)B * T > kMaxRows) return fail(TFLA_ERR_UNSUPPORTED, "B*T must be <= 2^30");
    if (D > (1 << 24)) return fail(TFLA_ERR_UNSUPPORTED, "D must be <= 2^24");
    *p = tfla::DiagProblem{};
    p->B = B;
    p->T = T;
    p->D = D;
    p->kind = kind;
    p->bf16 = (flags & TFLA_IO_BF16) != 0;
    return TFLA_OK;
}

int check_diag(const tfla_diag_args* a, bool bwd, tfla::DiagProblem* p, Views* w)
{
    if (!a) return fail(TFLA_ERR_INVALID_ARG, "args is NULL");
    const int B = a->B, T = a->T, D = a->D;
    int rc = check_diag_sizes(B, T, D, a->kind, a->flags, p);
    if (rc) return rc;
    const int64_t e = p->bf16 ? 2 : 4, sb = (int64_t)B * D * 4, db = (int64_t)D * 4;
    const int64_t cb = sb * (((int64_t)T + TFLA_DIAG_CHUNK - 1) / TFLA_DIAG_CHUNK);
    const bool two = a->kind != TFLA_DIAG_COUPLED, dec = a->kind == TFLA_DIAG_DECAY;
    const tfla_rows none{nullptr, 0, 0};
    auto strided = [&](const char* name, const tfla_rows& r, bool used) {
        return w->add(rows(name, used ? r : none, B, T, D, e), used ? r.data : nullptr, e, used);
    };
    auto plain = [&](const char* name, const void* q, int64_t bytes, bool required) {
        return w->add(flat(name, q, bytes), q, 4, required);
    };
    const float* decay = dec ? a->decay : nullptr;
    if ((rc = strided("x", a->x, true)) || (rc = strided("fgate", a->fgate, true)) ||
        (rc = strided("igate", a->igate, two)) || (rc = plain("decay", decay, db, dec)) ||
        (rc = plain("lengths", a->lengths, (int64_t)B * 4, false)))
        return rc;
    if (!bwd) {
        if ((rc = plain("state", a->state, sb, false))) return rc;
        w->ni = w->n;
        if ((rc = strided("y", a->y, true)) || (rc = plain("state_out", a->state_out, sb, false)) ||
            (rc = plain("starts", a->starts, cb, false)))
            return rc;
        const int twin[3] = {-1, 5, -1};   // state_out may be state
        if ((rc = w->check(twin))) return rc;
    } else {
        if ((rc = plain("starts", a->starts, cb, true)) || (rc = strided("dy", a->dy, true)) ||
            (rc = plain("dstate_out", a->dstate_out, sb, false)))
            return rc;
        w->ni = w->n;
        if ((rc = strided("dx", a->dx, true)) || (rc = strided("dfgate", a->dfgate, true)) ||
            (rc = strided("digate", a->digate, two)) || (rc = plain("ddecay", dec ? a->ddecay : nullptr, db, dec)) ||
            (rc = plain("dstate", a->dstate, sb, false)))
            return rc;
        if ((rc = w->check())) return rc;
    }
    p->x = dev(a->x);
    p->fgate = dev(a->fgate);
    p->igate = dev(two ? a->igate : none);
    p->decay = decay;
    p->lengths = a->lengths;
    p->starts = a->starts;
    if (!bwd) {
        p->state = a->state;
        p->y = dev(a->y);
        p->state_out = a->state_out;
        return TFLA_OK;
    }
    p->dy = dev(a->dy);
    p->dstate_out = a->dstate_out;
    p->dx = dev(a->dx);
    p->dfgate = dev(a->dfgate);
    p->digate = dev(two ? a->digate : none);
    p->ddecay = dec ? a->ddecay : nullptr;
    p->dstate = a->dstate;
    return TFLA_OK;
}

int run_diag(const tfla_diag_args* args, bool bwd, void* workspace, size_t workspace_bytes, void* stream)
{
    tfla::DiagProblem p;
    Views w;
    int rc = check_diag(args, bwd, &p, &w);
    if (rc) return rc;
    hipStream_t s = static_cast<hipStream_t>(stream);
    const size_t need = bwd ? tfla::diag_bwd_workspace(p) : tfla::diag_workspace(p);
    return with_workspace(workspace, workspace_bytes, need, w.v, w.n, s, [&](char* base) {
        p.ws = base;
        return bwd ? hip_status(tfla::launch_diag_bwd(p, s), "recurrence gradient kernel launch")
                   : hip_status(tfla::launch_diag_fwd(p, s), "recurrence kernel launch");
    });
}

// ---- residual sum with a norm ---------------------------------------------------------------

int check_addnorm_sizes(int B, int T, int C, int flags, tfla::AddNormProblem* p)
{
    if (flags & ~(TFLA_IO_BF16 | TFLA_ADDNORM_RMS | TFLA_ADDNORM_SUM_FP32))
        return fail(TFLA_ERR_INVALID_ARG, "unknown flags " + std::to_string(flags));
    if (B < 1 || T < 1 || C < 1) return fail(TFLA_ERR_INVALID_ARG, "B, T and C must be >= 1");
    if ((int64_t)B * T > kMaxRows) return fail(TFLA_ERR_UNSUPPORTED, "B*T must be <= 2^30");
    if (C > (1 << 24)) return fail(TFLA_ERR_UNSUPPORTED, "C must be <= 2^24");
    *p = tfla::AddNormProblem{};
    p->B = B;
    p->T = T;
    p->C = C;
    p->bf16 = (flags & TFLA_IO_BF16) != 0;
    p->sum_fp32 = p->bf16 && (flags & TFLA_ADDNORM_SUM_FP32);   // fp32 activations have an fp32 stream as it is
    p->rms = (flags & TFLA_ADDNORM_RMS) != 0;
    return TFLA_OK;
}

int check_addnorm(const tfla_addnorm_args* a, bool bwd, tfla::AddNormProblem* p, Views* w)
{
    if (!a) return fail(TFLA_ERR_INVALID_ARG, "args is NULL");
    const int B = a->B, T = a->T, C = a->C;
    int rc = check_addnorm_sizes(B, T, C, a->flags, p);
    if (rc) return rc;
    if (!(a->eps > 0.0f)) return fail(TFLA_ERR_INVALID_ARG, "eps must be > 0");
    const int64_t e = p->bf16 ? 2 : 4, es = p->sum_fp32 ? 4 : e, wb = (int64_t)C * 4;
    auto strided = [&](const char* name, const tfla_rows& r, int64_t size, bool required) {
        return w->add(rows(name, r, B, T, C, size), r.data, size, required);
    };
    auto plain = [&](const char* name, const void* q, bool required = false) {
        return w->add(flat(name, q, wb), q, 4, required);
    };
    if ((rc = plain("weight", a->weight))) return rc;
    if (!bwd) {
        const bool sum = a->residual.data != nullptr;
        if ((rc = strided("x", a->x, e, true)) || (rc = strided("residual", a->residual, es, false)) ||
            (rc = plain("bias", a->bias)))
            return rc;
        if (sum != (a->total.data != nullptr))
            return fail(TFLA_ERR_INVALID_ARG, "total must be given exactly when residual is");
        w->ni = w->n;
        if ((rc = strided("y", a->y, e, true)) || (rc = strided("total", a->total, es, false))) return rc;
        const int twin[2] = {-1, 2};   // total may be residual
        if ((rc = w->check(twin))) return rc;
    } else {
        if (a->dresidual.data && !p->sum_fp32)
            return fail(TFLA_ERR_INVALID_ARG, "dresidual is dx unless TFLA_ADDNORM_SUM_FP32 tells their types apart");
        if ((rc = strided("total", a->total, es, true)) || (rc = strided("dy", a->dy, e, true)) ||
            (rc = strided("dtotal", a->dtotal, es, false)))
            return rc;
        w->ni = w->n;
        if ((rc = strided("dx", a->dx, e, true)) || (rc = strided("dresidual", a->dresidual, es, false)) ||
            (rc = plain("dweight", a->dweight)) || (rc = plain("dbias", a->dbias)))
            return rc;
        if ((rc = w->check())) return rc;
    }
    p->eps = a->eps;
    p->weight = a->weight;
    p->total = dev(a->total);
    if (!bwd) {
        p->x = dev(a->x);
        p->residual = dev(a->residual);
        p->bias = a->bias;
        p->y = dev(a->y);
        return TFLA_OK;
    }
    p->dy = dev(a->dy);
    p->dtotal = dev(a->dtotal);
    p->dx = dev(a->dx);
    p->dresidual = dev(a->dresidual);
    p->dweight = a->dweight;
    p->dbias = a->dbias;
    return TFLA_OK;
}

}  // namespace

extern "C" {

int tfla_rotary_fwd(const tfla_rotary_args* args, void* stream)
{
    return guarded([&]() -> int { return run_rotary(args, false, stream); });
}

int tfla_rotary_bwd(const tfla_rotary_args* args, void* stream)
{
    return guarded([&]() -> int { return run_rotary(args, true, stream); });
}

size_t tfla_diag_workspace_bytes(int B, int T, int D, int kind, int flags)
{
    tfla::DiagProblem p;
    const int rc = guarded([&]() -> int { return check_diag_sizes(B, T, D, kind, flags, &p); });
    return rc == TFLA_OK ? tfla::diag_workspace(p) : 0;
}

int tfla_diag_fwd(const tfla_diag_args* args, void* workspace, size_t workspace_bytes, void* stream)
{
    return guarded([&]() -> int { return run_diag(args, false, workspace, workspace_bytes, stream); });
}

size_t tfla_diag_bwd_workspace_bytes(int B, int T, int D, int kind, int flags)
{
    tfla::DiagProblem p;
    const int rc = guarded([&]() -> int { return check_diag_sizes(B, T, D, kind, flags, &p); });
    return rc == TFLA_OK ? tfla::diag_bwd_workspace(p) : 0;
}

int tfla_diag_bwd(const tfla_diag_args* args, void* workspace, size_t workspace_bytes, void* stream)
{
    return guarded([&]() -> int { return run_diag(args, true, workspace, workspace_bytes, stream); });
}

int tfla_addnorm_fwd(const tfla_addnorm_args* args, void* stream)
{
    return guarded([&]() -> int {
        tfla::AddNormProblem p;
        Views w;
        int rc = check_addnorm(args, false, &p, &w);
        if (rc) return rc;
        return hip_status(tfla::launch_addnorm_fwd(p, static_cast<hipStream_t>(stream)), "norm kernel launch");
    });
}

size_t tfla_addnorm_bwd_workspace_bytes(int B, int T, int C, int flags)
{
    tfla::AddNormProblem p;
    const int rc = guarded([&]() -> int { return check_addnorm_sizes(B, T, C, flags, &p); });
    return rc == TFLA_OK ? tfla::addnorm_bwd_workspace(p) : 0;
}

int tfla_addnorm_bwd(const tfla_addnorm_args* args, void* workspace, size_t workspace_bytes, void* stream)
{
    return guarded([&]() -> int {
        tfla::AddNormProblem p;
        Views w;
        int rc = check_addnorm(args, true, &p, &w);
        if (rc) return rc;
        hipStream_t s = static_cast<hipStream_t>(stream);
        // the weights' gradients alone take memory
        const size_t need = p.dweight || p.dbias ? tfla::addnorm_bwd_workspace(p) : 0;
        return with_workspace(workspace, workspace_bytes, need, w.v, w.n, s, [&](char* base) {
            p.ws = base;
            return hip_status(tfla::launch_addnorm_bwd(p, s), "norm gradient kernel launch");
        });
    });
}

}  // extern "C"
