// blocks_api.cpp -- C entry points of the operators around the recurrences
// (include/tfla.h): argument checks (no HIP call before they pass), workspace
// and launches.  No exception leaves an entry point.
#include "tfla.h"

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>
#include <initializer_list>
#include <string>

#include "blocks.hpp"

namespace {

using tfla::fail;

// ---- memory an argument touches -----------------------------------------------------
//
// A view: up to three strided dimensions over runs of `width` contiguous
// bytes.  Offsets are kept below 2^47 bytes, so sums of them cannot overflow.
struct View {
    uintptr_t base = 0;
    int64_t width = 0;              // bytes
    int64_t n[3] = {1, 1, 1};
    int64_t stride[3] = {0, 0, 0};  // bytes
    const char* name = "";
};

constexpr int64_t kMaxSpan = int64_t(1) << 47;

// Bytes from the first to behind the last element; -1: out of range.
int64_t span(const View& v)
{
    int64_t s = v.width;
    for (int i = 0; i < 3; ++i) {
        if (v.n[i] <= 1) continue;
        int64_t x;
        if (v.stride[i] < 0 || __builtin_mul_overflow(v.n[i] - 1, v.stride[i], &x) || x > kMaxSpan) return -1;
        s += x;
    }
    return s > kMaxSpan ? -1 : s;
}

View flat(const char* name, const void* p, int64_t bytes)
{
    View v;
    v.name = name;
    v.base = reinterpret_cast<uintptr_t>(p);
    v.width = p ? bytes : 0;
    return v;
}

View rows(const char* name, const tfla_rows& r, int B, int T, int64_t width, int64_t esz)
{
    View v = flat(name, r.data, width * esz);
    if (!r.data) return v;
    v.n[0] = B;
    v.n[1] = T;
    // a stride beyond any address space is kept out of range, not wrapped
    const int64_t lim = kMaxSpan;
    v.stride[0] = r.batch > lim / esz ? lim + 1 : r.batch * esz;
    v.stride[1] = r.row > lim / esz ? lim + 1 : r.row * esz;
    return v;
}

// An output's elements are distinct: each stride reaches over everything the
// smaller ones span.
bool distinct(const View& v)
{
    int o[3] = {0, 1, 2};
    std::sort(o, o + 3, [&](int a, int b) { return v.stride[a] < v.stride[b]; });
    int64_t ext = v.width;
    for (int i : o) {
        if (v.n[i] <= 1) continue;
        if (v.stride[i] < ext) return false;
        ext = (v.n[i] - 1) * v.stride[i] + ext;
    }
    return true;
}

// The part of v inside one period `p`: the extent of its dimensions with
// smaller strides; -1 when a larger stride is no multiple of p.
int64_t extent_in(const View& v, int64_t p)
{
    int64_t e = v.width;
    for (int i = 0; i < 3; ++i) {
        if (v.n[i] <= 1) continue;
        if (v.stride[i] < p) e += (v.n[i] - 1) * v.stride[i];
        else if (v.stride[i] % p) return -1;
    }
    return e;
}

// Whether two views share a byte: their spans are disjoint, or some stride is
// a period in which they occupy disjoint columns (the halves of a row, the
// heads of a token); otherwise they are taken to overlap.
bool overlap(const View& a, const View& b)
{
    if (!a.width || !b.width) return false;
    const uintptr_t ea = a.base + span(a), eb = b.base + span(b);
    if (ea <= b.base || eb <= a.base) return false;
    for (const View* v : {&a, &b})
        for (int i = 0; i < 3; ++i) {
            const int64_t p = v->stride[i];
            if (v->n[i] <= 1 || p <= 0) continue;
            const int64_t xa = extent_in(a, p), xb = extent_in(b, p);
            if (xa < 0 || xb < 0 || xa > p || xb > p) continue;
            // columns of b relative to a's first, around the period
            const int64_t off = b.base >= a.base ? (int64_t)((b.base - a.base) % (uintptr_t)p)
                                                 : (p - (int64_t)((a.base - b.base) % (uintptr_t)p)) % p;
            if (off >= xa && off + xb <= p) return false;
        }
    return true;
}

int check_range(const View& v)
{
    if (span(v) < 0)
        return fail(TFLA_ERR_INVALID_ARG, std::string(v.name) + ": strides are negative or out of range");
    return TFLA_OK;
}

// Ranges of all views, distinct outputs, outputs apart from inputs and from
// each other.  An output that may be exactly one of the inputs is left out
// by its caller (same base) from `outs` against that input via `in_place`.
int check_views(const View* ins, size_t ni, const View* outs, size_t no, const void* in_place = nullptr)
{
    int rc;
    for (size_t i = 0; i < ni; ++i)
        if ((rc = check_range(ins[i]))) return rc;
    for (size_t i = 0; i < no; ++i) {
        if ((rc = check_range(outs[i]))) return rc;
        if (outs[i].width && !distinct(outs[i]))
            return fail(TFLA_ERR_INVALID_ARG, std::string(outs[i].name) + ": rows of an output overlap each other");
        for (size_t j = 0; j < ni; ++j) {
            if (in_place && outs[i].base == (uintptr_t)in_place && ins[j].base == (uintptr_t)in_place &&
                outs[i].width == ins[j].width)
                continue;
            if (overlap(outs[i], ins[j]))
                return fail(TFLA_ERR_INVALID_ARG, std::string(outs[i].name) + " overlaps " + ins[j].name);
        }
        for (size_t j = 0; j < i; ++j)
            if (overlap(outs[i], outs[j]))
                return fail(TFLA_ERR_INVALID_ARG, std::string(outs[i].name) + " overlaps " + outs[j].name);
    }
    return TFLA_OK;
}

int check_aligned(const char* name, const void* p, size_t n, bool required)
{
    if (!p) return required ? fail(TFLA_ERR_INVALID_ARG, std::string(name) + " must not be NULL") : TFLA_OK;
    if (reinterpret_cast<uintptr_t>(p) % n)
        return fail(TFLA_ERR_INVALID_ARG, std::string(name) + " is not " + std::to_string(n) + "-byte aligned");
    return TFLA_OK;
}

int check_flags(int flags)
{
    if (flags & ~TFLA_IO_BF16) return fail(TFLA_ERR_INVALID_ARG, "unknown flags " + std::to_string(flags));
    return TFLA_OK;
}

int hip_status(hipError_t e, const char* what)
{
    return e == hipSuccess ? TFLA_OK : fail(TFLA_ERR_HIP, std::string(what) + ": " + hipGetErrorString(e));
}

tfla::Rows dev(const tfla_rows& r)
{
    tfla::Rows o;
    o.p = r.data;
    o.batch = r.batch;
    o.row = r.row;
    return o;
}

// Runs `launch(base)` with a workspace of `need` bytes: the caller's, checked
// against the views, or one allocated and freed on the stream.
template <typename F>
int with_workspace(void* workspace, size_t bytes, size_t need, const View* views, size_t nv, hipStream_t s, F launch)
{
    if (need == 0) return launch(nullptr);
    if (workspace) {
        if (reinterpret_cast<uintptr_t>(workspace) % 256)
            return fail(TFLA_ERR_INVALID_ARG, "workspace is not 256-byte aligned");
        if (bytes < need)
            return fail(TFLA_ERR_OUT_OF_MEMORY, "workspace of " + std::to_string(bytes) +
                                                    " bytes is smaller than the " + std::to_string(need) + " needed");
        const View w = flat("workspace", workspace, (int64_t)need);
        for (size_t i = 0; i < nv; ++i)
            if (overlap(w, views[i]))
                return fail(TFLA_ERR_INVALID_ARG, std::string("workspace overlaps ") + views[i].name);
        return launch(static_cast<char*>(workspace));
    }
    if (tfla::inject_alloc_fault())
        return fail(TFLA_ERR_OUT_OF_MEMORY, "injected allocation failure (fault knob)");
    void* base = nullptr;
    hipError_t e = hipMallocAsync(&base, need, s);
    if (e != hipSuccess) {
        (void)hipGetLastError();
        return fail(TFLA_ERR_OUT_OF_MEMORY, std::string("workspace allocation of ") + std::to_string(need) +
                                                " bytes failed: " + hipGetErrorString(e));
    }
    int rc = launch(static_cast<char*>(base));
    e = hipFreeAsync(base, s);
    if (e != hipSuccess && rc == TFLA_OK) rc = hip_status(e, "workspace free");
    return rc;
}

// Exceptions (a message that cannot be allocated) end as a status here.
template <typename F>
int guarded(F f) noexcept
{
    try {
        return f();
    } catch (...) {
        return TFLA_ERR_OUT_OF_MEMORY;
    }
}

constexpr int64_t kMaxRows = int64_t(1) << 30;

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
    if ((rc = check_views(views, n, views + n, no, !bwd && state == state_out ? state : nullptr))) return rc;
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
    if ((rc = check_views(views, ni, views + ni, n - ni, !bwd && a->state == a->state_out ? a->state : nullptr))) return rc;
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

View heads(const char* name, const tfla_heads& r, const tfla_norm_args& a, int64_t esz)
{
    View v = rows(name, tfla_rows{r.data, r.batch, r.row}, a.B, a.T, a.C, esz);
    if (!r.data) return v;
    v.n[2] = a.G;
    v.stride[2] = r.group > kMaxSpan / esz ? kMaxSpan + 1 : r.group * esz;
    return v;
}

tfla::Heads dev(const tfla_heads& r)
{
    tfla::Heads o;
    o.p = r.data;
    o.batch = r.batch;
    o.row = r.row;
    o.group = r.group;
    return o;
}

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
        views[n++] = heads(name, r, *a, e);
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
