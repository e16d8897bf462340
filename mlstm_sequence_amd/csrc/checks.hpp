// checks.hpp -- argument checks and workspaces shared by the C entry points of
// the operators around the recurrences (host only).
#pragma once

#include "tfla.h"

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>
#include <initializer_list>
#include <string>

#include "blocks.hpp"

namespace tfla {
namespace checks {

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
inline int64_t span(const View& v)
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

inline View flat(const char* name, const void* p, int64_t bytes)
{
    View v;
    v.name = name;
    v.base = reinterpret_cast<uintptr_t>(p);
    v.width = p ? bytes : 0;
    return v;
}

inline View rows(const char* name, const tfla_rows& r, int B, int T, int64_t width, int64_t esz)
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
inline bool distinct(const View& v)
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
inline int64_t extent_in(const View& v, int64_t p)
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
inline bool overlap(const View& a, const View& b)
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

inline int check_range(const View& v)
{
    if (span(v) < 0)
        return fail(TFLA_ERR_INVALID_ARG, std::string(v.name) + ": strides are negative or out of range");
    return TFLA_OK;
}

// The same elements in the same places.
inline bool same_view(const View& a, const View& b)
{
    if (a.base != b.base || a.width != b.width) return false;
    for (int i = 0; i < 3; ++i)
        if (a.n[i] != b.n[i] || (a.n[i] > 1 && a.stride[i] != b.stride[i])) return false;
    return true;
}

// Ranges of all views, distinct outputs, outputs apart from inputs and from
// each other.  twin[i] (NULL: none) is the input that output i may be exactly,
// updated in place, or -1.
inline int check_views(const View* ins, size_t ni, const View* outs, size_t no, const int* twin = nullptr)
{
    int rc;
    for (size_t i = 0; i < ni; ++i)
        if ((rc = check_range(ins[i]))) return rc;
    for (size_t i = 0; i < no; ++i) {
        if ((rc = check_range(outs[i]))) return rc;
        if (outs[i].width && !distinct(outs[i]))
            return fail(TFLA_ERR_INVALID_ARG, std::string(outs[i].name) + ": rows of an output overlap each other");
        for (size_t j = 0; j < ni; ++j) {
            if (twin && twin[i] == (int)j && same_view(outs[i], ins[j])) continue;
            if (overlap(outs[i], ins[j]))
                return fail(TFLA_ERR_INVALID_ARG, std::string(outs[i].name) + " overlaps " + ins[j].name);
        }
        for (size_t j = 0; j < i; ++j)
            if (overlap(outs[i], outs[j]))
                return fail(TFLA_ERR_INVALID_ARG, std::string(outs[i].name) + " overlaps " + outs[j].name);
    }
    return TFLA_OK;
}

inline int check_aligned(const char* name, const void* p, size_t n, bool required)
{
    if (!p) return required ? fail(TFLA_ERR_INVALID_ARG, std::string(name) + " must not be NULL") : TFLA_OK;
    if (reinterpret_cast<uintptr_t>(p) % n)
        return fail(TFLA_ERR_INVALID_ARG, std::string(name) + " is not " + std::to_string(n) + "-byte aligned");
    return TFLA_OK;
}

inline int check_flags(int flags)
{
    if (flags & ~TFLA_IO_BF16) return fail(TFLA_ERR_INVALID_ARG, "unknown flags " + std::to_string(flags));
    return TFLA_OK;
}

inline int hip_status(hipError_t e, const char* what)
{
    return e == hipSuccess ? TFLA_OK : fail(TFLA_ERR_HIP, std::string(what) + ": " + hipGetErrorString(e));
}

inline Rows dev(const tfla_rows& r)
{
    Rows o;
    o.p = r.data;
    o.batch = r.batch;
    o.row = r.row;
    return o;
}

inline View heads(const char* name, const tfla_heads& r, int B, int T, int G, int64_t width, int64_t esz)
{
    View v = rows(name, tfla_rows{r.data, r.batch, r.row}, B, T, width, esz);
    if (!r.data) return v;
    v.n[2] = G;
    v.stride[2] = r.group > kMaxSpan / esz ? kMaxSpan + 1 : r.group * esz;
    return v;
}

inline Heads dev(const tfla_heads& r)
{
    Heads o;
    o.p = r.data;
    o.batch = r.batch;
    o.row = r.row;
    o.group = r.group;
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
    if (inject_alloc_fault())
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

}  // namespace checks
}  // namespace tfla
