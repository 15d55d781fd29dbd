// Argument checks shared by the C entry points (all of them run before any
// launch).
#pragma once

#include <initializer_list>

#include "common.cuh"

namespace mg {

constexpr int64_t kMaxDim = int64_t(1) << 40;

struct Buf {
    const void *p;
    size_t bytes;
    const char *name;
    bool output;
    bool optional = false;   // NULL allowed (the buffer is then not used)
    size_t align = 16;
};

// NULL, alignment and overlap checks.  Outputs may overlap nothing.
inline mg_status check_bufs(const char *fn, std::initializer_list<Buf> bufs)
{
    for (const Buf &b : bufs) {
        if (b.p == nullptr && b.optional) continue;
        if (b.p == nullptr) return fail(MG_ERR_INVALID_ARG, "%s: %s is NULL", fn, b.name);
        if (reinterpret_cast<uintptr_t>(b.p) % b.align != 0)
            return fail(MG_ERR_INVALID_ARG, "%s: %s is not %zu-byte aligned", fn, b.name, b.align);
    }
    for (const Buf &o : bufs) {
        if (!o.output || o.p == nullptr) continue;
        const uintptr_t o0 = reinterpret_cast<uintptr_t>(o.p), o1 = o0 + o.bytes;
        for (const Buf &x : bufs) {
            if (&x == &o || x.p == nullptr) continue;
            const uintptr_t x0 = reinterpret_cast<uintptr_t>(x.p), x1 = x0 + x.bytes;
            if (o0 < x1 && x0 < o1)
                return fail(MG_ERR_INVALID_ARG, "%s: output %s overlaps %s", fn, o.name, x.name);
        }
    }
    return MG_OK;
}

inline mg_status check_dims(const char *fn, std::initializer_list<int64_t> dims)
{
    int64_t prod = 1;
    for (int64_t d : dims) {
        if (d < 0) return fail(MG_ERR_INVALID_ARG, "%s: negative size %lld", fn, (long long)d);
        if (d > kMaxDim) return fail(MG_ERR_UNSUPPORTED, "%s: size %lld too large", fn, (long long)d);
        if (d > 0 && prod > (int64_t(1) << 58) / d)
            return fail(MG_ERR_UNSUPPORTED, "%s: tensor too large", fn);
        prod *= (d > 0 ? d : 1);
    }
    return MG_OK;
}

inline mg_status check_ws(const char *fn, const void *ws, size_t ws_bytes, size_t need)
{
    if (ws == nullptr) return fail(MG_ERR_INVALID_ARG, "%s: workspace is NULL", fn);
    if (reinterpret_cast<uintptr_t>(ws) % 256 != 0)
        return fail(MG_ERR_INVALID_ARG, "%s: workspace is not 256-byte aligned", fn);
    if (ws_bytes < need)
        return fail(MG_ERR_INVALID_ARG, "%s: workspace of %zu bytes, %zu needed", fn, ws_bytes, need);
    return MG_OK;
}

#define MG_TRY(...)                           \
    do {                                      \
        const mg_status st__ = (__VA_ARGS__); \
        if (st__ != MG_OK) return st__;       \
    } while (0)

}  // namespace mg
