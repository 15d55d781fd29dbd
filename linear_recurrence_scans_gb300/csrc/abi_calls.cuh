// Argument checks that the C entry points of mg_ssm.h and mg_block.h share.
#pragma once

#include <cstring>
#include <type_traits>
#include <utility>

#include "ssm.cuh"

namespace mg {

inline mg_status begin_call() { return fail(MG_OK, "%s", ""); }

inline size_t esize(mg_dtype dt) { return dt == MG_F32 ? 4 : 2; }

inline mg_status check_type(const char *fn, mg_dtype dt)
{
    if (dt != MG_F32 && dt != MG_BF16)
        return fail(MG_ERR_UNSUPPORTED, "%s: activation dtype %d not supported", fn, int(dt));
    return MG_OK;
}

// An input of `rows` rows of `width` values with row stride ld.
inline mg_status check_ld(const char *fn, const char *name, int64_t ld, int64_t width)
{
    if (ld < width)
        return fail(MG_ERR_INVALID_ARG, "%s: row stride %lld of %s is below its width %lld", fn,
                    (long long)ld, name, (long long)width);
    if (ld > kMaxDim) return fail(MG_ERR_UNSUPPORTED, "%s: row stride of %s too large", fn, name);
    return MG_OK;
}

inline size_t extent(int64_t rows, int64_t ld, int64_t width, size_t es)
{
    return rows > 0 ? (size_t(rows - 1) * ld + width) * es : 0;
}

// cu_seqlens and nseq against B and T.
inline mg_status check_seqs(const char *fn, const int64_t *cu, int64_t nseq, int64_t B)
{
    if (nseq < 0) return fail(MG_ERR_INVALID_ARG, "%s: negative nseq", fn);
    if (nseq > (int64_t(1) << 31) - 2) return fail(MG_ERR_UNSUPPORTED, "%s: nseq too large", fn);
    if (cu == nullptr) {
        if (nseq != B)
            return fail(MG_ERR_INVALID_ARG, "%s: nseq must be B without cu_seqlens", fn);
        return MG_OK;
    }
    if (B != 1) return fail(MG_ERR_INVALID_ARG, "%s: B must be 1 with cu_seqlens", fn);
    if (nseq == 0) return fail(MG_ERR_INVALID_ARG, "%s: cu_seqlens without sequences", fn);
    if (reinterpret_cast<uintptr_t>(cu) % 8 != 0)
        return fail(MG_ERR_INVALID_ARG, "%s: cu_seqlens is not 8-byte aligned", fn);
    return MG_OK;
}

inline mg_status check_slots(const char *fn, const int64_t *slots, int64_t nslots, int64_t B)
{
    if (nslots < 0) return fail(MG_ERR_INVALID_ARG, "%s: negative nslots", fn);
    if (slots == nullptr && nslots < B)
        return fail(MG_ERR_INVALID_ARG, "%s: %lld states for %lld rows without slots", fn,
                    (long long)nslots, (long long)B);
    return MG_OK;
}

// The grids' block counts are 32-bit; so many values at most in one call
// (rows x channels, and channels x states of a token call).
inline mg_status check_size(const char *fn, int64_t a, int64_t b)
{
    if (b > 0 && a > (int64_t(1) << 36) / b)
        return fail(MG_ERR_UNSUPPORTED, "%s: more than 2^36 values", fn);
    return MG_OK;
}

// dst = src, or zero without src: what a call without rows does to a state.
inline mg_status pass_state(const char *fn, void *dst, const void *src, size_t bytes, cudaStream_t s)
{
    if (dst == nullptr || bytes == 0) return MG_OK;
    MG_TRY(check_bufs(fn, {{dst, bytes, "state output", true}, {src, bytes, "state input", false, true}}));
    const cudaError_t e = src != nullptr
                              ? cudaMemcpyAsync(dst, src, bytes, cudaMemcpyDeviceToDevice, s)
                              : cudaMemsetAsync(dst, 0, bytes, s);
    return e == cudaSuccess ? MG_OK : fail(MG_ERR_LAUNCH, "%s: %s", fn, cudaGetErrorString(e));
}

inline mg_status zero(const char *fn, float *p, int64_t n, const char *name, cudaStream_t s)
{
    if (p == nullptr || n == 0) return MG_OK;
    MG_TRY(check_bufs(fn, {{p, size_t(n) * 4, name, true}}));
    const cudaError_t e = cudaMemsetAsync(p, 0, size_t(n) * 4, s);
    return e == cudaSuccess ? MG_OK : fail(MG_ERR_LAUNCH, "%s: %s", fn, cudaGetErrorString(e));
}

// Calls f with its arguments from 64-bit words.
template <typename A>
A from_word(uint64_t w)
{
    A a{};
    if constexpr (std::is_pointer_v<A>) {
        a = reinterpret_cast<A>(static_cast<uintptr_t>(w));
    } else if constexpr (std::is_same_v<A, double>) {
        memcpy(&a, &w, sizeof(a));
    } else {
        a = static_cast<A>(static_cast<int64_t>(w));
    }
    return a;
}
template <typename... A, size_t... I>
mg_status call_words(mg_status (*f)(A...), const uint64_t *w, std::index_sequence<I...>)
{
    return f(from_word<A>(w[I])...);
}
template <typename... A>
mg_status call_words(mg_status (*f)(A...), const uint64_t *w, int n)
{
    if (n != int(sizeof...(A)))
        return fail(MG_ERR_INVALID_ARG, "%d arguments, %d expected", n, int(sizeof...(A)));
    return call_words(f, w, std::index_sequence_for<A...>());
}

}  // namespace mg
