// The C entry points of mg_ssm.h: argument validation (all of it before any
// launch) and the calls without rows.
#include <cstring>
#include <type_traits>
#include <utility>

#include "ssm.cuh"

using namespace mg;

namespace {

mg_status begin_call() { return fail(MG_OK, "%s", ""); }

size_t esize(mg_dtype dt) { return dt == MG_F32 ? 4 : 2; }

mg_status check_type(const char *fn, mg_dtype dt)
{
    if (dt != MG_F32 && dt != MG_BF16)
        return fail(MG_ERR_UNSUPPORTED, "%s: activation dtype %d not supported", fn, int(dt));
    return MG_OK;
}

// An input of `rows` rows of `width` values with row stride ld.
mg_status check_ld(const char *fn, const char *name, int64_t ld, int64_t width)
{
    if (ld < width)
        return fail(MG_ERR_INVALID_ARG, "%s: row stride %lld of %s is below its width %lld", fn,
                    (long long)ld, name, (long long)width);
    if (ld > kMaxDim) return fail(MG_ERR_UNSUPPORTED, "%s: row stride of %s too large", fn, name);
    return MG_OK;
}

size_t extent(int64_t rows, int64_t ld, int64_t width, size_t es)
{
    return rows > 0 ? (size_t(rows - 1) * ld + width) * es : 0;
}

// cu_seqlens and nseq against B and T.
mg_status check_seqs(const char *fn, const int64_t *cu, int64_t nseq, int64_t B)
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

mg_status check_slots(const char *fn, const int64_t *slots, int64_t nslots, int64_t B)
{
    if (nslots < 0) return fail(MG_ERR_INVALID_ARG, "%s: negative nslots", fn);
    if (slots == nullptr && nslots < B)
        return fail(MG_ERR_INVALID_ARG, "%s: %lld states for %lld rows without slots", fn,
                    (long long)nslots, (long long)B);
    return MG_OK;
}

// The grids' block counts are 32-bit; so many values at most in one call
// (rows x channels, and channels x states of a token call).
mg_status check_size(const char *fn, int64_t a, int64_t b)
{
    if (b > 0 && a > (int64_t(1) << 36) / b)
        return fail(MG_ERR_UNSUPPORTED, "%s: more than 2^36 values", fn);
    return MG_OK;
}

// dst = src, or zero without src: what a call without rows does to a state.
mg_status pass_state(const char *fn, void *dst, const void *src, size_t bytes, cudaStream_t s)
{
    if (dst == nullptr || bytes == 0) return MG_OK;
    MG_TRY(check_bufs(fn, {{dst, bytes, "state output", true}, {src, bytes, "state input", false, true}}));
    const cudaError_t e = src != nullptr
                              ? cudaMemcpyAsync(dst, src, bytes, cudaMemcpyDeviceToDevice, s)
                              : cudaMemsetAsync(dst, 0, bytes, s);
    return e == cudaSuccess ? MG_OK : fail(MG_ERR_LAUNCH, "%s: %s", fn, cudaGetErrorString(e));
}

mg_status zero(const char *fn, float *p, int64_t n, const char *name, cudaStream_t s)
{
    if (p == nullptr || n == 0) return MG_OK;
    MG_TRY(check_bufs(fn, {{p, size_t(n) * 4, name, true}}));
    const cudaError_t e = cudaMemsetAsync(p, 0, size_t(n) * 4, s);
    return e == cudaSuccess ? MG_OK : fail(MG_ERR_LAUNCH, "%s: %s", fn, cudaGetErrorString(e));
}

mg_status check_conv(const char *fn, int64_t B, int64_t T, int64_t D, int W)
{
    MG_TRY(check_dims(fn, {B, T, D}));
    if (W < 1 || W > 8) return fail(MG_ERR_UNSUPPORTED, "%s: W = %d outside [1, 8]", fn, W);
    MG_TRY(check_size(fn, B * T, D));
    return check_size(fn, B, D * W);
}

mg_status check_ssm(const char *fn, int64_t B, int64_t T, int64_t D, int64_t N, int64_t G)
{
    MG_TRY(check_dims(fn, {B, T, D}));
    if (N < 1 || N > kSsmMaxN)
        return fail(MG_ERR_UNSUPPORTED, "%s: N = %lld outside [1, %d]", fn, (long long)N, kSsmMaxN);
    if (G < 1 || D % G != 0)
        return fail(MG_ERR_INVALID_ARG, "%s: D = %lld is not a multiple of G = %lld", fn,
                    (long long)D, (long long)G);
    if (G > (int64_t(1) << 24)) return fail(MG_ERR_UNSUPPORTED, "%s: G too large", fn);
    MG_TRY(check_size(fn, B * T, D));
    return check_size(fn, B, D * N);
}

mg_status check_norm(const char *fn, int64_t M, int64_t D, int64_t G, mg_gate gate)
{
    MG_TRY(check_dims(fn, {M, D}));
    if (G < 1 || D % G != 0)
        return fail(MG_ERR_INVALID_ARG, "%s: D = %lld is not a multiple of G = %lld", fn,
                    (long long)D, (long long)G);
    if (gate != MG_GATE_NONE && gate != MG_GATE_AFTER && gate != MG_GATE_FIRST)
        return fail(MG_ERR_INVALID_ARG, "%s: gate %d", fn, int(gate));
    if (D / G > 16384)
        return fail(MG_ERR_UNSUPPORTED, "%s: groups of %lld channels, at most 16384", fn,
                    (long long)(D / G));
    MG_TRY(check_size(fn, M, D));
    // the kernels count rows in 32 bits
    if (M > INT32_MAX / G) return fail(MG_ERR_UNSUPPORTED, "%s: M G beyond 2^31 - 1", fn);
    return MG_OK;
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
        return fail(MG_ERR_INVALID_ARG, "mg_ssm_call: %d arguments, %d expected", n, int(sizeof...(A)));
    return call_words(f, w, std::index_sequence_for<A...>());
}

}  // namespace

extern "C" {

size_t mg_causal_conv_workspace_size(int64_t B, int64_t T, int64_t D, int W)
{
    if (check_conv("mg_causal_conv_workspace_size", B, T, D, W) != MG_OK) return 0;
    if (B == 0 || T == 0 || D == 0) return kControlBytes;
    return conv_ws_bytes(B, T, D, W);
}

mg_status mg_causal_conv_fwd(const void *x, int64_t ldx, mg_dtype dt, const float *w,
                             const float *bias, const void *x0, const int64_t *cu_seqlens,
                             int64_t nseq, int silu, void *y, void *x_last, int64_t B, int64_t T,
                             int64_t D, int W, void *ws, size_t ws_bytes, cudaStream_t stream)
{
    const char *fn = "mg_causal_conv_fwd";
    begin_call();
    MG_TRY(check_type(fn, dt));
    MG_TRY(check_conv(fn, B, T, D, W));
    MG_TRY(check_seqs(fn, cu_seqlens, nseq, B));
    MG_TRY(check_ld(fn, "x", ldx, D));
    MG_TRY(check_size(fn, nseq, D * W));
    const size_t es = esize(dt), edge = size_t(nseq) * (W - 1) * D * es, rows = size_t(B) * T;
    if (D == 0) return MG_OK;
    if (rows == 0) return pass_state(fn, x_last, x0, edge, stream);
    MG_TRY(check_ws(fn, ws, ws_bytes, kControlBytes));
    MG_TRY(check_bufs(fn, {{x, extent(rows, ldx, D, es), "x", false},
                           {w, size_t(D) * W * 4, "w", false},
                           {bias, size_t(D) * 4, "bias", false, true},
                           {x0, edge, "x0", false, true},
                           {y, rows * D * es, "y", true},
                           {x_last, edge, "x_last", true, true},
                           {ws, ws_bytes, "workspace", true}}));
    ConvArgs p{};
    p.x = x, p.ldx = ldx, p.w = w, p.bias = bias, p.x0 = x0, p.cu = cu_seqlens, p.nseq = nseq;
    p.silu = silu, p.y = y, p.x_last = x_last, p.B = B, p.T = T, p.D = D, p.W = W, p.ws = ws;
    return launch_conv_fwd(p, dt, stream);
}

mg_status mg_causal_conv_bwd(const void *dy, int64_t lddy, const void *x, int64_t ldx, mg_dtype dt,
                             const float *w, const float *bias, const void *x0,
                             const void *dx_last, const int64_t *cu_seqlens, int64_t nseq,
                             int silu, void *dx, float *dw, float *dbias, void *dx0, int64_t B,
                             int64_t T, int64_t D, int W, void *ws, size_t ws_bytes,
                             cudaStream_t stream)
{
    const char *fn = "mg_causal_conv_bwd";
    begin_call();
    MG_TRY(check_type(fn, dt));
    MG_TRY(check_conv(fn, B, T, D, W));
    MG_TRY(check_seqs(fn, cu_seqlens, nseq, B));
    MG_TRY(check_ld(fn, "x", ldx, D));
    MG_TRY(check_ld(fn, "dy", lddy, D));
    MG_TRY(check_size(fn, nseq, D * W));
    const size_t es = esize(dt), edge = size_t(nseq) * (W - 1) * D * es, rows = size_t(B) * T;
    if (D == 0) return MG_OK;
    if (rows == 0) {
        MG_TRY(zero(fn, dw, D * W, "dw", stream));
        MG_TRY(zero(fn, dbias, D, "dbias", stream));
        return pass_state(fn, dx0, dx_last, edge, stream);
    }
    MG_TRY(check_ws(fn, ws, ws_bytes, conv_ws_bytes(B, T, D, W)));
    MG_TRY(check_bufs(fn, {{dy, extent(rows, lddy, D, es), "dy", false},
                           {x, extent(rows, ldx, D, es), "x", false},
                           {w, size_t(D) * W * 4, "w", false},
                           {bias, size_t(D) * 4, "bias", false, true},
                           {x0, edge, "x0", false, true},
                           {dx_last, edge, "dx_last", false, true},
                           {dx, rows * D * es, "dx", true},
                           {dw, size_t(D) * W * 4, "dw", true},
                           {dbias, size_t(D) * 4, "dbias", true, true},
                           {dx0, edge, "dx0", true, true},
                           {ws, ws_bytes, "workspace", true}}));
    ConvArgs p{};
    p.dy = dy, p.lddy = lddy, p.x = x, p.ldx = ldx, p.w = w, p.bias = bias, p.x0 = x0;
    p.dx_last = dx_last, p.cu = cu_seqlens, p.nseq = nseq, p.silu = silu, p.dx = dx, p.dw = dw;
    p.dbias = dbias, p.dx0 = dx0, p.B = B, p.T = T, p.D = D, p.W = W, p.ws = ws;
    return launch_conv_bwd(p, dt, stream);
}

mg_status mg_causal_conv_step(const void *x, int64_t ldx, mg_dtype dt, const float *w,
                              const float *bias, void *state, int64_t nslots,
                              const int64_t *slots, int silu, void *y, int64_t B, int64_t D, int W,
                              cudaStream_t stream)
{
    const char *fn = "mg_causal_conv_step";
    begin_call();
    MG_TRY(check_type(fn, dt));
    MG_TRY(check_conv(fn, B, 1, D, W));
    MG_TRY(check_slots(fn, slots, nslots, B));
    MG_TRY(check_ld(fn, "x", ldx, D));
    MG_TRY(check_dims(fn, {nslots, D, W}));
    if (B == 0 || D == 0) return MG_OK;
    const size_t es = esize(dt), pool = size_t(nslots) * (W - 1) * D * es;
    MG_TRY(check_bufs(fn, {{x, extent(B, ldx, D, es), "x", false},
                           {w, size_t(D) * W * 4, "w", false},
                           {bias, size_t(D) * 4, "bias", false, true},
                           {slots, size_t(B) * 8, "slots", false, true, 8},
                           {state, pool, "state", true, pool == 0},
                           {y, size_t(B) * D * es, "y", true}}));
    ConvStepArgs p{};
    p.x = x, p.ldx = ldx, p.w = w, p.bias = bias, p.state = state, p.nslots = nslots;
    p.slots = slots, p.silu = silu, p.y = y, p.B = B, p.D = D, p.W = W;
    return launch_conv_step(p, dt, stream);
}

size_t mg_selective_scan_fwd_workspace_size(int64_t B, int64_t T, int64_t D, int64_t N, int64_t G,
                                            int64_t nseq)
{
    if (check_ssm("mg_selective_scan_fwd_workspace_size", B, T, D, N, G) != MG_OK || nseq < 0)
        return 0;
    if (B == 0 || T == 0 || D == 0) return kControlBytes;
    return ssm_fwd_ws_bytes(B, T, D, int(N), int(G), nseq);
}

size_t mg_selective_scan_bwd_workspace_size(int64_t B, int64_t T, int64_t D, int64_t N, int64_t G,
                                            int64_t nseq)
{
    if (check_ssm("mg_selective_scan_bwd_workspace_size", B, T, D, N, G) != MG_OK || nseq < 0)
        return 0;
    if (B == 0 || T == 0 || D == 0) return kControlBytes;
    return ssm_bwd_ws_bytes(B, T, D, int(N), int(G), nseq);
}

size_t mg_selective_scan_saved_size(int64_t B, int64_t T, int64_t D, int64_t N)
{
    if (check_ssm("mg_selective_scan_saved_size", B, T, D, N, 1) != MG_OK) return 0;
    return ssm_saved_bytes(B, T, D, int(N));
}

int mg_selective_scan_saved_rows(void) { return ssm_saved_rows(); }

mg_status mg_selective_scan_fwd(const void *x, int64_t ldx, const void *raw, int64_t ldraw,
                                const float *A, const void *Bm, int64_t ldb, const void *Cm,
                                int64_t ldc, mg_dtype dt, const float *Dskip,
                                const float *dt_bias, int softplus, const float *h0,
                                const int64_t *cu_seqlens, int64_t nseq, void *y, float *h_last,
                                float *saved, int64_t B, int64_t T, int64_t D, int64_t N,
                                int64_t G, void *ws, size_t ws_bytes, cudaStream_t stream)
{
    const char *fn = "mg_selective_scan_fwd";
    begin_call();
    MG_TRY(check_type(fn, dt));
    MG_TRY(check_ssm(fn, B, T, D, N, G));
    MG_TRY(check_seqs(fn, cu_seqlens, nseq, B));
    MG_TRY(check_ld(fn, "x", ldx, D));
    MG_TRY(check_ld(fn, "raw", ldraw, D));
    MG_TRY(check_ld(fn, "Bm", ldb, G * N));
    MG_TRY(check_ld(fn, "Cm", ldc, G * N));
    MG_TRY(check_size(fn, nseq, D * N));
    const size_t es = esize(dt), st = size_t(nseq) * D * N * 4, rows = size_t(B) * T;
    if (D == 0) return MG_OK;
    if (rows == 0) return pass_state(fn, h_last, h0, st, stream);
    MG_TRY(check_ws(fn, ws, ws_bytes, ssm_fwd_ws_bytes(B, T, D, int(N), int(G), nseq)));
    MG_TRY(check_bufs(fn, {{x, extent(rows, ldx, D, es), "x", false},
                           {raw, extent(rows, ldraw, D, es), "raw", false},
                           {A, size_t(D) * N * 4, "A", false},
                           {Bm, extent(rows, ldb, G * N, es), "Bm", false},
                           {Cm, extent(rows, ldc, G * N, es), "Cm", false},
                           {Dskip, size_t(D) * 4, "Dskip", false, true},
                           {dt_bias, size_t(D) * 4, "dt_bias", false, true},
                           {h0, st, "h0", false, true},
                           {y, rows * D * es, "y", true},
                           {h_last, st, "h_last", true, true},
                           {saved, ssm_saved_bytes(B, T, D, int(N)), "saved", true, true},
                           {ws, ws_bytes, "workspace", true}}));
    SsmArgs p{};
    p.x = x, p.ldx = ldx, p.raw = raw, p.ldraw = ldraw, p.A = A, p.Bm = Bm, p.ldb = ldb;
    p.Cm = Cm, p.ldc = ldc, p.Dskip = Dskip, p.dt_bias = dt_bias, p.softplus = softplus;
    p.h0 = h0, p.cu = cu_seqlens, p.nseq = nseq, p.y = y, p.h_last = h_last, p.saved = saved;
    p.B = B, p.T = T, p.D = D, p.N = int(N), p.G = int(G), p.ws = ws;
    return launch_ssm_fwd(p, dt, stream);
}

mg_status mg_selective_scan_bwd(const void *dy, int64_t lddy, const float *saved, const void *x,
                                int64_t ldx, const void *raw, int64_t ldraw, const float *A,
                                const void *Bm, int64_t ldb, const void *Cm, int64_t ldc,
                                mg_dtype dt, const float *Dskip, const float *dt_bias,
                                int softplus, const float *h0, const float *dh_last,
                                const int64_t *cu_seqlens, int64_t nseq, void *dx, void *draw,
                                float *dA, void *dBm, void *dCm, float *dDskip, float *ddt_bias,
                                float *dh0, int64_t B, int64_t T, int64_t D, int64_t N, int64_t G,
                                void *ws, size_t ws_bytes, cudaStream_t stream)
{
    const char *fn = "mg_selective_scan_bwd";
    begin_call();
    MG_TRY(check_type(fn, dt));
    MG_TRY(check_ssm(fn, B, T, D, N, G));
    MG_TRY(check_seqs(fn, cu_seqlens, nseq, B));
    MG_TRY(check_ld(fn, "dy", lddy, D));
    MG_TRY(check_ld(fn, "x", ldx, D));
    MG_TRY(check_ld(fn, "raw", ldraw, D));
    MG_TRY(check_ld(fn, "Bm", ldb, G * N));
    MG_TRY(check_ld(fn, "Cm", ldc, G * N));
    MG_TRY(check_size(fn, nseq, D * N));
    const size_t es = esize(dt), st = size_t(nseq) * D * N * 4, rows = size_t(B) * T;
    if (D == 0) {
        // no channel sends anything to B and C
        const size_t n = rows * G * N * es;
        for (void *o : {dBm, dCm})
            if (n > 0) MG_TRY(pass_state(fn, o, nullptr, n, stream));
        return MG_OK;
    }
    if (rows == 0) {
        MG_TRY(zero(fn, dA, D * N, "dA", stream));
        MG_TRY(zero(fn, dDskip, D, "dDskip", stream));
        MG_TRY(zero(fn, ddt_bias, D, "ddt_bias", stream));
        return pass_state(fn, dh0, dh_last, st, stream);
    }
    MG_TRY(check_ws(fn, ws, ws_bytes, ssm_bwd_ws_bytes(B, T, D, int(N), int(G), nseq)));
    MG_TRY(check_bufs(fn, {{dy, extent(rows, lddy, D, es), "dy", false},
                           {saved, ssm_saved_bytes(B, T, D, int(N)), "saved", false},
                           {x, extent(rows, ldx, D, es), "x", false},
                           {raw, extent(rows, ldraw, D, es), "raw", false},
                           {A, size_t(D) * N * 4, "A", false},
                           {Bm, extent(rows, ldb, G * N, es), "Bm", false},
                           {Cm, extent(rows, ldc, G * N, es), "Cm", false},
                           {Dskip, size_t(D) * 4, "Dskip", false, true},
                           {dt_bias, size_t(D) * 4, "dt_bias", false, true},
                           {h0, st, "h0", false, true},
                           {dh_last, st, "dh_last", false, true},
                           {dx, rows * D * es, "dx", true},
                           {draw, rows * D * es, "draw", true},
                           {dA, size_t(D) * N * 4, "dA", true},
                           {dBm, rows * G * N * es, "dBm", true},
                           {dCm, rows * G * N * es, "dCm", true},
                           {dDskip, size_t(D) * 4, "dDskip", true, true},
                           {ddt_bias, size_t(D) * 4, "ddt_bias", true, true},
                           {dh0, st, "dh0", true, true},
                           {ws, ws_bytes, "workspace", true}}));
    SsmArgs p{};
    p.dy = dy, p.lddy = lddy, p.saved_in = saved, p.x = x, p.ldx = ldx, p.raw = raw;
    p.ldraw = ldraw, p.A = A, p.Bm = Bm, p.ldb = ldb, p.Cm = Cm, p.ldc = ldc, p.Dskip = Dskip;
    p.dt_bias = dt_bias, p.softplus = softplus, p.h0 = h0, p.dh_last = dh_last;
    p.cu = cu_seqlens, p.nseq = nseq, p.dx = dx, p.draw = draw, p.dA = dA, p.dBm = dBm;
    p.dCm = dCm, p.dDskip = dDskip, p.ddt_bias = ddt_bias, p.dh0 = dh0;
    p.B = B, p.T = T, p.D = D, p.N = int(N), p.G = int(G), p.ws = ws;
    return launch_ssm_bwd(p, dt, stream);
}

mg_status mg_selective_scan_step(const void *x, int64_t ldx, const void *raw, int64_t ldraw,
                                 const float *A, const void *Bm, int64_t ldb, const void *Cm,
                                 int64_t ldc, mg_dtype dt, const float *Dskip,
                                 const float *dt_bias, int softplus, float *state, int64_t nslots,
                                 const int64_t *slots, void *y, int64_t B, int64_t D, int64_t N,
                                 int64_t G, cudaStream_t stream)
{
    const char *fn = "mg_selective_scan_step";
    begin_call();
    MG_TRY(check_type(fn, dt));
    MG_TRY(check_ssm(fn, B, 1, D, N, G));
    MG_TRY(check_slots(fn, slots, nslots, B));
    MG_TRY(check_ld(fn, "x", ldx, D));
    MG_TRY(check_ld(fn, "raw", ldraw, D));
    MG_TRY(check_ld(fn, "Bm", ldb, G * N));
    MG_TRY(check_ld(fn, "Cm", ldc, G * N));
    MG_TRY(check_dims(fn, {nslots, D, N}));
    if (B == 0 || D == 0) return MG_OK;
    const size_t es = esize(dt), pool = size_t(nslots) * D * N * 4;
    MG_TRY(check_bufs(fn, {{x, extent(B, ldx, D, es), "x", false},
                           {raw, extent(B, ldraw, D, es), "raw", false},
                           {A, size_t(D) * N * 4, "A", false},
                           {Bm, extent(B, ldb, G * N, es), "Bm", false},
                           {Cm, extent(B, ldc, G * N, es), "Cm", false},
                           {Dskip, size_t(D) * 4, "Dskip", false, true},
                           {dt_bias, size_t(D) * 4, "dt_bias", false, true},
                           {slots, size_t(B) * 8, "slots", false, true, 8},
                           {state, pool, "state", true, pool == 0},
                           {y, size_t(B) * D * es, "y", true}}));
    SsmStepArgs p{};
    p.x = x, p.ldx = ldx, p.raw = raw, p.ldraw = ldraw, p.A = A, p.Bm = Bm, p.ldb = ldb;
    p.Cm = Cm, p.ldc = ldc, p.Dskip = Dskip, p.dt_bias = dt_bias, p.softplus = softplus;
    p.state = state, p.nslots = nslots, p.slots = slots, p.y = y, p.B = B, p.D = D;
    p.N = int(N), p.G = int(G);
    return launch_ssm_step(p, dt, stream);
}

size_t mg_group_norm_workspace_size(int64_t M, int64_t D, int64_t G)
{
    if (check_norm("mg_group_norm_workspace_size", M, D, G, MG_GATE_NONE) != MG_OK) return 0;
    if (M == 0 || D == 0) return kControlBytes;
    return norm_ws_bytes(M, D, G);
}

mg_status mg_group_norm_fwd(const void *x, int64_t ldx, const void *z, int64_t ldz, mg_dtype dt,
                            const float *w, const float *bias, double eps, int rms, mg_gate gate,
                            int silu, void *y, float *stats, int64_t M, int64_t D, int64_t G,
                            cudaStream_t stream)
{
    const char *fn = "mg_group_norm_fwd";
    begin_call();
    MG_TRY(check_type(fn, dt));
    MG_TRY(check_norm(fn, M, D, G, gate));
    MG_TRY(check_ld(fn, "x", ldx, D));
    if (gate != MG_GATE_NONE) MG_TRY(check_ld(fn, "z", ldz, D));
    if ((z == nullptr) != (gate == MG_GATE_NONE) && M > 0 && D > 0)
        return fail(MG_ERR_INVALID_ARG, "%s: z goes with a gate, and a gate with z", fn);
    if (!(eps >= 0.0)) return fail(MG_ERR_INVALID_ARG, "%s: eps must not be negative", fn);
    if (M == 0 || D == 0) return MG_OK;
    const size_t es = esize(dt);
    MG_TRY(check_bufs(fn, {{x, extent(M, ldx, D, es), "x", false},
                           {z, extent(M, ldz, D, es), "z", false, true},
                           {w, size_t(D) * 4, "w", false},
                           {bias, size_t(D) * 4, "bias", false, true},
                           {y, size_t(M) * D * es, "y", true},
                           {stats, size_t(M) * G * 8, "stats", true, true}}));
    NormArgs p{};
    p.x = x, p.ldx = ldx, p.z = z, p.ldz = ldz, p.w = w, p.bias = bias, p.eps = float(eps);
    p.rms = rms, p.gate = gate, p.silu = silu, p.y = y, p.stats = stats, p.M = M, p.D = D, p.G = G;
    return launch_norm_fwd(p, dt, stream);
}

mg_status mg_group_norm_bwd(const void *dy, int64_t lddy, const float *stats, const void *x,
                            int64_t ldx, const void *z, int64_t ldz, mg_dtype dt, const float *w,
                            const float *bias, int rms, mg_gate gate, int silu, void *dx, void *dz,
                            float *dw, float *dbias, int64_t M, int64_t D, int64_t G, void *ws,
                            size_t ws_bytes, cudaStream_t stream)
{
    const char *fn = "mg_group_norm_bwd";
    begin_call();
    MG_TRY(check_type(fn, dt));
    MG_TRY(check_norm(fn, M, D, G, gate));
    MG_TRY(check_ld(fn, "dy", lddy, D));
    MG_TRY(check_ld(fn, "x", ldx, D));
    if (gate != MG_GATE_NONE) MG_TRY(check_ld(fn, "z", ldz, D));
    if (((z == nullptr) != (gate == MG_GATE_NONE) || (dz == nullptr) != (gate == MG_GATE_NONE)) &&
        M > 0 && D > 0)
        return fail(MG_ERR_INVALID_ARG, "%s: z and dz go with a gate, and a gate with both", fn);
    if (D == 0) return MG_OK;
    if (M == 0) {
        MG_TRY(zero(fn, dw, D, "dw", stream));
        return zero(fn, dbias, D, "dbias", stream);
    }
    const size_t es = esize(dt), n = size_t(M) * D * es;
    MG_TRY(check_ws(fn, ws, ws_bytes, norm_ws_bytes(M, D, G)));
    MG_TRY(check_bufs(fn, {{dy, extent(M, lddy, D, es), "dy", false},
                           {stats, size_t(M) * G * 8, "stats", false},
                           {x, extent(M, ldx, D, es), "x", false},
                           {z, extent(M, ldz, D, es), "z", false, true},
                           {w, size_t(D) * 4, "w", false},
                           {bias, size_t(D) * 4, "bias", false, true},
                           {dx, n, "dx", true},
                           {dz, n, "dz", true, true},
                           {dw, size_t(D) * 4, "dw", true},
                           {dbias, size_t(D) * 4, "dbias", true, true},
                           {ws, ws_bytes, "workspace", true}}));
    NormArgs p{};
    p.dy = dy, p.lddy = lddy, p.stats_in = stats, p.x = x, p.ldx = ldx, p.z = z, p.ldz = ldz;
    p.w = w, p.bias = bias, p.rms = rms, p.gate = gate, p.silu = silu, p.dx = dx, p.dz = dz;
    p.dw = dw, p.dbias = dbias, p.M = M, p.D = D, p.G = G, p.ws = ws;
    return launch_norm_bwd(p, dt, stream);
}

mg_status mg_ssm_call(mg_ssm_op op, const uint64_t *args, int nargs)
{
    if (args == nullptr) return fail(MG_ERR_INVALID_ARG, "mg_ssm_call: args is NULL");
    switch (op) {
    case MG_CAUSAL_CONV_FWD: return call_words(mg_causal_conv_fwd, args, nargs);
    case MG_CAUSAL_CONV_BWD: return call_words(mg_causal_conv_bwd, args, nargs);
    case MG_CAUSAL_CONV_STEP: return call_words(mg_causal_conv_step, args, nargs);
    case MG_SELECTIVE_SCAN_FWD: return call_words(mg_selective_scan_fwd, args, nargs);
    case MG_SELECTIVE_SCAN_BWD: return call_words(mg_selective_scan_bwd, args, nargs);
    case MG_SELECTIVE_SCAN_STEP: return call_words(mg_selective_scan_step, args, nargs);
    case MG_GROUP_NORM_FWD: return call_words(mg_group_norm_fwd, args, nargs);
    case MG_GROUP_NORM_BWD: return call_words(mg_group_norm_bwd, args, nargs);
    }
    return fail(MG_ERR_INVALID_ARG, "mg_ssm_call: op %d", int(op));
}

}  // extern "C"
