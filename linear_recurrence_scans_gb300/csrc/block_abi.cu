// The C entry points of mg_block.h: argument validation (all of it before any
// launch) and the calls without rows.
#include <cmath>

#include "abi_calls.cuh"
#include "block.cuh"

using namespace mg;

namespace {

mg_status check_gated(const char *fn, int64_t B, int64_t T, int64_t H, int64_t G, int64_t N, int64_t P)
{
    MG_TRY(check_dims(fn, {B, T, H, P}));
    MG_TRY(check_dims(fn, {G, N}));
    if (N < 1 || N > kGatedMax || P < 1 || P > kGatedMax)
        return fail(MG_ERR_UNSUPPORTED, "%s: N = %lld, P = %lld outside [1, %d]", fn, (long long)N, (long long)P, kGatedMax);
    if (G < 1 || H % G != 0)
        return fail(MG_ERR_INVALID_ARG, "%s: H = %lld is not a multiple of G = %lld", fn, (long long)H, (long long)G);
    if (H > (int64_t(1) << 16)) return fail(MG_ERR_UNSUPPORTED, "%s: %lld heads, at most 2^16", fn, (long long)H);
    MG_TRY(check_size(fn, B * T, H * P));
    return check_size(fn, B * T, G * N);
}

// Sequences, and the 32-bit counts of chunks.
mg_status check_gated_seqs(const char *fn, const int64_t *cu, int64_t nseq, int64_t B, int64_t T, int64_t H, int64_t N,
                           int64_t P)
{
    MG_TRY(check_seqs(fn, cu, nseq, B));
    if (B * T / 64 + nseq > INT32_MAX) return fail(MG_ERR_UNSUPPORTED, "%s: too many rows", fn);
    return check_size(fn, nseq, H * N * P);
}

// A factor that the kernels take as a float.
mg_status check_scale(const char *fn, double v, const char *name)
{
    return std::isfinite(float(v)) ? MG_OK : fail(MG_ERR_INVALID_ARG, "%s: %s must be finite in float32", fn, name);
}

mg_status check_rms(const char *fn, int64_t M, int64_t D)
{
    MG_TRY(check_dims(fn, {M, D}));
    if (D > kRmsMaxD)
        return fail(MG_ERR_UNSUPPORTED, "%s: rows of %lld channels, at most %lld", fn, (long long)D, (long long)kRmsMaxD);
    return check_size(fn, M, D);
}

// What mg_rms_norm_fwd and _quant share: x, res, w and r.
mg_status check_rms_in(const char *fn, const void *res, int64_t ldx, int64_t ldres, const void *r, double eps, int64_t M,
                       int64_t D)
{
    MG_TRY(check_ld(fn, "x", ldx, D));
    if (res != nullptr) MG_TRY(check_ld(fn, "res", ldres, D));
    if (M > 0 && D > 0 && (res == nullptr) != (r == nullptr))
        return fail(MG_ERR_INVALID_ARG, "%s: r goes with res", fn);
    if (M > 0 && D == 0) return fail(MG_ERR_INVALID_ARG, "%s: rows without channels have no mean", fn);
    if (eps < 0.0) return fail(MG_ERR_INVALID_ARG, "%s: eps must not be negative", fn);
    return check_scale(fn, eps, "eps");
}

}  // namespace

extern "C" {

size_t mg_gated_scan_workspace_size(int64_t B, int64_t T, int64_t H, int64_t G, int64_t N, int64_t P, int64_t nseq,
                                    int packed, mg_dtype dt, int bwd)
{
    const char *fn = "mg_gated_scan_workspace_size";
    if (check_type(fn, dt) != MG_OK || check_gated(fn, B, T, H, G, N, P) != MG_OK || nseq < 0 ||
        nseq > INT32_MAX - 1 || B * T / 64 + nseq > INT32_MAX)
        return 0;
    if (B == 0 || T == 0 || H == 0) return kControlBytes;
    return gated_ws_bytes(B, T, H, G, N, P, nseq, packed != 0, dt, bwd != 0);
}

size_t mg_gated_scan_saved_size(int64_t B, int64_t T, int64_t H, int64_t N, int64_t P, int64_t nseq, int packed,
                                mg_dtype dt)
{
    const char *fn = "mg_gated_scan_saved_size";
    if (check_type(fn, dt) != MG_OK || check_gated(fn, B, T, H, 1, N, P) != MG_OK || nseq < 0 ||
        nseq > INT32_MAX - 1 || B * T / 64 + nseq > INT32_MAX)
        return 0;
    if (B == 0 || T == 0 || H == 0) return 0;
    return gated_saved_bytes(B, T, H, N, P, nseq, packed != 0, dt);
}

mg_status mg_gated_scan_fwd(const void *q, int64_t ldq, const void *k, int64_t ldk, const void *v, int64_t ldv,
                            const float *g, int64_t ldg, mg_dtype dt, double scale, const float *S0,
                            const int64_t *cu_seqlens, int64_t nseq, void *o, float *S_last, float *saved, int64_t B,
                            int64_t T, int64_t H, int64_t G, int64_t N, int64_t P, void *ws, size_t ws_bytes,
                            cudaStream_t stream)
{
    const char *fn = "mg_gated_scan_fwd";
    begin_call();
    MG_TRY(check_type(fn, dt));
    MG_TRY(check_gated(fn, B, T, H, G, N, P));
    MG_TRY(check_gated_seqs(fn, cu_seqlens, nseq, B, T, H, N, P));
    MG_TRY(check_ld(fn, "q", ldq, G * N));
    MG_TRY(check_ld(fn, "k", ldk, G * N));
    MG_TRY(check_ld(fn, "v", ldv, H * P));
    MG_TRY(check_ld(fn, "g", ldg, H));
    MG_TRY(check_scale(fn, scale, "scale"));
    const size_t es = esize(dt), st = size_t(nseq) * H * N * P * 4, rows = size_t(B) * T;
    if (H == 0) return MG_OK;
    if (rows == 0) return pass_state(fn, S_last, S0, st, stream);
    const bool packed = cu_seqlens != nullptr;
    MG_TRY(check_ws(fn, ws, ws_bytes,
                    gated_ws_bytes(B, T, H, G, N, P, nseq, packed, dt, false)));
    MG_TRY(check_bufs(fn, {{q, extent(rows, ldq, G * N, es), "q", false},
                           {k, extent(rows, ldk, G * N, es), "k", false},
                           {v, extent(rows, ldv, H * P, es), "v", false},
                           {g, extent(rows, ldg, H, 4), "g", false, false, 4},
                           {S0, st, "S0", false, true},
                           {o, rows * H * P * es, "o", true},
                           {S_last, st, "S_last", true, true},
                           {saved, gated_saved_bytes(B, T, H, N, P, nseq, packed, dt), "saved", true, true},
                           {ws, ws_bytes, "workspace", true}}));
    GatedArgs p{};
    p.q = q, p.ldq = ldq, p.k = k, p.ldk = ldk, p.v = v, p.ldv = ldv, p.g = g, p.ldg = ldg, p.scale = float(scale);
    p.S0 = S0, p.cu = cu_seqlens, p.nseq = nseq, p.o = o, p.S_last = S_last, p.saved = saved;
    p.B = B, p.T = T, p.H = int(H), p.G = int(G), p.N = int(N), p.P = int(P), p.ws = ws;
    return launch_gated_fwd(p, dt, stream);
}

mg_status mg_gated_scan_bwd(const void *dout, int64_t lddo, const float *saved, const void *q, int64_t ldq,
                            const void *k, int64_t ldk, const void *v, int64_t ldv, const float *g, int64_t ldg,
                            mg_dtype dt, double scale, const float *dS_last, const int64_t *cu_seqlens, int64_t nseq,
                            void *dq, void *dk, void *dv, float *dg, float *dS0, int64_t B, int64_t T, int64_t H,
                            int64_t G, int64_t N, int64_t P, void *ws, size_t ws_bytes, cudaStream_t stream)
{
    const char *fn = "mg_gated_scan_bwd";
    begin_call();
    MG_TRY(check_type(fn, dt));
    MG_TRY(check_gated(fn, B, T, H, G, N, P));
    MG_TRY(check_gated_seqs(fn, cu_seqlens, nseq, B, T, H, N, P));
    MG_TRY(check_ld(fn, "dout", lddo, H * P));
    MG_TRY(check_ld(fn, "q", ldq, G * N));
    MG_TRY(check_ld(fn, "k", ldk, G * N));
    MG_TRY(check_ld(fn, "v", ldv, H * P));
    MG_TRY(check_ld(fn, "g", ldg, H));
    MG_TRY(check_scale(fn, scale, "scale"));
    const size_t es = esize(dt), st = size_t(nseq) * H * N * P * 4, rows = size_t(B) * T;
    const bool packed = cu_seqlens != nullptr;
    if (H == 0) {   // no head sends anything to q and k
        const size_t n = rows * G * N * es;
        for (void *out : {dq, dk})
            if (n > 0) MG_TRY(pass_state(fn, out, nullptr, n, stream));
        return MG_OK;
    }
    if (rows == 0) return pass_state(fn, dS0, dS_last, st, stream);
    MG_TRY(check_ws(fn, ws, ws_bytes, gated_ws_bytes(B, T, H, G, N, P, nseq, packed, dt, true)));
    MG_TRY(check_bufs(fn, {{dout, extent(rows, lddo, H * P, es), "dout", false},
                           {saved, gated_saved_bytes(B, T, H, N, P, nseq, packed, dt), "saved", false},
                           {q, extent(rows, ldq, G * N, es), "q", false},
                           {k, extent(rows, ldk, G * N, es), "k", false},
                           {v, extent(rows, ldv, H * P, es), "v", false},
                           {g, extent(rows, ldg, H, 4), "g", false, false, 4},
                           {dS_last, st, "dS_last", false, true},
                           {dq, rows * G * N * es, "dq", true},
                           {dk, rows * G * N * es, "dk", true},
                           {dv, rows * H * P * es, "dv", true},
                           {dg, rows * H * 4, "dg", true},
                           {dS0, st, "dS0", true, true},
                           {ws, ws_bytes, "workspace", true}}));
    GatedArgs p{};
    p.dout = dout, p.lddo = lddo, p.saved_in = saved, p.q = q, p.ldq = ldq, p.k = k, p.ldk = ldk, p.v = v, p.ldv = ldv;
    p.g = g, p.ldg = ldg, p.scale = float(scale), p.dS_last = dS_last, p.cu = cu_seqlens, p.nseq = nseq;
    p.dq = dq, p.dk = dk, p.dv = dv, p.dg = dg, p.dS0 = dS0;
    p.B = B, p.T = T, p.H = int(H), p.G = int(G), p.N = int(N), p.P = int(P), p.ws = ws;
    return launch_gated_bwd(p, dt, stream);
}

mg_status mg_gated_scan_step(const void *q, int64_t ldq, const void *k, int64_t ldk, const void *v, int64_t ldv,
                             const float *g, int64_t ldg, mg_dtype dt, double scale, float *state, int64_t nslots,
                             const int64_t *slots, void *o, int64_t B, int64_t H, int64_t G, int64_t N, int64_t P,
                             cudaStream_t stream)
{
    const char *fn = "mg_gated_scan_step";
    begin_call();
    MG_TRY(check_type(fn, dt));
    MG_TRY(check_gated(fn, B, 1, H, G, N, P));
    MG_TRY(check_slots(fn, slots, nslots, B));
    MG_TRY(check_ld(fn, "q", ldq, G * N));
    MG_TRY(check_ld(fn, "k", ldk, G * N));
    MG_TRY(check_ld(fn, "v", ldv, H * P));
    MG_TRY(check_ld(fn, "g", ldg, H));
    MG_TRY(check_scale(fn, scale, "scale"));
    MG_TRY(check_dims(fn, {nslots, H, N, P}));
    if (B == 0 || H == 0) return MG_OK;
    const size_t es = esize(dt), pool = size_t(nslots) * H * N * P * 4;
    MG_TRY(check_bufs(fn, {{q, extent(B, ldq, G * N, es), "q", false},
                           {k, extent(B, ldk, G * N, es), "k", false},
                           {v, extent(B, ldv, H * P, es), "v", false},
                           {g, extent(B, ldg, H, 4), "g", false, false, 4},
                           {slots, size_t(B) * 8, "slots", false, true, 8},
                           {state, pool, "state", true, pool == 0},
                           {o, size_t(B) * H * P * es, "o", true}}));
    GatedStepArgs p{};
    p.q = q, p.ldq = ldq, p.k = k, p.ldk = ldk, p.v = v, p.ldv = ldv, p.g = g, p.ldg = ldg, p.scale = float(scale);
    p.state = state, p.nslots = nslots, p.slots = slots, p.o = o;
    p.B = B, p.H = int(H), p.G = int(G), p.N = int(N), p.P = int(P);
    return launch_gated_step(p, dt, stream);
}

mg_status mg_rms_norm_fwd(const void *x, int64_t ldx, const void *res, int64_t ldres, mg_dtype dt, const float *w,
                          double eps, void *y, void *r, float *rstd, int64_t M, int64_t D, cudaStream_t stream)
{
    const char *fn = "mg_rms_norm_fwd";
    begin_call();
    MG_TRY(check_type(fn, dt));
    MG_TRY(check_rms(fn, M, D));
    MG_TRY(check_rms_in(fn, res, ldx, ldres, r, eps, M, D));
    if (M == 0) return MG_OK;
    const size_t es = esize(dt), n = size_t(M) * D * es;
    const bool in_place = res != nullptr && res == r && ldres == D;
    MG_TRY(check_bufs(fn, {{x, extent(M, ldx, D, es), "x", false},
                           {in_place ? nullptr : res, extent(M, ldres, D, es), "res", false, true},
                           {w, size_t(D) * 4, "w", false},
                           {y, n, "y", true},
                           {r, n, "r", true, true},
                           {rstd, size_t(M) * 4, "rstd", true, true}}));
    RmsArgs p{};
    p.x = x, p.ldx = ldx, p.res = res, p.ldres = ldres, p.w = w, p.eps = float(eps), p.y = y, p.r = r, p.rstd = rstd;
    p.M = M, p.D = D;
    return launch_rms_fwd(p, dt, stream);
}

mg_status mg_rms_norm_quant(const void *x, int64_t ldx, const void *res, int64_t ldres, mg_dtype dt, const float *w,
                            double eps, void *q, float *scale, void *r, int64_t block, int64_t M, int64_t D,
                            cudaStream_t stream)
{
    const char *fn = "mg_rms_norm_quant";
    begin_call();
    MG_TRY(check_type(fn, dt));
    MG_TRY(check_rms(fn, M, D));
    MG_TRY(check_rms_in(fn, res, ldx, ldres, r, eps, M, D));
    if (block != 0 && block != 32 && block != 64 && block != 128 && block != 256)
        return fail(MG_ERR_UNSUPPORTED, "%s: blocks of %lld channels (32, 64, 128, 256, or 0 for the row)", fn,
                    (long long)block);
    if (block != 0 && D % block != 0)
        return fail(MG_ERR_INVALID_ARG, "%s: D = %lld is not a multiple of the block of %lld", fn, (long long)D,
                    (long long)block);
    if (M == 0) return MG_OK;
    const size_t es = esize(dt), n = size_t(M) * D;
    const bool in_place = res != nullptr && res == r && ldres == D;
    MG_TRY(check_bufs(fn, {{x, extent(M, ldx, D, es), "x", false},
                           {in_place ? nullptr : res, extent(M, ldres, D, es), "res", false, true},
                           {w, size_t(D) * 4, "w", false},
                           {q, n, "q", true},
                           {scale, size_t(M) * (block != 0 ? D / block : 1) * 4, "scale", true},
                           {r, n * es, "r", true, true}}));
    RmsArgs p{};
    p.x = x, p.ldx = ldx, p.res = res, p.ldres = ldres, p.w = w, p.eps = float(eps), p.q = q, p.scale = scale, p.r = r;
    p.block = block, p.M = M, p.D = D;
    return launch_rms_quant(p, dt, stream);
}

size_t mg_rms_norm_workspace_size(int64_t M, int64_t D)
{
    if (check_rms("mg_rms_norm_workspace_size", M, D) != MG_OK) return 0;
    if (M == 0 || D == 0) return kControlBytes;
    return rms_ws_bytes(M, D);
}

mg_status mg_rms_norm_bwd(const void *dy, int64_t lddy, const float *rstd, const void *r, int64_t ldr, const void *dr,
                          int64_t lddr, mg_dtype dt, const float *w, void *dx, float *dw, int64_t M, int64_t D,
                          void *ws, size_t ws_bytes, cudaStream_t stream)
{
    const char *fn = "mg_rms_norm_bwd";
    begin_call();
    MG_TRY(check_type(fn, dt));
    MG_TRY(check_rms(fn, M, D));
    MG_TRY(check_ld(fn, "dy", lddy, D));
    MG_TRY(check_ld(fn, "r", ldr, D));
    if (dr != nullptr) MG_TRY(check_ld(fn, "dr", lddr, D));
    if (D == 0) return MG_OK;
    if (M == 0) return zero(fn, dw, D, "dw", stream);
    const size_t es = esize(dt);
    MG_TRY(check_ws(fn, ws, ws_bytes, rms_ws_bytes(M, D)));
    MG_TRY(check_bufs(fn, {{dy, extent(M, lddy, D, es), "dy", false},
                           {rstd, size_t(M) * 4, "rstd", false},
                           {r, extent(M, ldr, D, es), "r", false},
                           {dr, extent(M, lddr, D, es), "dr", false, true},
                           {w, size_t(D) * 4, "w", false},
                           {dx, size_t(M) * D * es, "dx", true},
                           {dw, size_t(D) * 4, "dw", true},
                           {ws, ws_bytes, "workspace", true}}));
    RmsArgs p{};
    p.dy = dy, p.lddy = lddy, p.rstd_in = rstd, p.x = r, p.ldx = ldr, p.dr = dr, p.lddr = lddr, p.w = w, p.dx = dx;
    p.dw = dw, p.M = M, p.D = D, p.ws = ws;
    return launch_rms_bwd(p, dt, stream);
}

mg_status mg_block_call(mg_block_op op, const uint64_t *args, int nargs)
{
    if (args == nullptr) return fail(MG_ERR_INVALID_ARG, "mg_block_call: args is NULL");
    switch (op) {
    case MG_GATED_SCAN_FWD: return call_words(mg_gated_scan_fwd, args, nargs);
    case MG_GATED_SCAN_BWD: return call_words(mg_gated_scan_bwd, args, nargs);
    case MG_GATED_SCAN_STEP: return call_words(mg_gated_scan_step, args, nargs);
    case MG_RMS_NORM_FWD: return call_words(mg_rms_norm_fwd, args, nargs);
    case MG_RMS_NORM_QUANT: return call_words(mg_rms_norm_quant, args, nargs);
    case MG_RMS_NORM_BWD: return call_words(mg_rms_norm_bwd, args, nargs);
    }
    return fail(MG_ERR_INVALID_ARG, "mg_block_call: op %d", int(op));
}

}  // extern "C"
