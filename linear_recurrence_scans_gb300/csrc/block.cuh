// Shared by the gated block's kernels (rms_norm.cu, gated_scan*.cu): argument
// blocks and launchers.
#pragma once

#include "mg_block.h"
#include "ssm.cuh"

namespace mg {

struct RmsArgs {
    const void *x, *res, *dy, *dr;
    int64_t ldx, ldres, lddy, lddr;
    const float *w;
    float eps;
    void *y, *r, *q, *dx;
    float *rstd, *scale, *dw;
    const float *rstd_in;
    int64_t block, M, D;
    void *ws;
};
constexpr int64_t kRmsMaxD = 16384;
size_t rms_ws_bytes(int64_t M, int64_t D);
mg_status launch_rms_fwd(const RmsArgs &p, mg_dtype dt, cudaStream_t s);
mg_status launch_rms_quant(const RmsArgs &p, mg_dtype dt, cudaStream_t s);
mg_status launch_rms_bwd(const RmsArgs &p, mg_dtype dt, cudaStream_t s);

struct GatedArgs {
    const void *q, *k, *v, *dout;
    const float *g;
    int64_t ldq, ldk, ldv, ldg, lddo;
    float scale;
    const float *S0, *dS_last;
    const int64_t *cu;
    int64_t nseq;
    void *o, *dq, *dk, *dv;
    float *S_last, *saved, *dg, *dS0;
    const float *saved_in;
    int64_t B, T;
    int H, G, N, P;
    void *ws;
};
constexpr int kGatedMax = 128;   // N and P
size_t gated_saved_bytes(int64_t B, int64_t T, int64_t H, int64_t N, int64_t P, int64_t nseq, bool packed, mg_dtype dt);
size_t gated_ws_bytes(int64_t B, int64_t T, int64_t H, int64_t G, int64_t N, int64_t P, int64_t nseq, bool packed,
                      mg_dtype dt, bool bwd);
mg_status launch_gated_fwd(const GatedArgs &p, mg_dtype dt, cudaStream_t s);
mg_status launch_gated_bwd(const GatedArgs &p, mg_dtype dt, cudaStream_t s);

struct GatedStepArgs {
    const void *q, *k, *v;
    const float *g;
    int64_t ldq, ldk, ldv, ldg;
    float scale;
    float *state;
    int64_t nslots;
    const int64_t *slots;
    void *o;
    int64_t B;
    int H, G, N, P;
};
mg_status launch_gated_step(const GatedStepArgs &p, mg_dtype dt, cudaStream_t s);

}  // namespace mg
