/*
 * mg_block.h -- the operators of a gated block, next to those of mg_ssm.h: a
 * gated linear recurrence whose state is a matrix per head, and the
 * root-mean-square norm with the residual's addition that such a block begins
 * with, for prompts, for training and for single tokens.
 *
 * The conventions are those of mg_ssm.h (types, row strides, sequences, slots,
 * workspaces, errors before any launch, empty calls), with these additions:
 *
 * Heads.  v and o have H heads of P values, q and k G groups of N values, a row
 *   being H*P (G*N) values with its heads (groups) one after another.  H is a
 *   multiple of G, and head h reads group h / (H/G).  1 <= N, P <= 128.
 * Gates.  g (B,T,H), row stride ldg, is float32 whatever dt is: the logarithm
 *   of a row's decay, meant to be <= 0.  A gate below -128 counts as -128 (its
 *   decay, 2.6e-56, is 0 in float32); -inf forgets everything.
 * Arithmetic.  Products of bf16 calls run on the tensor cores with float32 sums:
 *   a factor that is no input (weights, states) goes in as bf16 pieces that add up
 *   to 2^-16 of it where the result is an activation, to 2^-24 where it is float32.
 * Not-a-numbers.  The recurrence works on chunks of rows: an infinity or NaN in
 *   a row may make NaN of the rows of the same sequence and head after it, and
 *   of those before it in the same chunk of 128 rows (backwards the other way
 *   round).  Nothing of one sequence reaches another.
 */
#ifndef MG_BLOCK_H
#define MG_BLOCK_H

#include "mg_ssm.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Gated recurrence.  Per head, with the N x P state S:
 *   S_t = exp(g_t) S_{t-1} + k_t v_t^T,   o_t = scale S_t^T q_t
 * from S0 (nseq,H,N,P) float32 (NULL: zero).  q, k (B,T,G,N) and v (B,T,H,P)
 * have type dt; o is dense, type dt; S_last (nseq,H,N,P) float32 (may be NULL)
 * receives each sequence's last state.  saved (may be NULL) receives
 * mg_gated_scan_saved_size bytes that mg_gated_scan_bwd reads.
 */
mg_status mg_gated_scan_fwd(const void *q, int64_t ldq, const void *k, int64_t ldk, const void *v,
                            int64_t ldv, const float *g, int64_t ldg, mg_dtype dt, double scale,
                            const float *S0, const int64_t *cu_seqlens, int64_t nseq, void *o,
                            float *S_last, float *saved, int64_t B, int64_t T, int64_t H,
                            int64_t G, int64_t N, int64_t P, void *ws, size_t ws_bytes,
                            cudaStream_t stream);

/* Bytes of the workspace of mg_gated_scan_fwd (of mg_gated_scan_bwd with
 * bwd != 0) and of `saved`, for nseq sequences, packed or dense (0: invalid or
 * unsupported sizes; nothing is saved of a batch without rows or heads either). */
size_t mg_gated_scan_workspace_size(int64_t B, int64_t T, int64_t H, int64_t G, int64_t N,
                                    int64_t P, int64_t nseq, int packed, mg_dtype dt, int bwd);
size_t mg_gated_scan_saved_size(int64_t B, int64_t T, int64_t H, int64_t N, int64_t P,
                                int64_t nseq, int packed, mg_dtype dt);

/*
 * Gradients of sum(dout*o) + sum(dS_last*S_last) for mg_gated_scan_fwd, from
 * `saved` of a forward call on the same inputs.  With D_t the adjoint of S_t,
 *   D_t = scale q_t dout_t^T + exp(g_{t+1}) D_{t+1}  (+ dS_last at a sequence's last row):
 *   dq_t = scale sum_h S_t dout_t,  dk_t = sum_h D_t v_t  (sums over the heads of a group),
 *   dv_t = D_t^T k_t,  dg_t = <D_t, exp(g_t) S_{t-1}>,  dS0 = exp(g_1) D_1
 * (dS_last, or 0, for an empty sequence).  dS_last may be NULL (zero), dS0 may
 * be NULL (not written).  dq, dk (B,T,G,N) and dv (B,T,H,P) are dense, type dt;
 * dg (B,T,H) and dS0 float32.  Sums are taken in a fixed order: repeated calls
 * give the same bits.
 */
mg_status mg_gated_scan_bwd(const void *dout, int64_t lddo, const float *saved, const void *q,
                            int64_t ldq, const void *k, int64_t ldk, const void *v, int64_t ldv,
                            const float *g, int64_t ldg, mg_dtype dt, double scale,
                            const float *dS_last, const int64_t *cu_seqlens, int64_t nseq,
                            void *dq, void *dk, void *dv, float *dg, float *dS0, int64_t B,
                            int64_t T, int64_t H, int64_t G, int64_t N, int64_t P, void *ws,
                            size_t ws_bytes, cudaStream_t stream);

/*
 * One token: row i of q, k (B,G,N), v (B,H,P) and g (B,H) advances the state
 * slots[i] of state (nslots,H,N,P) float32 in place by one row of
 * mg_gated_scan_fwd; o (B,H,P), type dt.
 */
mg_status mg_gated_scan_step(const void *q, int64_t ldq, const void *k, int64_t ldk, const void *v,
                             int64_t ldv, const float *g, int64_t ldg, mg_dtype dt, double scale,
                             float *state, int64_t nslots, const int64_t *slots, void *o,
                             int64_t B, int64_t H, int64_t G, int64_t N, int64_t P,
                             cudaStream_t stream);

/*
 * Root-mean-square norm behind a residual's addition, rows of 1 <= D <= 16384
 * channels:
 *   r = x + res, rounded to dt (r = x without res),  y = r rstd w,
 *   rstd = (mean(r^2) + eps)^(-1/2)
 * x and res (M,D) have type dt (res may be NULL); w (D) float32.  r (M,D),
 * dense, type dt, is written where res is given (NULL without it); y is dense,
 * type dt; rstd (M) float32 (may be NULL) is for the gradients.  r may be the
 * residual's own buffer (res == r, both dense); other outputs overlap nothing.
 */
mg_status mg_rms_norm_fwd(const void *x, int64_t ldx, const void *res, int64_t ldres, mg_dtype dt,
                          const float *w, double eps, void *y, void *r, float *rstd, int64_t M,
                          int64_t D, cudaStream_t stream);

/*
 * The same with y in 8 bits: for each block of `block` neighbouring channels (32,
 * 64, 128 or 256, a divisor of D; 0: the whole row)
 *   scale = max(largest |y|, 1e-30) / 448,   q = y / scale, rounded to e4m3
 * from the float32 y.  q (M,D) dense, one byte a value; scale (M, D/block)
 * float32.  A block with a NaN has a scale of NaN.
 */
mg_status mg_rms_norm_quant(const void *x, int64_t ldx, const void *res, int64_t ldres,
                            mg_dtype dt, const float *w, double eps, void *q, float *scale,
                            void *r, int64_t block, int64_t M, int64_t D, cudaStream_t stream);

/* Workspace of mg_rms_norm_bwd (0: invalid sizes). */
size_t mg_rms_norm_workspace_size(int64_t M, int64_t D);

/*
 * Gradients of sum(dy*y) + sum(dr*r) for mg_rms_norm_fwd, from its r (x without
 * a residual) and rstd: dx (M,D), dense, type dt, is the gradient of x and of
 * res alike (dr, type dt, may be NULL); dw (D) float32.  Sums over rows are
 * taken in a fixed order.
 */
mg_status mg_rms_norm_bwd(const void *dy, int64_t lddy, const float *rstd, const void *r,
                          int64_t ldr, const void *dr, int64_t lddr, mg_dtype dt, const float *w,
                          void *dx, float *dw, int64_t M, int64_t D, void *ws, size_t ws_bytes,
                          cudaStream_t stream);

/* The calls above with their arguments as 64-bit words (see mg_ssm_call). */
typedef enum mg_block_op {
    MG_GATED_SCAN_FWD = 0,
    MG_GATED_SCAN_BWD = 1,
    MG_GATED_SCAN_STEP = 2,
    MG_RMS_NORM_FWD = 3,
    MG_RMS_NORM_QUANT = 4,
    MG_RMS_NORM_BWD = 5
} mg_block_op;
mg_status mg_block_call(mg_block_op op, const uint64_t *args, int nargs);

#ifdef __cplusplus
}
#endif

#endif /* MG_BLOCK_H */
