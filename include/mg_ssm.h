/*
 * mg_ssm.h -- the operators of a selective state space mixer, next to the
 * scans of mg_scan.h: the short causal depthwise convolution, the selective
 * scan and the gated group norm, for prompts, for training and for single
 * tokens.
 *
 * The conventions are those of mg_scan.h (device pointers 16-byte aligned,
 * outputs overlapping nothing, caller-owned 256-byte aligned workspace that
 * any op may reuse, asynchronous calls on `stream`, argument errors reported
 * before any launch), with these additions:
 *
 * Activations have the type `dt` (MG_F32 or MG_BF16), the same for all
 *   activations of a call; parameters, states and parameter gradients are
 *   float32 (the convolution's state has the activations' type).  Arithmetic
 *   is float32; an activation output is rounded once, at its store.
 * Rows.  An activation input (x, z, raw step sizes, B, C, upstream gradients)
 *   is given with its row stride `ld*` in elements: element (b, t, i) sits at
 *   (b*T + t)*ld + i, so a slice of a wider projection is read in place.
 *   Any ld >= the row's width is accepted; wide loads are used where the rows
 *   keep 16-byte alignment.  Outputs are dense.
 * Sequences.  With cu_seqlens = NULL a batch is B sequences of T rows.
 *   Otherwise B must be 1 and T is the packed length: sequence s holds rows
 *   cu_seqlens[s] .. cu_seqlens[s+1]-1 (DEVICE array of nseq + 1 int64
 *   offsets, non-decreasing from 0 to T, empty sequences allowed).  States
 *   have one entry for each sequence: nseq = B in the dense case.  Nothing of
 *   one sequence, not even a NaN, reaches another.  A cu_seqlens that breaks
 *   the rules is detected on the device: outputs are then unspecified, no
 *   memory outside the buffers is touched, and the next mg_workspace_status
 *   on the workspace returns MG_ERR_INVALID_ARG.
 * Slots.  A token call works on a pool of `nslots` states: row i uses state
 *   slots[i] (DEVICE int64 array of B, 8-byte aligned; NULL: state i, and
 *   nslots >= B).  A row whose slot is negative or not below nslots is idle:
 *   its output is 0 and no state changes.  Rows of one call must use
 *   different slots.
 * Infinities.  The selective scan's results are finite where the formulas' are;
 *   where an infinite input makes them infinite they may be NaN instead (a sum
 *   over states may take in states of 0 beside N, and a run of decays one
 *   product that is 0 in float32: 0 times infinity).
 * Empty calls (no rows) return MG_OK; the states that a call returns are then
 *   the states that it was given.
 */
#ifndef MG_SSM_H
#define MG_SSM_H

#include "mg_scan.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Sizes.  A call has at most 2^36 values (rows x channels, and states), and no
 * launch more than 2^31 - 1 blocks; beyond either MG_ERR_UNSUPPORTED is
 * returned before any launch.
 */

/*
 * Short causal depthwise convolution with an activation:
 *   v_r[d] = bias[d] + sum_{k<W} w[d,k] x_{r-W+1+k}[d],
 *   y_r = silu(v_r) = v_r sigmoid(v_r) if silu, else v_r.
 * Rows before a sequence's first are its x0 (nseq, W-1, D), type dt (NULL:
 * zero; row W-2 is the latest).  w is (D, W) and bias (D) float32 (bias may
 * be NULL); 1 <= W <= 8.  x_last (nseq, W-1, D), type dt (may be NULL)
 * receives each sequence's last W-1 inputs, x0's where it has fewer rows.
 */
mg_status mg_causal_conv_fwd(const void *x, int64_t ldx, mg_dtype dt, const float *w,
                             const float *bias, const void *x0, const int64_t *cu_seqlens,
                             int64_t nseq, int silu, void *y, void *x_last,
                             int64_t B, int64_t T, int64_t D, int W,
                             void *ws, size_t ws_bytes, cudaStream_t stream);

/* Workspace of mg_causal_conv_fwd and mg_causal_conv_bwd (0: invalid sizes). */
size_t mg_causal_conv_workspace_size(int64_t B, int64_t T, int64_t D, int W);

/*
 * Gradients for mg_causal_conv_fwd of sum(dy*y) + sum(dx_last*x_last):
 *   dv_r = dy_r silu'(v_r),  dx_r = sum_k w[:,k] dv_{r+W-1-k}  (rows of the
 *   same sequence), dw[d,k] = sum_r dv_r x_{r-W+1+k}, dbias = sum_r dv_r,
 * and dx0 (nseq, W-1, D) the same for the rows before a sequence.  dx_last
 * may be NULL (zero); dbias and dx0 may be NULL (not written).  dx is dense
 * (B,T,D), type dt; dw (D,W), dbias (D) float32.  Sums over rows are taken
 * in a fixed order: repeated calls give the same bits.
 */
mg_status mg_causal_conv_bwd(const void *dy, int64_t lddy, const void *x, int64_t ldx, mg_dtype dt,
                             const float *w, const float *bias, const void *x0,
                             const void *dx_last, const int64_t *cu_seqlens, int64_t nseq,
                             int silu, void *dx, float *dw, float *dbias, void *dx0,
                             int64_t B, int64_t T, int64_t D, int W,
                             void *ws, size_t ws_bytes, cudaStream_t stream);

/*
 * One token: row i of x (B, D) enters the convolution state slots[i] of
 * state (nslots, W-1, D), type dt, which is shifted by one row in place;
 * y (B, D).
 */
mg_status mg_causal_conv_step(const void *x, int64_t ldx, mg_dtype dt, const float *w,
                              const float *bias, void *state, int64_t nslots,
                              const int64_t *slots, int silu, void *y,
                              int64_t B, int64_t D, int W, cudaStream_t stream);

/*
 * Selective scan.  x and raw step sizes `raw` are (B,T,D); Bm and Cm are
 * (B,T,G,N), a row being G*N values; A (D,N), Dskip (D, may be NULL) and
 * dt_bias (D, may be NULL) float32.  Channel d belongs to group d / (D/G),
 * D a multiple of G.  With delta = raw + dt_bias, or softplus of that:
 *   h_r[d,n] = exp(delta_r[d] A[d,n]) h_{r-1}[d,n] + delta_r[d] x_r[d] Bm_r[g,n]
 *   y_r[d]   = sum_n Cm_r[g,n] h_r[d,n] + Dskip[d] x_r[d]
 * from h0 (nseq,D,N) float32 (NULL: zero).  y is dense, type dt; h_last
 * (nseq,D,N) float32 (may be NULL) receives each sequence's last state.
 * 1 <= N <= 64.  saved (may be NULL) receives mg_selective_scan_saved_size
 * bytes that mg_selective_scan_bwd reads: the states before every
 * mg_selective_scan_saved_rows() rows, (B, ceil(T/rows), D, N) float32.
 */
mg_status mg_selective_scan_fwd(const void *x, int64_t ldx, const void *raw, int64_t ldraw,
                                const float *A, const void *Bm, int64_t ldb, const void *Cm,
                                int64_t ldc, mg_dtype dt, const float *Dskip,
                                const float *dt_bias, int softplus, const float *h0,
                                const int64_t *cu_seqlens, int64_t nseq,
                                void *y, float *h_last, float *saved,
                                int64_t B, int64_t T, int64_t D, int64_t N, int64_t G,
                                void *ws, size_t ws_bytes, cudaStream_t stream);

/* Workspace of mg_selective_scan_fwd and _bwd for nseq sequences (0: invalid
 * or unsupported sizes). */
size_t mg_selective_scan_fwd_workspace_size(int64_t B, int64_t T, int64_t D, int64_t N, int64_t G,
                                            int64_t nseq);
size_t mg_selective_scan_bwd_workspace_size(int64_t B, int64_t T, int64_t D, int64_t N, int64_t G,
                                            int64_t nseq);

/* Bytes of `saved` (0: invalid or unsupported sizes), and the rows between
 * two of its states. */
size_t mg_selective_scan_saved_size(int64_t B, int64_t T, int64_t D, int64_t N);
int mg_selective_scan_saved_rows(void);

/*
 * Gradients for mg_selective_scan_fwd of sum(dy*y) + sum(dh_last*h_last),
 * from `saved` of a forward call on the same inputs.  With g_r the adjoint
 * of h_r:  g_r = Cm_r dy_r + a_{r+1} g_{r+1}  (+ dh_last at a sequence's last
 * row), a_r = exp(delta_r A):
 *   dCm_r[g,n] = sum_{d in g} dy_r[d] h_r[d,n]
 *   dBm_r[g,n] = sum_{d in g} g_r[d,n] delta_r[d] x_r[d]
 *   dx_r = delta_r sum_n g_r Bm_r + Dskip dy_r
 *   ddelta_r = x_r sum_n g_r Bm_r + sum_n A g_r a_r h_{r-1};  draw = ddelta sigmoid(raw + dt_bias)
 *   dA = sum_r delta_r g_r a_r h_{r-1}, dDskip = sum_r dy_r x_r, ddt_bias = sum_r draw_r
 *   dh0 = a_1 g_1 (dh_last, or 0, for an empty sequence)
 * dh_last may be NULL (zero); dDskip, ddt_bias and dh0 may be NULL (not
 * written).  dx, draw (B,T,D) and dBm, dCm (B,T,G,N) are dense, type dt; the
 * other gradients float32.  Sums over rows and channels are taken in a fixed
 * order: repeated calls give the same bits.
 */
mg_status mg_selective_scan_bwd(const void *dy, int64_t lddy, const float *saved, const void *x,
                                int64_t ldx, const void *raw, int64_t ldraw, const float *A,
                                const void *Bm, int64_t ldb, const void *Cm, int64_t ldc,
                                mg_dtype dt, const float *Dskip, const float *dt_bias,
                                int softplus, const float *h0, const float *dh_last,
                                const int64_t *cu_seqlens, int64_t nseq,
                                void *dx, void *draw, float *dA, void *dBm, void *dCm,
                                float *dDskip, float *ddt_bias, float *dh0,
                                int64_t B, int64_t T, int64_t D, int64_t N, int64_t G,
                                void *ws, size_t ws_bytes, cudaStream_t stream);

/*
 * One token: row i of x, raw (B,D), Bm, Cm (B,G,N) advances the state
 * slots[i] of state (nslots,D,N) float32 in place by one row of
 * mg_selective_scan_fwd; y (B,D), type dt.
 */
mg_status mg_selective_scan_step(const void *x, int64_t ldx, const void *raw, int64_t ldraw,
                                 const float *A, const void *Bm, int64_t ldb, const void *Cm,
                                 int64_t ldc, mg_dtype dt, const float *Dskip,
                                 const float *dt_bias, int softplus, float *state, int64_t nslots,
                                 const int64_t *slots, void *y, int64_t B, int64_t D, int64_t N,
                                 int64_t G, cudaStream_t stream);

/* How mg_group_norm_* uses z. */
typedef enum mg_gate {
    MG_GATE_NONE = 0,   /* no z                                            */
    MG_GATE_AFTER = 1,  /* the norm's output is multiplied by act(z)       */
    MG_GATE_FIRST = 2   /* x is multiplied by act(z) before the norm       */
} mg_gate;

/*
 * Group norm with an activation, channels last.  x is (M, D), each row in G
 * groups of D/G neighbouring channels, each normalised by itself (a row is a
 * token: nothing passes from one row to another).  act is silu, or the
 * identity if silu = 0.
 *   p = x act(z) for MG_GATE_FIRST, else x
 *   mean, var of p over the group (rms: mean = 0),  rstd = (var + eps)^(-1/2)
 *   o = (p - mean) rstd w + bias
 *   y = o (MG_GATE_FIRST), o act(z) (MG_GATE_AFTER), act(o) (MG_GATE_NONE)
 * w, bias (D) float32 (bias may be NULL); y dense, type dt; stats (M, G, 2)
 * float32 (may be NULL) receives mean and rstd.  Groups have at most 16384
 * channels, and M G is below 2^31.
 */
mg_status mg_group_norm_fwd(const void *x, int64_t ldx, const void *z, int64_t ldz, mg_dtype dt,
                            const float *w, const float *bias, double eps, int rms, mg_gate gate,
                            int silu, void *y, float *stats, int64_t M, int64_t D, int64_t G,
                            cudaStream_t stream);

/* Workspace of mg_group_norm_bwd (0: invalid sizes). */
size_t mg_group_norm_workspace_size(int64_t M, int64_t D, int64_t G);

/*
 * Gradients of sum(dy*y) for mg_group_norm_fwd, with stats of a forward call
 * on the same inputs: dx and dz (dense, type dt; dz for a gate only), dw and
 * dbias (float32; dbias may be NULL).  Sums over rows are taken in a fixed
 * order: repeated calls give the same bits.
 */
mg_status mg_group_norm_bwd(const void *dy, int64_t lddy, const float *stats, const void *x,
                            int64_t ldx, const void *z, int64_t ldz, mg_dtype dt, const float *w,
                            const float *bias, int rms, mg_gate gate, int silu,
                            void *dx, void *dz, float *dw, float *dbias,
                            int64_t M, int64_t D, int64_t G,
                            void *ws, size_t ws_bytes, cudaStream_t stream);

/*
 * The calls above with their arguments as an array of 64-bit words, in the
 * declared order (integers and enums sign-extended, pointers and sizes as they
 * are, eps as the bits of a double): one argument instead of up to 36 for
 * bindings that pay for each.  `nargs` is the array's length.
 */
typedef enum mg_ssm_op {
    MG_CAUSAL_CONV_FWD = 0,
    MG_CAUSAL_CONV_BWD = 1,
    MG_CAUSAL_CONV_STEP = 2,
    MG_SELECTIVE_SCAN_FWD = 3,
    MG_SELECTIVE_SCAN_BWD = 4,
    MG_SELECTIVE_SCAN_STEP = 5,
    MG_GROUP_NORM_FWD = 6,
    MG_GROUP_NORM_BWD = 7
} mg_ssm_op;
mg_status mg_ssm_call(mg_ssm_op op, const uint64_t *args, int nargs);

#ifdef __cplusplus
}
#endif

#endif /* MG_SSM_H */
