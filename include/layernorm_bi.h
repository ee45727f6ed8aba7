/*
 * layernorm_bi.h - batch-invariant layer norm (forward, backward, parameter
 * gradients) and dropout from a counter-based generator, for GB300 (sm_103a).
 * The layout descriptor, plan, error codes, status bits and conventions are
 * those of rmsnorm_bi.h.
 *
 * The operations, for every active physical row holding logical row g, with
 * hidden size H, weight w and bias c:
 *     mean_g = mean_h(x_gh),  rstd_g = 1 / sqrt(mean_h((x_gh - mean_g)^2) + eps)
 *     xhat = (x - mean) * rstd,  y = xhat * w + c
 *     a = dy * w,  dx = rstd * (a - mean_h(a) - xhat * mean_h(a * xhat))
 *     dweight_h = sum over active logical rows of dy_gh * xhat_gh   (FP32)
 *     dbias_h   = sum over active logical rows of dy_gh             (FP32)
 * and dropout with probability p:
 *     drop(x)_gh = keep_gh ? x_gh * 65536 / (65536 - t) : 0,  t = rint(65536 p)
 *     keep_gh = u_gh >= t
 * where u_gh is the 16-bit half number h % 8 (low half of word 0 first) of the
 * four words of Philox4x32-10 (Salmon, Moraes, Dror and Shaw, "Parallel random
 * numbers: as easy as 1, 2, 3", SC 2011) with key = seed (low word first) and
 * counter = (h / 8, g, offset low word, offset high word).  The mask is never
 * stored: whoever has the seed and the offset has it again, so dropout's
 * backward pass is the same function of dy.  p acts in steps of 2^-16 (below
 * 2^-17 nothing is dropped).
 *
 * The row in the counter is the call's own logical row, tok_id * rows_per_token
 * + head.  Ranks that number their rows locally therefore draw the SAME masks
 * from one state, each those of rows 0, 1, 2, ...: give such ranks different
 * seeds or offsets.  For one device's masks on several ranks, give the calls
 * with a dropout the rows' global ids (they need no plan, and ids are not
 * compared with n_logical_tokens there), and take the parameter gradients from
 * layernorm_bwd under local ids, with dx NULL.
 *
 * The guarantee.  y, dx, dweight, dbias and the mask are bitwise identical for
 * the same logical token multiset whatever its physical layout.  Row sums use
 * a fixed tree that depends only on H and the element type.  The parameter
 * gradients sum per-logical-row FP32 terms in canonical logical order: groups
 * of 8 logical rows from the first to the last, the groups of a 64-row block
 * from the first to the last, then the pairwise tree with odd carry over the
 * blocks (dweight_combine's tree).  Groups that a call holds only partly spill
 * their rows to the workspace and are summed by layernorm_finalize in the same
 * order.  Inactive rows are neither read nor written.
 *
 * Element types.  x, y, h, dy, dx and their like have one type per call
 * (`dtype`); weight and bias have that type or FP32 (`param_dtype`).  Sums,
 * statistics and parameter gradients are FP32; each output element is rounded
 * to its type once.  A dropped element is +0 whatever it was (NaN included).
 *
 * Lost copies.  Rows of more than 512 columns wait for asynchronous copies, at
 * most about one second each; a wait that runs out ends the CTA with the rest of
 * its rows unwritten.  With a workspace RMSNORM_STATUS_TIMEOUT is set.  Calls
 * without one (forward, dx alone) have no device-side report, of this or
 * anything else: their outputs then keep what was there.
 *
 * Supported hidden sizes: multiples of 8 up to 16384 for 16-bit types, up to
 * 8192 for FP32; dropout alone: multiples of 8 up to 2^20.  Data pointers are
 * 16-byte aligned, mean, rstd, the ids and the plan to 4 bytes; layout->token_stride
 * is a multiple of 8.
 */
#ifndef LAYERNORM_BI_H
#define LAYERNORM_BI_H

#include "rmsnorm_bi.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types (dtype, param_dtype). */
enum { LAYERNORM_BF16 = 0, LAYERNORM_FP16 = 1, LAYERNORM_FP32 = 2 };

/*
 * Dropout of one call.  state: DEVICE pointer to two 64-bit words, seed and
 * offset, read when the kernel runs (so a captured graph that is replayed
 * after they changed draws a new mask).  Two calls that must not share a mask
 * differ in seed or offset.  0 <= p <= 1; p = 1 drops everything.
 */
typedef struct rmsnorm_dropout {
    const uint64_t *state;
    double p;
} rmsnorm_dropout_t;

/*
 * Forward.  weight and bias may be NULL (1 and 0).  mean, rstd: optional FP32
 * [n_tokens * rows_per_token], written for active rows only.  y may alias x.
 */
int layernorm_fwd(const void *x, const void *weight, const void *bias, int64_t hidden, float eps,
                  int32_t dtype, int32_t param_dtype, const rmsnorm_layout_t *layout, void *y, float *mean,
                  float *rstd, rmsnorm_stream_t stream);

/*
 * Dropout and residual add fused with the norm: h = round(drop(x) + residual)
 * is written to h_out, and y is layernorm_fwd's of h (so the fused call equals
 * add then norm bit for bit).  dropout may be NULL (h = round(x + residual)).
 * h_out and y may alias x or residual, h_out != y.
 */
int layernorm_add_fwd(const void *x, const void *residual, const void *weight, const void *bias, int64_t hidden,
                      float eps, int32_t dtype, int32_t param_dtype, const rmsnorm_layout_t *layout,
                      const rmsnorm_dropout_t *dropout, void *h_out, void *y, float *mean, float *rstd,
                      rmsnorm_stream_t stream);

/*
 * Backward: dx on every active row (mean and rstd recomputed bitwise as in the
 * forward).  With a workspace the same pass contributes this call's rows to
 * dweight and dbias (layout->plan required); dx may then be NULL, as for a
 * call of no slots.  dx may alias dy or x.
 */
int layernorm_bwd(const void *x, const void *weight, const void *dy, int64_t hidden, float eps, int32_t dtype,
                  int32_t param_dtype, const rmsnorm_layout_t *layout, void *dx, void *workspace,
                  rmsnorm_stream_t stream);

/*
 * Backward of layernorm_add_fwd; h is its h_out.  With dn the norm's dx of h,
 *     dh = round(grad_scale * dn + dres)        (the residual's gradient)
 *     dx = round(drop(grad_scale * dn + dres))  (x's gradient, one rounding)
 * dres may be NULL.  dx is written only with a dropout (without one it equals
 * dh) and must then be non-NULL.  grad_scale is the loss seed's factor as in
 * rmsnorm_add_bwd; the workspace's terms stay unscaled (layernorm_finalize
 * takes the factor).  dh may be NULL only with a workspace and neither dres
 * nor dropout, or for a call of no slots (n_tokens == 0), whose data pointers
 * are not looked at.  dh and dx may alias dy, dres or h, dh != dx.
 */
int layernorm_add_bwd(const void *h, const void *weight, const void *dy, const void *dres, int64_t hidden,
                      float eps, float grad_scale, int32_t dtype, int32_t param_dtype,
                      const rmsnorm_layout_t *layout, const rmsnorm_dropout_t *dropout, void *dh, void *dx,
                      void *workspace, rmsnorm_stream_t stream);

/*
 * Workspace of one reduction of dweight and dbias over n_logical_rows rows of
 * width hidden: header with the status word, a state byte per 8-row group, a
 * flag per row, the group or block partials of both gradients, scratch of the
 * final tree, and a dense FP32 spill area for rows of cut groups.  Returns 0
 * for unsupported sizes.  begin, any number of contributions that hold every
 * logical row exactly once in all, finalize: as rmsnorm_dweight_begin and
 * dweight_finalize_scaled.  finalize multiplies both roots once by grad_scale
 * and may be repeated; dweight or dbias may be NULL (not both).
 * n_logical_rows == 0 gives +0.0.
 */
size_t layernorm_workspace_bytes(int64_t n_logical_rows, int64_t hidden);
int layernorm_begin(void *workspace, size_t bytes, int64_t n_logical_rows, int64_t hidden,
                    rmsnorm_stream_t stream);
int layernorm_finalize(void *workspace, int64_t n_logical_rows, int64_t hidden, float grad_scale, float *dweight,
                       float *dbias, rmsnorm_stream_t stream);

/* Synchronises `stream` and copies the workspace's status word to *status. */
int layernorm_status(const void *workspace, rmsnorm_stream_t stream, int32_t *status);

/*
 * Dropout alone: y = round(drop(x)) on every active row, dx = round(drop(dy)).
 * In place is allowed.  The plan is not used.
 */
int dropout_fwd(const void *x, int64_t hidden, int32_t dtype, const rmsnorm_layout_t *layout,
                const rmsnorm_dropout_t *dropout, void *y, rmsnorm_stream_t stream);
int dropout_bwd(const void *dy, int64_t hidden, int32_t dtype, const rmsnorm_layout_t *layout,
                const rmsnorm_dropout_t *dropout, void *dx, rmsnorm_stream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* LAYERNORM_BI_H */
