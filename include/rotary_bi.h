/*
 * rotary_bi.h - rotary positions of queries and keys, alone and behind an RMS
 * norm of every head, forward and backward, for GB300 (sm_103a).  The layout
 * descriptor, error codes, status bits and conventions are those of
 * rmsnorm_bi.h, the element types those of layernorm_bi.h.
 *
 * The operations, for every head x (D columns) of an active token slot at
 * position p, with the rotated columns in r / 2 pairs (a_i, b_i):
 *     half:         a_i = first + i,   b_i = first + r/2 + i
 *     interleaved:  a_i = first + 2i,  b_i = first + 2i + 1
 *     theta_i = p * frequency_i,  c_i = scale * cos(theta_i),  s_i = scale * sin(theta_i)
 *     rot(x):   y_a = x_a c - x_b s,   y_b = x_b c + x_a s   (other columns unchanged)
 *     rot'(g):  z_a = g_a c + g_b s,   z_b = g_b c - g_a s   (its transpose)
 * and, behind the norm with weight w,
 *     rstd = 1 / sqrt(mean(x^2) + eps),  xhat = x * rstd,  y = rot(xhat * w)
 *     g = rot'(dy),  a = g * w,  dx = rstd * (a - xhat * mean(a * xhat))
 *     dweight_h = sum over active tokens and heads of g_h * xhat_h   (FP32)
 * The angle is formed from the position itself, as the fraction of a turn in
 * 64-bit fixed point (position times the turns per position, modulo one turn),
 * so it is as exact at position 2^31 - 1 as at 0 and needs no table.  Negative
 * positions turn backwards (for instance to move cached keys by a distance).
 *
 * The guarantee.  Every output is bitwise identical for the same logical token
 * multiset whatever its physical layout (and whatever the strides).  Row sums
 * use a fixed tree that depends only on D and the rotary parameters.  A weight
 * gradient is summed in canonical order: a token's heads, queries then keys, in
 * chunks of equal size (at most 16 heads, by the sizes; the last one shorter),
 * each from its first to its last head of the kind; the logical tokens of a
 * group (2 to 10, by the sizes) in a fixed order; then chunks and groups by a
 * fixed tree over their number.  Groups that a call does not hold whole and in
 * consecutive slots leave their tokens' sums in the workspace, and
 * qk_norm_finalize adds them in the same order.  No plan is
 * needed.  Inactive slots are neither read nor written.
 *
 * Element types.  All tensors of a call have one type, weights that type or
 * FP32.  Sums, angles and weight gradients are FP32 or wider; each output
 * element is rounded to its type once.  rotary_fwd and rotary_bwd copy the
 * columns outside the rotation bit for bit.
 *
 * Supported sizes: head_dim a multiple of 8, 8 .. 512; rotary_dim a multiple of
 * 4, 4 .. head_dim; first even, first + rotary_dim <= head_dim; 1 .. 65535
 * heads a tensor; n_tokens * (heads of both tensors) < 2^31.
 */
#ifndef ROTARY_BI_H
#define ROTARY_BI_H

#include "layernorm_bi.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * The rotation of a call.  position: DEVICE int32, one per token slot (any value
 * in padding).  turns: DEVICE array (16-byte aligned) of rotary_dim / 2 words, the
 * turns per position of pair i in units of 2^-64 turn (rotary_turns).  scale multiplies
 * cos and sin (1 unless a long-context scaling asks for another factor).
 */
typedef struct rmsnorm_rotary {
    const int32_t *position;
    const uint64_t *turns;
    int32_t rotary_dim;
    int32_t first;               /* first rotated column of a head */
    int32_t interleaved;         /* 0: halves, 1: neighbouring columns */
    float scale;
} rmsnorm_rotary_t;

/*
 * The heads of one tensor (queries or keys) in a call.  Head h of token slot t
 * starts at element t * token_stride + h * head_stride of its tensor, so slices
 * of a joined projection and head-major tensors need no copy.  Data pointers are
 * 16-byte aligned (FP32: 32) and strides multiples of 8 and not negative; strides of inputs
 * may be 0 (one head or token read by all), outputs may not overlap themselves.
 * A stride that is never taken (one slot, one head) is not looked at.  out may
 * be `in` or `dy` with that tensor's strides (other overlaps are not allowed).
 */
typedef struct rmsnorm_heads {
    const void *in;              /* x; in rotary_bwd the gradient of y */
    int64_t in_token, in_head;
    const void *dy;              /* qk_norm_rotary_bwd: the gradient of y; else not used */
    int64_t dy_token, dy_head;
    void *out;                   /* y; in the backward passes dx */
    int64_t out_token, out_head;
    const void *weight;          /* [head_dim], NULL = 1; not used without the norm */
    int32_t heads;
    int32_t reserved0;           /* must be 0 */
} rmsnorm_heads_t;

/*
 * Host function: turns[i] = frequency[i] / (2 pi) in units of 2^-64 turn, modulo
 * one turn, rounded to nearest from the double's exact value.  frequency is in
 * radians per position, finite and of magnitude below 2^31; negative values turn
 * the other way.  RMSNORM_ERR_VALUE otherwise.  The array is then copied to the
 * device by the caller.
 */
int rotary_turns(const double *frequency, int32_t n, uint64_t *turns);

/*
 * rotary_fwd: out = rot(in); rotary_bwd: out = rot'(in), for the queries q and
 * the keys k of a call in one launch.  k may be NULL (one tensor).  layout:
 * rows_per_token must be 1; token_stride and the plan are not used.
 */
int rotary_fwd(const rmsnorm_heads_t *q, const rmsnorm_heads_t *k, int64_t head_dim, int32_t dtype,
               const rmsnorm_layout_t *layout, const rmsnorm_rotary_t *rotary, rmsnorm_stream_t stream);
int rotary_bwd(const rmsnorm_heads_t *q, const rmsnorm_heads_t *k, int64_t head_dim, int32_t dtype,
               const rmsnorm_layout_t *layout, const rmsnorm_rotary_t *rotary, rmsnorm_stream_t stream);

/*
 * qk_norm_rotary_fwd: out = rot(xhat * weight) of every head.
 * qk_norm_rotary_bwd: out = dx from the saved x (`in`) and dy; with a workspace
 * the same pass adds the call's tokens to both weight gradients.
 */
int qk_norm_rotary_fwd(const rmsnorm_heads_t *q, const rmsnorm_heads_t *k, int64_t head_dim, float eps, int32_t dtype,
                       int32_t param_dtype, const rmsnorm_layout_t *layout, const rmsnorm_rotary_t *rotary,
                       rmsnorm_stream_t stream);
int qk_norm_rotary_bwd(const rmsnorm_heads_t *q, const rmsnorm_heads_t *k, int64_t head_dim, float eps, int32_t dtype,
                       int32_t param_dtype, const rmsnorm_layout_t *layout, const rmsnorm_rotary_t *rotary,
                       void *workspace, rmsnorm_stream_t stream);

/*
 * Workspace of one reduction of the weight gradients of q_heads query heads and
 * k_heads key heads (0 without keys) over n_logical_tokens tokens: header with
 * the status word, a flag per token, the groups' partial sums, and a dense area
 * for the sums of tokens of cut groups.  0 for unsupported sizes.  begin, any
 * number of qk_norm_rotary_bwd calls that hold every token exactly once in all,
 * finalize.  finalize multiplies both roots once by grad_scale and may be
 * repeated; dq_weight or dk_weight may be NULL (not both; dk_weight without keys
 * must be), and they may not overlap.  Status bits: RMSNORM_STATUS_DOUBLE / _MISSING tokens, _HEADER for a
 * workspace begun for other sizes (or a call with other head counts; it then
 * contributes nothing), _PLAN for an id that is not below n_logical_tokens (its
 * dx is written, its contribution dropped).
 */
size_t qk_norm_workspace_bytes(int64_t n_logical_tokens, int32_t q_heads, int32_t k_heads, int64_t head_dim);
int qk_norm_begin(void *workspace, size_t bytes, int64_t n_logical_tokens, int32_t q_heads, int32_t k_heads,
                  int64_t head_dim, rmsnorm_stream_t stream);
int qk_norm_finalize(void *workspace, int64_t n_logical_tokens, int32_t q_heads, int32_t k_heads, int64_t head_dim,
                     float grad_scale, float *dq_weight, float *dk_weight, rmsnorm_stream_t stream);

/* Synchronises `stream` and copies the workspace's status word to *status. */
int qk_norm_status(const void *workspace, rmsnorm_stream_t stream, int32_t *status);

#ifdef __cplusplus
}
#endif
#endif /* ROTARY_BI_H */
