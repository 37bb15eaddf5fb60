/*
 * block_norm.h — C ABI of the norms around a transformer block for MI355X
 * (gfx950): the norm behind a block, its gate, the update of the residual
 * stream and the norm in front of the next block in one pass, forward and
 * backward.  They stand between the output projection of one block and the
 * first projection of the next (gemm_fwd.h).
 *
 * For every row (token) of `width` values, with norm(v, w) = v r w and
 * r = rsqrt(mean v^2 + eps):
 *
 *   n     = norm(y, post_weight)                    (y without post_weight)
 *   x_out = residual_scale x + block_scale gate n   (gate 1 without one)
 *   h     = norm(x_out, pre_weight)                 (no h without pre_weight)
 *
 * Without y (in front of the first block, behind the last) x_out is x, which
 * is not written, and h = norm(x, pre_weight).  The gate is one row of width
 * values, or one for each sequence.
 *
 * The backward pass, from the gradients dx_out (of x_out, from what reads the
 * residual stream later; none counts as zero) and dh, and from x_out and y:
 *
 *   g  = dh pre_weight, dt = dx_out + r (g - x_out r^2 mean(g x_out))
 *   dx = residual_scale dt,  u = block_scale dt,  dn = u gate
 *   g' = dn post_weight, dy = r' (g' - y r'^2 mean(g' y))   (dn without post_weight)
 *   dpre_weight = sum dh x_out r,  dpost_weight = sum dn y r'   (over rows)
 *   dgate = sum u n   (over the gate's rows)
 *
 * with r of x_out and r' of y.  Without y, dx = dt.
 *
 * Rows: with cu_seqlens, sequence b is rows cu_seqlens[b] ..
 * cu_seqlens[b + 1] - 1; rows in front of cu_seqlens[0] and from
 * cu_seqlens[num_seqs] on belong to none: what they hold takes no part, and
 * x_out, h, dx and dy are zero there.  Entries outside [0, tokens] are clamped
 * to it; with entries that decrease the results are unspecified, but no access
 * leaves the arrays.  Nothing passes between rows but the sums over them.
 *
 * Layout: [tokens, width] of fp32, given by the first element and the stride
 * of a row in elements; a row's values are contiguous, addresses multiples of
 * 4 bytes.  All device pointers are owned by the caller; a call allocates
 * nothing and only enqueues work on `stream` (a hipStream_t, NULL for the null
 * stream).  A row's sums are fp32.  The sums over rows are fp32 over at most 64
 * rows of a wave or workgroup, joined in fp32 over four waves for widths up to
 * 1024 (256 rows), and fp64 from there.  Each has a fixed order: results are
 * bitwise reproducible.
 *
 * Errors are returned synchronously, before anything is enqueued, except
 * GEMM_ERR_LAUNCH from a later one of a call's launches (the status values are
 * those of gemm_fwd.h).
 */
#ifndef BLOCK_NORM_H
#define BLOCK_NORM_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* A [tokens, width] fp32 matrix; data NULL where a call has none. */
typedef struct block_rows {
    void *data;
    int64_t row_stride;
} block_rows;

/* The sizes of a call and what all rows share. */
typedef struct block_norm_problem {
    const float *pre_weight;   /* [width], or NULL: no norm in front of the next block */
    const float *post_weight;  /* [width], or NULL: no norm behind the block */
    const float *gate;         /* [width] or [num_seqs, width], or NULL */
    int64_t gate_by_sequence;  /* 0 or 1; 1 needs cu_seqlens */
    int64_t gate_stride;       /* elements from one sequence's gate to the next; ignored otherwise */
    const int32_t *cu_seqlens; /* [num_seqs + 1] device array, or NULL: all rows are one sequence */
    int64_t num_seqs;          /* ignored when cu_seqlens is NULL */
    int64_t tokens;
    int64_t width;             /* 1 to 8192 */
    double residual_scale;     /* finite in fp32; 1 without y */
    double block_scale;        /* finite in fp32; 1 without y */
    double eps;                /* finite in fp32, not negative */
} block_norm_problem;

/*
 * x_out and h.  Each may be the very same matrix as x or y; they may not
 * overlap one another or, otherwise, anything else of the call.
 *
 * GEMM_ERR_NULL for a missing array (or neither y nor pre_weight),
 * GEMM_ERR_SHAPE for sizes outside the above (tokens < 2^30, num_seqs < 2^24),
 * for strides that are negative, overlap an output's own rows or reach 2^56
 * elements over all rows, and for arrays that the call has no use for (x_out,
 * post_weight or gate without y, h without pre_weight), GEMM_ERR_ALIGN,
 * GEMM_ERR_DTYPE for a scale, eps or flag outside the above, GEMM_ERR_ALIAS,
 * and GEMM_ERR_LAUNCH when the runtime rejects the launch.  tokens == 0
 * enqueues nothing.
 */
typedef struct block_norm_args {
    block_norm_problem p;
    block_rows x, y, x_out, h;
} block_norm_args;
int block_norm(const block_norm_args *args, void *stream);

/*
 * dx, dy (with y) and the gradients of the weights and the gate that the call
 * has, [width], [width] and the gate's shape, the latter's rows dgate_stride
 * elements apart (at least width with a gate for each of several sequences).
 * dx_out may be NULL only with pre_weight.  dx and dy may each be the very same
 * matrix as dx_out, dh, x_out or y; they may not overlap one another or,
 * otherwise, anything else.
 * The workspace holds at least block_norm_backward_workspace_bytes bytes (-1
 * for sizes the call refuses), 16-byte aligned, of any contents; calls that
 * may run at the same time need one each (GEMM_ERR_WORKSPACE when it is too
 * small).  With tokens == 0 the sums over rows are zero.
 */
typedef struct block_norm_backward_args {
    block_norm_problem p;
    block_rows dx_out, dh, x_out, y, dx, dy;
    float *dpre_weight, *dpost_weight, *dgate;
    int64_t dgate_stride;
    void *workspace;
    int64_t workspace_bytes;
} block_norm_backward_args;
int block_norm_backward(const block_norm_backward_args *args, void *stream);
int64_t block_norm_backward_workspace_bytes(const block_norm_problem *problem);

#ifdef __cplusplus
}
#endif

#endif /* BLOCK_NORM_H */
