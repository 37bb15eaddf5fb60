/*
 * attention.h — C ABI of the attention kernels for MI355X (gfx950): attention
 * over packed sequences, its backward pass, and the per-head norm of queries
 * and keys with the position rotation, forward and backward.  They stand
 * between the query/key/value projection and the output projection of
 * gemm_fwd.h and take the projection's output in place, as strided views.
 *
 * Attention.  `tokens` rows hold sequences one behind the other: sequence b
 * is rows cu_seqlens[b] .. cu_seqlens[b + 1] - 1, or all rows are one
 * sequence when cu_seqlens is NULL.  Row i sees row j of its own sequence
 * when, with causal, j <= i, and, with window > 0, |i - j| < window (every
 * row sees itself).  Query head h reads key/value head h / (q_heads /
 * kv_heads).  For every row i and query head:
 *
 *   s_ij   = scale q_i . k_j                 over the visible j (or as below)
 *   lse_i  = log sum_j exp(s_ij)             (natural logarithm)
 *   out_i  = sum_j exp(s_ij - lse_i) v_j
 *
 * and the backward pass, from dout and the forward's out and lse:
 *
 *   p_ij = exp(s_ij - lse_i), delta_i = dout_i . out_i,
 *   ds_ij = p_ij (dout_i . v_j - delta_i)
 *   dq_i = scale sum_j ds_ij k_j
 *   dk_j = scale sum_{heads of the group, i} ds_ij q_i
 *   dv_j = sum_{heads of the group, i} p_ij dout_i
 *
 * Rows in front of cu_seqlens[0] and from cu_seqlens[num_seqs] on belong to
 * no sequence: what they hold takes no part, their out, dq, dk and dv are
 * zero and their lse is minus infinity.  Nothing passes between sequences, whatever
 * the rows of another one or of none hold; inside a sequence a NaN, an
 * infinity or a score of 2^30 or more in magnitude can reach all of its rows
 * (as NaN).  The backward pass forms p_ij from the score and from lse, both
 * rounded to fp32: each is off by about 2^-23 |s_ij| of itself, except where
 * one key holds all of a row's probability: that key's is 1 at any score.
 * cu_seqlens must not decrease; entries
 * outside [0, tokens] are clamped to it and a decreasing entry reads as an
 * empty sequence (the results are then unspecified, but no access leaves the
 * arrays).
 *
 * Norm and rotation.  For every token t and head, with r = rsqrt(mean_d
 * x[d]^2 + eps) over the head's head_dim values:
 *
 *   n[d] = x[d] r weight[d]
 *   (y_a, y_b) = (n_a cos - n_b sin, n_b cos + n_a sin),
 *       angle = positions[t] inv_freq[p]     for pair p < rotated / 2
 *
 * where pair p is (p, p + rotated / 2), or (2p, 2p + 1) when interleaved,
 * and y = n from `rotated` on.  With positions of several axes (the time,
 * height and width of a patch, say) pair p turns by its own axis's position,
 * angle = positions[pair_axis[p]][t] inv_freq[p].  The angle is reduced to a part of a
 * turn without loss for positions up to 2^53 in magnitude, and its sine and
 * cosine are good to fp32 relative to themselves.
 * The backward pass gives dx from dy, and the weight's gradient summed over
 * tokens and heads:
 *
 *   dn = the inverse rotation of dy, g = dn weight
 *   dx[d] = r (g[d] - x[d] r mean(g x r)), dweight[d] = sum dn[d] x[d] r
 *
 * Layout: a tensor [tokens, heads, head_dim] of fp32 is given by its first
 * element and the strides of a token and of a head in elements; a head's
 * values are contiguous.  Token strides are at least head_dim, base
 * addresses are 16-byte aligned and strides multiples of 4.  lse is
 * [q_heads, tokens], dense.  All device pointers are owned by the caller; a
 * call allocates nothing and only enqueues work on `stream` (a hipStream_t,
 * NULL for the null stream).  Every sum has a fixed order: results are
 * bitwise reproducible.
 *
 * Errors are returned synchronously, before anything is enqueued, except
 * GEMM_ERR_LAUNCH from a later one of a call's launches (the status values are
 * those of gemm_fwd.h).
 */
#ifndef ATTENTION_H
#define ATTENTION_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* A [tokens, heads, head_dim] fp32 tensor: strides in elements. */
typedef struct attn_tensor {
    void *data;
    int64_t token_stride;
    int64_t head_stride;
} attn_tensor;

/* The sizes and the mask of an attention call.  The tiles of all heads,
 * q_heads (tokens / 16 + num_seqs) or fewer, number less than 2^31
 * (GEMM_ERR_SHAPE), those of q_heads and kv_heads together in the backward
 * pass. */
typedef struct attn_problem {
    const int32_t *cu_seqlens; /* [num_seqs + 1] device array, or NULL: one sequence of all tokens */
    int64_t num_seqs;          /* ignored when cu_seqlens is NULL; tokens / num_seqs, empty sequences
                                  included, is what the host takes for their length when it deals out
                                  the work (speed only) */
    int64_t tokens;
    int64_t q_heads;
    int64_t kv_heads;          /* divides q_heads */
    int64_t head_dim;          /* a multiple of 4, 4 to 128 */
    int64_t causal;            /* 0 or 1 */
    int64_t window;            /* 0: none */
    double scale;              /* positive, scale log2(e) finite in fp32 (up to 2.35e38) */
} attn_problem;

/*
 * out and lse from q, k, v.  out may be the very same tensor as q; it may
 * not overlap q otherwise, nor k, v, lse or cu_seqlens, and lse overlaps no
 * other array of the call.
 *
 * GEMM_ERR_NULL for a missing array, GEMM_ERR_SHAPE for sizes outside the
 * above (tokens < 2^30 - 64, heads <= 65535, num_seqs < 2^24) or strides that are
 * too small, overlap an output's own elements or reach 2^22 elements from one
 * token to the next, GEMM_ERR_ALIGN, GEMM_ERR_DTYPE for a scale outside the
 * above or a causal that is neither 0 nor 1, GEMM_ERR_ALIAS,
 * and GEMM_ERR_LAUNCH when the runtime rejects the launch.  tokens == 0
 * enqueues nothing.
 */
typedef struct attn_forward_args {
    attn_problem p;
    attn_tensor q, k, v, out;
    float *lse;
} attn_forward_args;
int attn_forward(const attn_forward_args *args, void *stream);

/*
 * dq, dk, dv from dout, q, k, v and the forward's out and lse.  No output may
 * overlap another array of the call (views of one buffer whose elements do
 * not overlap are fine).  The workspace holds at least
 * attn_backward_workspace_bytes bytes (0 for small problems, -1 for ones the
 * call refuses), 4-byte aligned, of any contents; calls that may run at the
 * same time need one each (GEMM_ERR_WORKSPACE when it is too small).
 */
typedef struct attn_backward_args {
    attn_problem p;
    attn_tensor dout, q, k, v, out;
    const float *lse;
    attn_tensor dq, dk, dv;
    void *workspace;
    int64_t workspace_bytes;
} attn_backward_args;
int64_t attn_backward_workspace_bytes(const attn_problem *problem);
int attn_backward(const attn_backward_args *args, void *stream);

/*
 * Scores of other forms, in any combination (attn_scored_*):
 *
 *   s_ij = softcap tanh(scale q_i . k_j / softcap) - slopes[h] |i - j|
 *
 * for query head h, and with prefix_lens row i sees, beside the keys j <= i,
 * the first prefix_lens[b] keys of its sequence b (entries below 0 and past
 * the sequence's length are clamped), less than `window` away as ever.  The
 * backward pass is that of the final scores,
 *
 *   dslopes[h] = - sum_{i,j} ds_ij |i - j|,
 *
 * with ds_ij (1 - tanh^2) in the place of ds_ij in dq and dk.  Distances are
 * fp32, slopes finite (others spread NaN over their head).  A key whose final
 * score is below -2^30, as a bias by far distances makes it, has probability
 * zero; a row's largest final score is less than 2^30 in magnitude, as above.
 */
typedef struct attn_scores {
    double softcap;             /* 0: none; 1e-6 to 1e6, with scale / softcap normal in fp32 */
    const float *slopes;        /* [q_heads], or NULL */
    const int32_t *prefix_lens; /* [num_seqs] ([1] without cu_seqlens) device array, or NULL; only with causal */
} attn_scores;

/* As attn_forward; out and lse overlap neither slopes nor prefix_lens.
 * GEMM_ERR_DTYPE also for a softcap outside the above or prefix_lens without
 * causal. */
typedef struct attn_scored_forward_args {
    attn_problem p;
    attn_scores s;
    attn_tensor q, k, v, out;
    float *lse;
} attn_scored_forward_args;
int attn_scored_forward(const attn_scored_forward_args *args, void *stream);

/* As attn_backward, and dslopes [q_heads], or NULL where it is not wanted
 * (GEMM_ERR_NULL for dslopes without slopes); it may not overlap another array
 * of the call, and with tokens == 0 it is zero.  With dslopes the workspace is
 * 8-byte aligned, and its size is the one for a slopes_gradient other than 0. */
typedef struct attn_scored_backward_args {
    attn_problem p;
    attn_scores s;
    attn_tensor dout, q, k, v, out;
    const float *lse;
    attn_tensor dq, dk, dv;
    float *dslopes;
    void *workspace;
    int64_t workspace_bytes;
} attn_scored_backward_args;
int64_t attn_scored_backward_workspace_bytes(const attn_problem *problem, int slopes_gradient);
int attn_scored_backward(const attn_scored_backward_args *args, void *stream);

/* The sizes of a norm and rotation and what all rows share. */
typedef struct attn_norm {
    const void *positions;     /* [tokens] int32 or int64, any values */
    int64_t positions64;       /* 0: int32, 1: int64 */
    const float *inv_freq;     /* [rotated / 2] */
    const float *q_weight;     /* [head_dim] */
    const float *k_weight;     /* [head_dim] */
    int64_t tokens;
    int64_t q_heads;
    int64_t k_heads;
    int64_t head_dim;          /* even, 2 to 256 */
    int64_t rotated;           /* even, 0 to head_dim */
    int64_t interleaved;       /* 0 or 1 */
    double eps;                /* finite, not negative */
} attn_norm;

/*
 * q_out and k_out from q and k; each may be the very same tensor as its
 * input, and may not overlap anything else of the call.  Any strides and
 * 4-byte alignment; 16-byte accesses where bases and strides are multiples
 * of 16 bytes, head_dim is a multiple of 8 and, unless interleaved,
 * rotated / 2 and (head_dim - rotated) / 2 are multiples of 4.  tokens == 0
 * enqueues nothing.
 *
 * GEMM_ERR_SHAPE for sizes outside the above (tokens < 2^30, heads <= 65535)
 * or an output whose rows overlap, GEMM_ERR_DTYPE for a flag that is neither
 * 0 nor 1 or a bad eps, GEMM_ERR_NULL, GEMM_ERR_ALIGN, GEMM_ERR_ALIAS and
 * GEMM_ERR_LAUNCH as above.
 */
typedef struct attn_qk_norm_rope_args {
    attn_norm n;
    attn_tensor q, k, q_out, k_out;
} attn_qk_norm_rope_args;
int attn_qk_norm_rope(const attn_qk_norm_rope_args *args, void *stream);

/* Positions of several axes: n.positions is [axes, tokens], dense. */
typedef struct attn_axes {
    const int32_t *pair_axis;  /* [rotated / 2] device array; entries outside [0, axes) are clamped to it */
    int64_t axes;              /* 1 to 65535 */
} attn_axes;

/* The same by positions of several axes. */
typedef struct attn_qk_norm_rope_axes_args {
    attn_norm n;
    attn_axes x;
    attn_tensor q, k, q_out, k_out;
} attn_qk_norm_rope_axes_args;
int attn_qk_norm_rope_axes(const attn_qk_norm_rope_axes_args *args, void *stream);

/*
 * dq, dk and the weights' gradients [head_dim] from dq_out, dk_out, q and k.
 * dq may be the very same tensor as dq_out or q, dk as dk_out or k.  The
 * workspace holds at least attn_qk_norm_rope_workspace_bytes bytes (-1 for
 * sizes the call refuses), 8-byte aligned, of any contents; calls that may
 * run at the same time need one each (GEMM_ERR_WORKSPACE when it is too
 * small).  With tokens == 0 the weights' gradients are zero.
 */
typedef struct attn_qk_norm_rope_backward_args {
    attn_norm n;
    attn_tensor dq_out, dk_out, q, k, dq, dk;
    float *dq_weight, *dk_weight;
    void *workspace;
    int64_t workspace_bytes;
} attn_qk_norm_rope_backward_args;
int attn_qk_norm_rope_backward(const attn_qk_norm_rope_backward_args *args, void *stream);
int64_t attn_qk_norm_rope_workspace_bytes(int64_t tokens, int64_t head_dim);

/* The same by positions of several axes. */
typedef struct attn_qk_norm_rope_axes_backward_args {
    attn_norm n;
    attn_axes x;
    attn_tensor dq_out, dk_out, q, k, dq, dk;
    float *dq_weight, *dk_weight;
    void *workspace;
    int64_t workspace_bytes;
} attn_qk_norm_rope_axes_backward_args;
int attn_qk_norm_rope_axes_backward(const attn_qk_norm_rope_axes_backward_args *args, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* ATTENTION_H */
