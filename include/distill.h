/*
 * distill.h — C ABI of the distillation loss for MI355X (gfx950): the loss of
 * loss.h mixed with distillation from a teacher's K best logits of each row.
 * With the teacher's columns id[j] and logits z[j] (j < K) of the row and the
 * temperature tau:
 *
 *   t[j]  = exp(z[j] / tau) / sum over the row's used entries
 *   kd    = tau^2 sum_j t[j] (log t[j] - log softmax(l / tau)[id[j]])
 *   dl[v] = ((1 - mix) d ce / d l[v]
 *            + mix tau (softmax(l / tau)[v] - sum_{j: id[j] = v} t[j])) inv_norm
 *
 * ce and its gradient as in cross_entropy.  losses [2 x S] receives ce in its
 * first S values and kd in its second; dlogits [S x V] receives the gradient
 * and may be logits itself.  An entry whose id is outside [0, V) is not used,
 * whatever its logit; one column may be named by several entries, whose
 * masses add; a row with no used entry, or none with a logit above minus
 * infinity, has kd 0 and no gradient of it.  A row whose target is outside
 * [0, V) is padding: both losses 0 and a zero gradient row.  targets may be
 * NULL when mix is 1: then every row counts and its ce is 0.
 *
 * Probabilities e^x, x <= 0 the logit's distance from the row's maximum (over
 * tau), are formed in fp32 with x log2(e) rounded once: each is off by about
 * |x| 2^-24 of itself.
 *
 * Index arrays hold int32 or int64, teacher logits fp32 or binary16.  Rows
 * of up to 65536 logits are read once when logits and dlogits lie at the same
 * offset from a 16-byte boundary (they do when one call's arrays are both
 * 16-byte aligned, or the same); others twice.  Errors as for cross_entropy,
 * with GEMM_ERR_SHAPE for K outside 0 to 1024, GEMM_ERR_DTYPE for a
 * temperature that is not positive or whose reciprocal or square is not
 * finite, a mix outside [0, 1] or a type flag that is neither 0 nor 1, and
 * GEMM_ERR_ALIAS when an output overlaps another array (dlogits == logits
 * excepted).
 */
#ifndef DISTILL_H
#define DISTILL_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct loss_distill_args {
    const float *logits;
    float *dlogits;
    const void *targets;
    const void *teacher_ids;
    const void *teacher_logits;
    float *losses;
    int64_t targets64, ids64, teacher_f16; /* 0 or 1 */
    int64_t S, V, K;
    double temperature, mix, alpha, beta, inv_norm;
} loss_distill_args;
int loss_distill_cross_entropy(const loss_distill_args *args, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* DISTILL_H */
