// Attention whose scores are capped by a tanh, biased by the distance of row
// and key, or masked with a prefix that all rows see, forward and backward
// (definitions in attention.h, kernels in attention_kernels.h): the choice of
// the form, and the form with a prefix alone.

#include "attention_kernels.h"
#include "attention_scores.h"

namespace attention_scores {

int forward_prefix(const attn_scored_forward_args &a, void *stream) { return forward<kPrefix>(a, a.s, stream); }
int backward_prefix(const attn_scored_backward_args &a, void *stream) {
    return backward<kPrefix>(a, a.s, a.dslopes, stream);
}

}  // namespace attention_scores

using namespace attention_scores;

extern "C" {

int attn_scored_forward(const attn_scored_forward_args *args, void *stream) {
    if (args == nullptr) return GEMM_ERR_NULL;
    const bool cap = args->s.softcap != 0.0, bias = args->s.slopes != nullptr;
    return (cap && bias ? forward_cap_bias : cap ? forward_cap : bias ? forward_bias : forward_prefix)(*args, stream);
}

int64_t attn_scored_backward_workspace_bytes(const attn_problem *problem, int slopes_gradient) {
    if (problem == nullptr || check_problem(*problem) != GEMM_OK) return -1;
    return scratch_of(*problem, slopes_gradient != 0).bytes;
}

int attn_scored_backward(const attn_scored_backward_args *args, void *stream) {
    if (args == nullptr) return GEMM_ERR_NULL;
    const bool cap = args->s.softcap != 0.0, bias = args->s.slopes != nullptr;
    return (cap && bias ? backward_cap_bias : cap ? backward_cap : bias ? backward_bias : backward_prefix)(*args, stream);
}

}  // extern "C"
