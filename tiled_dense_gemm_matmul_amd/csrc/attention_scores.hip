// Attention whose scores are capped by a tanh, biased by the distance of row
// and key, or masked with a prefix that all rows see, forward and backward
// (definitions in attention.h, kernels in attention_kernels.h).

#include "attention_kernels.h"

extern "C" {

int attn_scored_forward(const attn_scored_forward_args *args, void *stream) {
    return args == nullptr ? GEMM_ERR_NULL : forward<true>(*args, args->s, stream);
}

int64_t attn_scored_backward_workspace_bytes(const attn_problem *problem, int slopes_gradient) {
    if (problem == nullptr || check_problem(*problem) != GEMM_OK) return -1;
    return scratch_of<true>(*problem, slopes_gradient != 0).bytes;
}

int attn_scored_backward(const attn_scored_backward_args *args, void *stream) {
    return args == nullptr ? GEMM_ERR_NULL : backward<true>(*args, args->s, args->dslopes, stream);
}

}  // extern "C"
