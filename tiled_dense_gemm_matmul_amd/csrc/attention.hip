// Attention over packed sequences, forward and backward (definitions in
// attention.h, kernels in attention_kernels.h).

#include "attention_kernels.h"

extern "C" {

int attn_forward(const attn_forward_args *args, void *stream) {
    return args == nullptr ? GEMM_ERR_NULL : forward<0>(*args, kPlain, stream);
}

int64_t attn_backward_workspace_bytes(const attn_problem *problem) {
    if (problem == nullptr || check_problem(*problem) != GEMM_OK) return -1;
    return scratch_of(*problem, false).bytes;
}

int attn_backward(const attn_backward_args *args, void *stream) {
    return args == nullptr ? GEMM_ERR_NULL : backward<0>(*args, kPlain, nullptr, stream);
}

}  // extern "C"
