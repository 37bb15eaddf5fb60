// Attention whose scores are capped by a tanh, with or without a prefix that
// all rows see (definitions in attention.h, kernels in attention_kernels.h).

#include "attention_kernels.h"
#include "attention_scores.h"

namespace attention_scores {

int forward_cap(const attn_scored_forward_args &a, void *stream) { return forward<kPrefix | kCap>(a, a.s, stream); }
int backward_cap(const attn_scored_backward_args &a, void *stream) {
    return backward<kPrefix | kCap>(a, a.s, a.dslopes, stream);
}

}  // namespace attention_scores
