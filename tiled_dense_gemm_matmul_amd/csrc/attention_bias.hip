// Attention whose scores are biased by the distance of row and key, with or
// without a prefix that all rows see (definitions in attention.h, kernels in
// attention_kernels.h).

#include "attention_kernels.h"
#include "attention_scores.h"

namespace attention_scores {

int forward_bias(const attn_scored_forward_args &a, void *stream) { return forward<kPrefix | kBias>(a, a.s, stream); }
int backward_bias(const attn_scored_backward_args &a, void *stream) {
    return backward<kPrefix | kBias>(a, a.s, a.dslopes, stream);
}

}  // namespace attention_scores
