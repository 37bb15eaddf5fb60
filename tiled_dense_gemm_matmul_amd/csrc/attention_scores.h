// The forms of attention's scores beside the plain one, each built by itself
// (they take a minute each to compile).
#ifndef ATTENTION_SCORES_H
#define ATTENTION_SCORES_H

#include "attention.h"

namespace attention_scores {

int forward_prefix(const attn_scored_forward_args &a, void *stream);
int forward_bias(const attn_scored_forward_args &a, void *stream);
int forward_cap(const attn_scored_forward_args &a, void *stream);
int forward_cap_bias(const attn_scored_forward_args &a, void *stream);
int backward_prefix(const attn_scored_backward_args &a, void *stream);
int backward_bias(const attn_scored_backward_args &a, void *stream);
int backward_cap(const attn_scored_backward_args &a, void *stream);
int backward_cap_bias(const attn_scored_backward_args &a, void *stream);

}  // namespace attention_scores

#endif  // ATTENTION_SCORES_H
