// [tokens, heads, head_dim] tensors of attention.h: what the kernels take of
// them, and the host's checks.
#ifndef STRIDED_H
#define STRIDED_H

#include <stddef.h>
#include <stdint.h>

#include "attention.h"

namespace {

struct Strided {
    float *p;
    int64_t st, sh;
};

Strided strided(const attn_tensor &t, int64_t tokens, int64_t heads) {
    // the stride of an axis of one element is never stepped over
    return {static_cast<float *>(t.data), tokens > 1 ? t.token_stride : 0, heads > 1 ? t.head_stride : 0};
}

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

struct View {
    const attn_tensor *t;
    int64_t heads;
    bool output;
};

// Bytes from the first to behind the last element.
int64_t extent(const View &v, int64_t tokens, int64_t d) {
    return ((tokens - 1) * v.t->token_stride + (v.heads - 1) * v.t->head_stride + d) * 4;
}

// Whether two tensors may share an element.  Tensors in separate ranges do
// not; nor do views of one buffer with the same token stride whose spans
// within a token's row lie apart, or whose heads lie between one another's.
bool overlap(const View &a, const View &b, int64_t tokens, int64_t d) {
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.t->data), b0 = reinterpret_cast<uintptr_t>(b.t->data);
    if (a0 >= b0 + (uintptr_t)extent(b, tokens, d) || b0 >= a0 + (uintptr_t)extent(a, tokens, d)) return false;
    const int64_t st = a.t->token_stride * 4, sh = a.t->head_stride * 4, bytes = d * 4;
    const int64_t sa = (a.heads - 1) * sh + bytes, sb = (b.heads - 1) * b.t->head_stride * 4 + bytes;
    if (a.t->token_stride != b.t->token_stride || sa > st || sb > st) return true;
    const int64_t from_a = (int64_t)(((int64_t)(b0 - a0) % st + st) % st);  // b's place in a token's row of a
    if (from_a >= sa && from_a + sb <= st) return false;
    auto between = [&](int64_t off) {  // heads at this distance fall between the other's
        const int64_t r = (off % sh + sh) % sh;
        return r >= bytes && sh - r >= bytes;
    };
    return !(a.heads > 1 && b.heads > 1 && a.t->head_stride == b.t->head_stride && sh > 0 && between(from_a) &&
             between(from_a - st));
}

bool in_range(const View &v, const void *p, int64_t bytes, int64_t tokens, int64_t d) {
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(v.t->data), b0 = reinterpret_cast<uintptr_t>(p);
    return p != nullptr && a0 < b0 + (uintptr_t)bytes && b0 < a0 + (uintptr_t)extent(v, tokens, d);
}

struct Span {
    const void *p;
    int64_t bytes;
};
bool spans_overlap(const Span &a, const Span &b) {
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
    return a.p && b.p && a.bytes > 0 && b.bytes > 0 && a0 < b0 + (uintptr_t)b.bytes && b0 < a0 + (uintptr_t)a.bytes;
}

// The strides of an output keep its rows apart: heads inside a token's row, or
// tokens inside a head.
bool rows_apart(const View &v, int64_t tokens, int64_t d) {
    const int64_t st = v.t->token_stride, sh = v.t->head_stride;
    if (tokens > 1 && st < d) return false;
    if (v.heads <= 1) return true;
    const bool inside = sh >= d && (tokens <= 1 || st >= (v.heads - 1) * sh + d);
    return inside || sh >= (tokens - 1) * st + d;
}

bool same_tensor(const attn_tensor &a, const attn_tensor &b) {
    return a.data == b.data && a.token_stride == b.token_stride && a.head_stride == b.head_stride;
}

}  // namespace

#endif /* STRIDED_H */
