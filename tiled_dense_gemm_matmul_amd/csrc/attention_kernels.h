// Attention over packed sequences for MI355X (gfx950), forward and backward,
// in fp32 on v_mfma_f32_16x16x4_f32 (definitions in attention.h).
//
// The work is bound by the fp32 matrix instructions: 4 D flops a visible
// (row, key) pair and head forward, and 14 D backward, where the scores and
// the products with dout are formed twice, once for dq with the rows held
// fixed and once for dk and dv with the keys held fixed.  (Forming them once
// is 10 D flops, but then dq or dk and dv would be summed by atomics, whose
// order changes results, or kept as [tokens, tokens] arrays.)
//
//  * A wave holds 16 or 32 rows (or keys) in registers and walks over blocks
//    of 16 of the other side, whose operands it loads from memory straight
//    into the registers that the MFMA reads, each under one product or more
//    before its own (a load of 4 KiB takes place of 32 to 64 MFMAs' 1024 to
//    2048 cycles).  Only the backward pass over heads of up to 64 takes
//    operands through LDS, where it turns them for their second product.
//  * The probabilities never leave the registers either.  A 16 x 16 product
//    leaves lane (g, m) = (lane / 16, lane % 16) with its rows 4g .. 4g + 3
//    of column m.  That is the B operand of the next product when its
//    contraction step i takes row 4g + i from lane group g, so the scores are
//    formed with the side that is contracted next as their rows: keys for
//    out and dq, query rows for dk and dv.
//  * The other operand of that product is read along the head: lane (g, m)
//    takes the 4 consecutive values 64c + 4m .. + 3 of row 4g + i with one
//    16-byte load, which serve as row m of four MFMA tiles.  Result tile
//    4c + e then holds dimension 64c + 4m + e in its row m, so a lane ends up
//    with 16 consecutive values of a row's result.
//  * Loads are buffer loads whose descriptor starts at the block's first row
//    and ends at its last row in the sequence, so rows past it and head
//    values past head_dim read as zeros, and offsets stay small however long
//    the buffer is.
//
// A workgroup owns a tile of rows of one sequence and one head.  Either its
// waves own rows of their own (WS = 1), or all of them own the same rows, take
// every WS-th block of the other side and are joined through LDS in order
// (WS = 4).
//
// fp32 MFMAs and vector instructions do not overlap on a SIMD, so beside the
// MFMAs' 32 cycles each the exponentials (16 cycles for a 16 x 4 block of
// scores) and the few other instructions a score takes are what is left: at
// 4096 rows, 16 heads of 64 the forward pass runs at 130 TFLOP/s, 85% of the
// rate of a large fp32 product on this card, with the MFMAs busy 83% of the
// time.
//
// The same kernels serve every form of scores: FORM 0 is plain, kPrefix the
// mask with a prefix, kBias the bias by distance and kCap the cap, the latter
// two with or without a prefix.  They only change what is between the two
// products of a block.  The form is a template argument because each of these
// steps behind a branch made the compiler copy a block's scores from register
// to register: 16 x 512 tokens, 12 heads of 64, backward, prefixes of no rows,
// took 256 us that way and 230 as FORM 0.
#ifndef ATTENTION_KERNELS_H
#define ATTENTION_KERNELS_H

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <algorithm>
#include <cmath>

#include "attention.h"
#include "gemm_fwd.h"
#include "launch.h"
#include "strided.h"

namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int u32x4v __attribute__((vector_size(16)));
typedef unsigned int u32x2v __attribute__((vector_size(8)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __amdgpu_buffer_rsrc_t Rsrc;

constexpr int kPrefix = 1, kBias = 2, kCap = 4;  // bits of FORM

constexpr int kOOB = (int)0x80000000u;  // past every descriptor's end (they end below 2^31)
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;
// The running maximum of a row that has seen no key yet: low enough that any
// score replaces it, finite so that differences with it are not NaN.
constexpr float kNoMax = -3.0e38f;
// The same with a bias, which pushes keys below any score: -2^30 log2(e), the
// least score that is served.  Keys below it never become the reference and
// add exp2 of a large negative number, which is zero.  (As a reference, rounded
// to fp32, such a key was off by up to half an ulp of its score from the
// exponent that it was taken from, 128 from 2^30 on: its exponential and the
// sums were infinite, and NaN once they were rescaled by zero.)
constexpr float kNoBiasedMax = -0x1p30f * kLog2e;

struct Problem {
    const int *cu;
    int nseq, tokens, hq, group, d, causal, window;
    int first;       // workgroups in front of this launch's
    float scale, c;  // c = scale log2(e): scores go through exp2
    float factor;    // of dq and dk: the call's scale
    const int *prefix;  // [nseq], or NULL
    float bend;         // kCap: the raw scores are tanh(bend q.k), and scale is the cap
    float times;        // kBias: of the raw scores, before the bias; scale is 1
};

// A row's lse from the sum of exp2(s c - top) over its raw scores s and the
// largest of them, most: the largest score, rounded to fp32 once, plus the
// logarithm of the sum relative to that score.  Where one key holds all of
// the probability the second part is next to nothing, so lse is that score to
// the bit and the backward pass gets 1 back however large the score is.
// (Taken as (top + log2(sum)) ln 2, it came back an ulp or two of the score
// away: probabilities were off by up to 14% at scores of 2^20 and by up to a
// factor of 2^96 at 2^29.)
__device__ __forceinline__ float lse_of(const Problem &p, float sum, float top, float most) {
#pragma clang fp contract(off)  // the largest score's rounding is the backward pass's
    const float score = most * p.scale;
    const float rest = (__builtin_amdgcn_logf(sum) - fmaf(most, p.c, -top)) * kLn2;
    return score + rest;
}
// The probability of a raw score in the backward pass.  The score is rounded
// as in lse_of before lse is taken from it: two instructions a score more than
// one multiply-add with scale log2(e).
template <int FORM>
__device__ __forceinline__ float probability(const Problem &p, float s, float lse) {
#pragma clang fp contract(off)
    const float score = FORM & kBias ? s : s * p.scale;
    return __builtin_amdgcn_exp2f((score - lse) * kLog2e);
}

// tanh(x) for |x| up to kSmall is x times a polynomial in x^2 (a minimax fit,
// off by a quarter of fp32's rounding).  A block of scores that all lie in
// there, as most do under a cap of a few times their size, takes no
// exponential; in others the rest of the scores take (1 - e) / (1 + e) with e =
// exp(-2 |x|), off by at most 8 roundings from there on: 3.4 from e (its
// argument's two and the instruction's ulp, at 0.5 and less further out), two
// from the sums, three from the reciprocal and the product.
constexpr float kSmall = 0.5f;
__device__ __forceinline__ float small_tanh(float x) {
    const float y = x * x;
    const float f = fmaf(fmaf(fmaf(0.0172414780429774f, y, -0.053045488615601204f), y, 0.13325878887208747f), y,
                         -0.33333143893843536f);
    return x * fmaf(f, y, 1.0f);
}

// a where mask is -1, b where it is 0, without a branch over a's exponential.
__device__ __forceinline__ float choose(int mask, float a, float b) {
    return __builtin_bit_cast(float, (__builtin_bit_cast(int, a) & mask) | (__builtin_bit_cast(int, b) & ~mask));
}

// Bends the 16 x 16 blocks s of q.k by the cap, 7 instructions a score, and
// takes the bias from them, 3 (without a bias the cap stays a factor for the
// exponent to take in).  A lane holds keys (or rows) at the distances |away[b]
// - i| from its row (or key); `steep` gets the derivative 1 - tanh^2.  Both
// passes take the same steps, so their scores agree to the bit.  (A bias in
// units of the raw scores took one instruction less, but rounded the slopes:
// that moves all of a head's scores one way, and the slopes' gradient, which
// sums over them, came out up to twice as far off.)
template <int FORM, int RB, bool GRAD>
__device__ __forceinline__ void bend_scores(float bend, float times, float slope, const float (&away)[RB], f32x4 (&s)[RB],
                                            f32x4 (&steep)[RB]) {
#pragma clang fp contract(off)
    if constexpr (FORM & kCap) {
        float most = 0.0f;
#pragma unroll
        for (int b = 0; b < RB; ++b) {
            s[b] *= bend;
#pragma unroll
            for (int i = 0; i < 4; ++i) most = fmaxf(most, fabsf(s[b][i]));
        }
        if (!__any(most > kSmall)) {
#pragma unroll
            for (int b = 0; b < RB; ++b)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float t = small_tanh(s[b][i]);
                    s[b][i] = t;
                    if (GRAD) steep[b][i] = fmaf(-t, t, 1.0f);
                }
        } else {
#pragma unroll
            for (int b = 0; b < RB; ++b) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float x = s[b][i];
                    // an unknown value from here on, or both sides would be
                    // computed for every block and one of them chosen
                    asm volatile("" : "+v"(x));
                    const float t = small_tanh(x);
                    const float e = __builtin_amdgcn_exp2f(fabsf(x) * (-2.0f * kLog2e));
                    const float r = __builtin_amdgcn_rcpf(1.0f + e);
                    const int far = fabsf(x) > kSmall ? -1 : 0;
                    s[b][i] = choose(far, copysignf((1.0f - e) * r, x), t);
                    if (GRAD) steep[b][i] = choose(far, 4.0f * e * r * r, fmaf(-t, t, 1.0f));
                    if (i % 2) __builtin_amdgcn_sched_barrier(0);  // two scores' temporaries at a time
                }
            }
        }
    }
    if constexpr (FORM & kBias) {
#pragma unroll
        for (int b = 0; b < RB; ++b)
#pragma unroll
            for (int i = 0; i < 4; ++i) s[b][i] = fmaf(-slope, fabsf(away[b] - (float)i), s[b][i] * times);
    }
}
// What no kernel of a call writes, for scalar loads at uniform places.
template <class T>
using Constant = const __attribute__((address_space(4))) T *;
__device__ __forceinline__ float slope_of(const float *slopes, int h) { return ((Constant<float>)slopes)[h]; }

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// Rows [row, end) of a head, at most 16 of them, as a buffer.
__device__ __forceinline__ Rsrc rows_rsrc(const float *base, int64_t st, int row, int end, int d) {
    const int n = min(end - row, 16);
    const int bytes = n > 0 ? (int)(((n - 1) * st + d) * 4) : 0;
    return __builtin_amdgcn_make_buffer_rsrc((void *)(base + row * st), (short)0, bytes, 0x00020000);
}

__device__ __forceinline__ f32x4 load4(Rsrc r, int off) {
    return __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0));
}
__device__ __forceinline__ f32x2 load2(Rsrc r, int off) {
    return __builtin_bit_cast(f32x2, __builtin_amdgcn_raw_buffer_load_b64(r, off, 0, 0));
}
__device__ __forceinline__ void store4(Rsrc r, int off, f32x4 v) {
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4v, v), r, off, 0, 0);
}
__device__ __forceinline__ f32x4 mfma(float a, float b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0);
}

// Between a wave's writes of staged rows and its reads of them by other lanes,
// and the other way round.  A wave's LDS accesses complete in the order they
// are issued, so this only keeps the compiler from moving LDS accesses across
// (a fence of all memory also holds back the loads in flight and cost up to
// 2.8%: 16 x 512 rows backward, 229 against 236 us).  The verification build
// waits in full; the results are compared bit for bit.
__device__ __forceinline__ void staged_order() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
#ifdef GEMM_SYNC_CHECK
    __builtin_amdgcn_s_waitcnt(0);
#endif
}

// 16 rows of a head with lane (g, m) holding values 16j + 4g .. + 3 of row m:
// the A or B operand of a product contracted along the head.
template <int DP>
struct Rows {
    static constexpr int NJ = DP / 16;
    f32x4 x[NJ];

    // byte offset of this lane's first value; col(j) past head_dim is out of range
    template <bool EX>
    __device__ __forceinline__ void load(Rsrc r, int64_t st, int d) {
        const int lane = threadIdx.x & 63, g = lane >> 4, m = lane & 15;
        const int at = m * (int)st * 4 + g * 16;
#pragma unroll
        for (int j = 0; j < NJ; ++j) x[j] = load4(r, (EX || 16 * j + 4 * g < d) ? at + 64 * j : kOOB);
    }
    // Lays the rows out in LDS, DP + 4 values apart: the 16 lanes that write or
    // read together then meet 64 different banks, along a row or across.
    __device__ __forceinline__ void stage(float *to) const {
        staged_order();
        const int lane = threadIdx.x & 63, g = lane >> 4, m = lane & 15;
#pragma unroll
        for (int j = 0; j < NJ; ++j) *(f32x4 *)(to + m * (DP + 4) + 16 * j + 4 * g) = x[j];
    }
};

// 16 rows of a head with lane (g, m) holding, of rows 4g + i, the values that
// are row m of the MFMA tiles: 4 of them for each 64 of the head, 2 for a
// last 32.  The A operand of a product contracted over the rows.
template <int DP>
struct Cols {
    static constexpr int N4 = DP / 64, N2 = DP % 64 / 32;
    f32x4 x[4][N4 > 0 ? N4 : 1];
    f32x2 y[4];

    template <bool EX>
    __device__ __forceinline__ void load(Rsrc r, int64_t st, int d) {
        const int lane = threadIdx.x & 63, g = lane >> 4, m = lane & 15;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int row = (4 * g + i) * (int)st * 4;
#pragma unroll
            for (int c = 0; c < N4; ++c) x[i][c] = load4(r, (EX || 64 * c + 4 * m < d) ? row + 256 * c + 16 * m : kOOB);
            if (N2) y[i] = load2(r, (EX || 64 * N4 + 2 * m < d) ? row + 256 * N4 + 8 * m : kOOB);
        }
    }
    // the same from a wave's staged rows (Rows::stage)
    __device__ __forceinline__ void take(const float *staged) {
        staged_order();
        const int lane = threadIdx.x & 63, g = lane >> 4, m = lane & 15;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float *row = staged + (4 * g + i) * (DP + 4);
#pragma unroll
            for (int c = 0; c < N4; ++c) x[i][c] = *(const f32x4 *)(row + 64 * c + 4 * m);
            if (N2) y[i] = *(const f32x2 *)(row + 64 * N4 + 2 * m);
        }
    }
    // the value of row 4g + i that belongs to MFMA tile t
    __device__ __forceinline__ float at(int i, int t) const { return t < 4 * N4 ? x[i][t / 4][t % 4] : y[i][t % 2]; }
};

// The transposed result of 16 rows, [dimension, row], in DP / 16 MFMA tiles.
template <int DP>
struct Acc {
    static constexpr int NT = DP / 16, N4 = DP / 64, N2 = DP % 64 / 32;
    f32x4 t[NT];

    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < NT; ++i) t[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }
    __device__ __forceinline__ void mul(float f) {
#pragma unroll
        for (int i = 0; i < NT; ++i) t[i] *= f;
    }
    // += cols^T p, one row of p a register
    __device__ __forceinline__ void add(const Cols<DP> &a, f32x4 p) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < NT; ++j) t[j] = mfma(a.at(i, j), p[i], t[j]);
    }
    // Calls f(first dimension, 4 consecutive values) for all of the lane's
    // values of row m.
    template <class F>
    __device__ __forceinline__ void each4(F f) const {
        const int g = (threadIdx.x & 63) >> 4;
#pragma unroll
        for (int c = 0; c < N4; ++c)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                f(64 * c + 16 * g + 4 * i, f32x4{t[4 * c][i], t[4 * c + 1][i], t[4 * c + 2][i], t[4 * c + 3][i]});
        if (N2) {
#pragma unroll
            for (int i = 0; i < 4; i += 2)
                f(64 * N4 + 8 * g + 2 * i, f32x4{t[NT - 2][i], t[NT - 1][i], t[NT - 2][i + 1], t[NT - 1][i + 1]});
        }
    }
};

// [rows of a, rows of b] scores: += a b^T.
template <int DP>
__device__ __forceinline__ f32x4 dots(const Rows<DP> &a, const Rows<DP> &b) {
    f32x4 s = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int j = 0; j < DP / 16; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) s = mfma(a.x[j][e], b.x[j][e], s);
    return s;
}

// The same products as four sums of DP / 4, added in pairs: a partial sum
// that is rounded at every step is half as large, over a quarter of the steps.
// For scores with a bias (3 instructions a score): the slopes' gradient sums
// ds_ij |i - j| over a head, terms of both signs that all but cancel, and is
// off by the scores' roundings more than by all others together.  Over 240
// drawn problems its error was 1.04 to 1.10 of an elementary torch
// implementation's with single sums, 0.62 to 0.66 with four (geometric means of
// two halves).  Single sums and four, us: 16 x 512 tokens, 12 heads of 64,
// forward 81.2 and 82.2, backward 258 and 257; 6144, 12 heads on 4, 489 and 504,
// 1575 and 1606; 4 x 2048, 16 heads on 4 of 128, 588 and 598, 2145 and 2215.
template <int DP>
__device__ __forceinline__ f32x4 split_dots(const Rows<DP> &a, const Rows<DP> &b) {
    f32x4 s[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        s[c] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int i = c * DP / 16; i < (c + 1) * DP / 16; ++i) s[c] = mfma(a.x[i / 4][i % 4], b.x[i / 4][i % 4], s[c]);
    }
    return (s[0] + s[1]) + (s[2] + s[3]);
}
template <int DP, int FORM>
__device__ __forceinline__ f32x4 scores(const Rows<DP> &a, const Rows<DP> &b) {
    if constexpr (FORM & kBias) return split_dots<DP>(a, b);
    else return dots<DP>(a, b);
}

// A value of the four lane groups (lanes of one m) combined in all of them.
// Swapping a register's odd rows of 16 lanes with a copy's even rows, and its
// upper half with a copy's lower half, leaves each lane's partner's value
// beside its own, without a trip through LDS.
template <class F>
__device__ __forceinline__ float across_groups(float v, F f) {
    unsigned u = __builtin_bit_cast(unsigned, v);
    const auto a = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    v = f(__builtin_bit_cast(float, (unsigned)a[0]), __builtin_bit_cast(float, (unsigned)a[1]));
    u = __builtin_bit_cast(unsigned, v);
    const auto b = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    return f(__builtin_bit_cast(float, (unsigned)b[0]), __builtin_bit_cast(float, (unsigned)b[1]));
}
__device__ __forceinline__ float group_sum(float v) {
    return across_groups(v, [](float x, float y) { return x + y; });
}
__device__ __forceinline__ float group_max(float v) {
    return across_groups(v, [](float x, float y) { return fmaxf(x, y); });
}

// Sum over the wave's lanes up to each one, itself included: shifts within
// rows of 16 lanes, then broadcasts into the next rows.
__device__ __forceinline__ int lanes_scan(int v) {
    v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, true);   // row_shr:1
    v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, true);   // row_shr:2
    v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, true);   // row_shr:4
    v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, true);   // row_shr:8
    v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false);  // row_bcast:15 into rows 1 and 3
    v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false);  // row_bcast:31 into rows 2 and 3
    return v;
}
// Sum over all of them, the same in every lane.
__device__ __forceinline__ int lanes_sum(int v) { return __builtin_amdgcn_readlane(lanes_scan(v), 63); }

// What a workgroup finds in cu_seqlens for its x-th tile of TILE rows, each
// sequence being cut into tiles by itself: the sequence [s0, s1) and the
// tile's first row r0 (none when r0 < 0), and the rows [first, last) that
// belong to sequences.  Bounds are clamped to the buffer.
//
// The tiles that take longest come first, over all sequences (of the next
// 64).  In causal attention those are, with `back`, a sequence's last tiles,
// whose rows see most keys, else its first, whose keys the most rows see: tile
// n - 1 - l or l of a sequence of n tiles has level l, work grows with the
// level, and S(l) = sum over sequences of max(0, n - l) tiles have level l or
// more, so x's level is the largest l with S(l) > x.  Otherwise all tiles of a
// sequence take as long as it is, and S(l) = sum of n over sequences with n >
// l counts the tiles of those.  (Sequence by sequence, a long tile of the
// last sequence starts when the chip is nearly done: dk and dv of 4 x 2048
// rows, 2 heads of 128, took 910 us in a launch of their own; without a causal
// mask, six documents of 1 to 1531 rows took 686 us by level, 560 by length.)
//
// A prefix of G tiles (PREFIX) makes its tiles alike: G tiles of rows see at
// least its keys and have level G - 1, or G tiles of keys are seen by all rows
// and have level n - 1; the others keep theirs, and the tiles of one level are
// found by a sum over the lanes.  (With the levels of a plain causal mask, the
// last tiles to start were those of the longest prefixes: 7 documents of 1 to
// 4096 tokens, a third of them prefixes, 16 heads on 4 of 128, forward, took
// 1119 us, and take 1001.)
//
// That search looks at every sequence, 64 at a time, in every workgroup, which
// with 2^24 sequences would take hours.  Past kScanned of them sequence b,
// which starts at row c, has the numbers from c / TILE + b on, of which there
// are enough up to the next sequence's, and b is found by a search in which
// the wave looks at 64 bounds at once: two looks up to 4096 sequences, four up
// to 2^24.  The tiles then come in the order of the sequences (12 heads of 64,
// sequences of 100 rows, forward and backward: 200 of them 72 and 268 us by
// level against 78 and 288, 400 of them 161 and 553 against 163 and 572, 1000
// of them 430 and 1517 against 392 and 1409).
constexpr int kScanned = 512;
struct Tile {
    int s0, s1, r0, first, last, seq;
};
template <int TILE, bool PREFIX>
__device__ __forceinline__ Tile find_tile(const Problem &p, int x, bool back) {
    Tile t = {0, p.tokens, -1, 0, p.tokens, 0};
    int n = 0, level = 0;
    if (p.nseq == 1) {
        if (p.cu) {
            t.first = t.s0 = min(max(uniform(p.cu[0]), 0), p.tokens);
            t.last = t.s1 = max(t.s0, min(uniform(p.cu[1]), p.tokens));
        }
        n = (t.s1 - t.s0 + TILE - 1) / TILE;
        if (x >= n) return t;
        level = n - 1 - x;
    } else if (p.nseq > kScanned) {
        const int lane = threadIdx.x & 63;
        const int c0 = p.cu[0], c1 = p.cu[p.nseq];
        auto bound = [&](int b) { return min(max(p.cu[b], 0), p.tokens); };
        int lo = 0, hi = p.nseq, step;
        do {  // of [lo, hi), the last sequence whose first number is x or less
            step = (hi - lo + 63) / 64;
            const int b = lo + lane * step;
            const int below = __popcll(__ballot(b < hi && bound(min(b, hi)) / TILE + b <= x));
            lo += max(below - 1, 0) * step;
            hi = min(lo + step, hi);
        } while (step > 1);
        t.first = min(max(uniform(c0), 0), p.tokens);
        t.last = max(t.first, min(uniform(c1), p.tokens));
        t.seq = lo = uniform(lo);
        t.s0 = uniform(bound(lo));
        t.s1 = max(t.s0, min(uniform(p.cu[lo + 1]), p.tokens));
        n = (t.s1 - t.s0 + TILE - 1) / TILE;
        const int at = x - (t.s0 / TILE + lo);
        if (at < 0 || at >= n) return t;
        level = n - 1 - at;
    } else {
        const int lane = threadIdx.x & 63;
        const int c0 = p.cu[0], c1 = p.cu[p.nseq];
        bool found = false;
        for (int b = 0; b < p.nseq; b += 64) {
            const int c = p.cu[min(b + lane, p.nseq)], d = p.cu[min(b + lane + 1, p.nseq)];
            const int lo = min(max(c, 0), p.tokens), hi = max(lo, min(d, p.tokens));
            const int mine = (hi - lo + TILE - 1) / TILE;
            const int total = lanes_sum(mine);
            if (x >= total) {
                x -= total;
                continue;
            }
            int alike = 1;  // tiles of the prefix
            if (PREFIX && p.prefix)
                alike = max(1, (min(p.prefix[min(b + lane, p.nseq - 1)], hi - lo) + TILE - 1) / TILE);
            auto own_from = [&](int l) {  // the lane's sequence's part of S(l)
                if (!p.causal) return mine > l ? mine : 0;
                if (PREFIX && l < (back ? alike : mine)) return back ? mine : max(mine - l, alike);
                return max(0, mine - l);
            };
            auto tiles_from = [&](int l) { return lanes_sum(own_from(l)); };  // S(l)
            for (int bit = 1 << (31 - __builtin_clz(total)); bit > 0; bit >>= 1) {
                if (!__any(mine > level + bit)) continue;
                if (tiles_from(level + bit) > x) level += bit;
            }
            x -= tiles_from(level + 1);
            int at;
            if (PREFIX && p.prefix) {
                const int here = own_from(level) - own_from(level + 1), sum = lanes_scan(here);
                at = __builtin_ctzll(__ballot(sum > x));
                const int rank = x - __builtin_amdgcn_readlane(sum - here, at);
                const int n_at = __builtin_amdgcn_readlane(mine, at);
                if (level == (back ? __builtin_amdgcn_readlane(alike, at) : n_at) - 1) level = back ? rank : n_at - 1 - rank;
            } else {
                const int each = p.causal ? 1 : level + 1;  // tiles of a sequence in a row
                const bool has = p.causal ? mine > level : mine == level + 1;
                const uint64_t all = __ballot(has);
                const int rank =
                    __builtin_amdgcn_mbcnt_hi((unsigned)(all >> 32), __builtin_amdgcn_mbcnt_lo((unsigned)all, 0));
                at = __builtin_ctzll(__ballot(has && rank == x / each));
                if (!p.causal) level = x % each;
            }
            t.seq = b + at;
            t.s0 = __builtin_amdgcn_readlane(lo, at);
            t.s1 = __builtin_amdgcn_readlane(hi, at);
            n = __builtin_amdgcn_readlane(mine, at);
            found = true;
            break;
        }
        t.first = min(max(uniform(c0), 0), p.tokens);
        t.last = max(t.first, min(uniform(c1), p.tokens));
        if (!found) return t;
    }
    t.r0 = t.s0 + (back ? level : n - 1 - level) * TILE;
    return t;
}

// The head and tile of a workgroup.  Tiles come head by head, the longest
// tiles of every head first, so that what is left at the end is short.
// Workgroups reach the 8 XCDs, each with its own L2, in turn; the heads of a
// step are ordered by the key/value head they read, so that with 4 or 8 of
// those (or a multiple) an XCD meets the same one or two throughout.
__device__ __forceinline__ void head_and_tile(int id, int heads, int group, int &h, int &x) {
    x = id / heads;
    const int slot = id - x * heads, shared = heads / group;
    const int turn = slot / shared;
    h = (slot - turn * shared) * group + turn;
}

// Calls f for this workgroup's share of the rows that belong to no sequence:
// rows [x TILE, x TILE + TILE) in front of the first sequence or behind the last.
template <int TILE, class F>
__device__ __forceinline__ void outside_rows(const Problem &p, const Tile &t, int x, F f) {
    const int64_t a = (int64_t)x * TILE;
    if (a >= p.tokens) return;
    const int b = (int)min(a + TILE, (int64_t)p.tokens);
    if (a >= t.first && b <= t.last) return;
    for (int r = (int)a + (int)(threadIdx.x >> 6); r < b; r += blockDim.x >> 6)
        if (r < t.first || r >= t.last) f(r);
}
__device__ __forceinline__ void zero_row(float *row, int d) {
    for (int i = threadIdx.x & 63; i < d; i += 64) row[i] = 0.0f;
}

// The keys that rows [r, r + n) of a sequence may see, and the rows that may
// see keys [k, k + n): ranges inside the sequence.
struct Range {
    int lo, hi;
};
// The row behind the prefix of a tile's sequence, whose keys all of its rows see.
template <bool PREFIX>
__device__ __forceinline__ int prefix_end(const Problem &p, const Tile &t) {
    return PREFIX && p.prefix ? t.s0 + min(max(((Constant<int>)p.prefix)[t.seq], 0), t.s1 - t.s0) : t.s0;
}
template <bool PREFIX>
__device__ __forceinline__ Range keys_of(const Problem &p, int s0, int s1, int pe, int r, int n) {
    const int last = min(r + n, s1) - 1;
    Range k = {s0, s1};
    if (p.window) {
        k.lo = max(s0, r - p.window + 1);
        if (s1 - last > p.window) k.hi = last + p.window;
    }
    if (p.causal) k.hi = PREFIX ? min(k.hi, max(last + 1, pe)) : last + 1;
    return k;
}
template <bool PREFIX>
__device__ __forceinline__ Range rows_of(const Problem &p, int s0, int s1, int pe, int k, int n) {
    const int last = min(k + n, s1) - 1;
    Range r = {s0, s1};
    if (p.window) {
        r.lo = max(s0, k - p.window + 1);
        if (s1 - last > p.window) r.hi = last + p.window;
    }
    if (p.causal && !(PREFIX && k < pe)) r.lo = k;
    return r;
}
__device__ __forceinline__ bool inside(Range r, int x) { return (unsigned)(x - r.lo) < (unsigned)(r.hi - r.lo); }
// Whether rows [r, r + n) of the sequence all see keys [k, k + m), both whole inside it.
template <bool PREFIX>
__device__ __forceinline__ bool all_see(const Problem &p, int s1, int pe, int r, int n, int k, int m) {
    if (r + n > s1 || k + m > s1) return false;
    if (p.causal && k + m - 1 > (PREFIX ? max(r, pe - 1) : r)) return false;
    return !p.window || ((int64_t)r + n - 1 - k < p.window && (int64_t)k + m - 1 - r < p.window);
}

// --- forward ---
//
// Online softmax over blocks of 16 keys.  The reference value of a row is
// moved, and the sums rescaled, only when a score exceeds it by 2^8: the
// probabilities then stay below 2^8 of the reference, which fp32 holds
// without loss, and most blocks need neither the maximum across lanes nor
// the rescaling.
//
// Four waves a SIMD leave each 128 registers, which two blocks of rows of
// heads of 64 fill; the cap's and the bias's steps spill some of the loads'
// offsets then, and loading these again waits for the keys in flight.  Those
// kernels run three waves (12 heads of 64, us with three and with four: cap 50,
// 16 x 512 tokens 79.6 and 85.5, 64 x 128 tokens 28.3 and 35.2; biases 81.3 and
// 118, 28.6 and 46.1).
template <int DP, bool EX, int RB, int WS, int FORM>
__global__ __launch_bounds__(256, DP > 64 ? 2 : DP == 64 && RB == 2 && FORM > kPrefix ? 3 : 4) void attention_fwd(Problem p, Strided q, Strided k, Strided v, Strided o,
                                                        float *lse, const float *slopes) {
    constexpr int WROWS = 16 * RB, WR = 4 / WS, TILE = WR * WROWS;
    const int lane = threadIdx.x & 63, g = lane >> 4, m = lane & 15;
    const int wave = uniform(threadIdx.x >> 6);
    int h, x;
    head_and_tile(p.first + (int)blockIdx.x, p.hq, p.group, h, x);
    const Tile t = find_tile<TILE, FORM != 0>(p, x, p.causal);
    outside_rows<TILE>(p, t, x, [&](int r) {
        zero_row(o.p + r * o.st + h * o.sh, p.d);
        if (lane == 0) lse[(int64_t)h * p.tokens + r] = -INFINITY;
    });
    if (t.r0 < 0) return;
    const int s0 = t.s0, s1 = t.s1, pe = prefix_end<FORM != 0>(p, t);
    const int part_of = wave / WR, r0 = t.r0 + wave % WR * WROWS;
    if (WS == 1 && r0 >= s1) return;
    const float *kp = k.p + (h / p.group) * k.sh, *vp = v.p + (h / p.group) * v.sh;

    Rows<DP> Q[RB];
    Acc<DP> O[RB];
    float top[RB], sum[RB], largest[RB];  // the reference in units of log 2, the sum, the largest raw score
#pragma unroll
    for (int b = 0; b < RB; ++b) {
        Q[b].template load<EX>(rows_rsrc(q.p + h * q.sh, q.st, r0 + 16 * b, s1, p.d), q.st, p.d);
        O[b].clear();
        top[b] = FORM & kBias ? kNoBiasedMax : kNoMax;
        sum[b] = 0.0f;
        largest[b] = -INFINITY;
    }
    const Range kr = keys_of<FORM != 0>(p, s0, s1, pe, r0, WROWS);
    const int step = 16 * WS;
    int kb = kr.lo + 16 * part_of;
    const float slope = FORM & kBias ? slope_of(slopes, h) : 0.0f;
    // The values of a block are asked for when its scores begin, the keys of
    // the next one when they are done, so each load has a product to arrive under.
    Rows<DP> K;
    Cols<DP> V;
    K.template load<EX>(rows_rsrc(kp, k.st, kb, s1, p.d), k.st, p.d);
    for (; kb < kr.hi; kb += step) {
        f32x4 s[RB];
        V.template load<EX>(rows_rsrc(vp, v.st, kb, s1, p.d), v.st, p.d);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int b = 0; b < RB; ++b) s[b] = scores<DP, FORM>(K, Q[b]);
        __builtin_amdgcn_sched_barrier(0);
        K.template load<EX>(rows_rsrc(kp, k.st, kb + step, s1, p.d), k.st, p.d);
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (FORM & (kBias | kCap)) {
            float away[RB];
            f32x4 steep[RB];
#pragma unroll
            for (int b = 0; b < RB; ++b) away[b] = (float)(r0 + 16 * b + m - kb - 4 * g);
            bend_scores<FORM, RB, false>(p.bend, p.times, slope, away, s, steep);
        }
        if (!all_see<FORM != 0>(p, s1, pe, r0, WROWS, kb, 16)) {
#pragma unroll
            for (int b = 0; b < RB; ++b) {
                const Range seen = keys_of<FORM != 0>(p, s0, s1, pe, r0 + 16 * b + m, 1);
#pragma unroll
                for (int i = 0; i < 4; ++i) s[b][i] = inside(seen, kb + 4 * g + i) ? s[b][i] : -INFINITY;
            }
        }
#pragma unroll
        for (int b = 0; b < RB; ++b) {
            largest[b] = fmaxf(fmaxf(fmaxf(fmaxf(largest[b], s[b][0]), s[b][1]), s[b][2]), s[b][3]);
            const float most = largest[b] * p.c;  // once the reference has moved, no longer above it
            if (__any(most > top[b] + 8.0f)) {
                const float to = fmaxf(top[b], group_max(most));
                const float f = __builtin_amdgcn_exp2f(top[b] - to);
                top[b] = to;
                sum[b] *= f;
                O[b].mul(f);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                s[b][i] = __builtin_amdgcn_exp2f(fmaf(s[b][i], p.c, -top[b]));
                sum[b] += s[b][i];
            }
            O[b].add(V, s[b]);
        }
    }
#pragma unroll
    for (int b = 0; b < RB; ++b) {
        sum[b] = group_sum(sum[b]);
        largest[b] = group_max(largest[b]);
    }

    if (WS == 1) {
#pragma unroll
        for (int b = 0; b < RB; ++b) {
            const int r = r0 + 16 * b;
            if (r >= s1) break;
            const Rsrc ro = rows_rsrc(o.p + h * o.sh, o.st, r, s1, p.d);
            const float inv = 1.0f / sum[b];
            O[b].each4([&](int d0, f32x4 y) {
                store4(ro, (EX || d0 < p.d) ? m * (int)o.st * 4 + d0 * 4 : kOOB, y * inv);
            });
            if (g == 0 && r + m < s1)
                lse[(int64_t)h * p.tokens + r + m] = lse_of(p, sum[b], top[b], largest[b]);
        }
    } else {
        // join the waves of the same rows, in order, 16 rows at a time
        constexpr int LD = DP + 4;
        __shared__ __align__(16) float part[WS == 1 ? 1 : 4][WS == 1 ? 1 : 16 * LD];
        __shared__ float ptop[4][16], psum[4][16], plargest[4][16];
        const int mine = wave % WR, e = threadIdx.x & 15;
#pragma unroll
        for (int b = 0; b < RB; ++b) {
            if (b > 0) __syncthreads();
            O[b].each4([&](int d0, f32x4 y) { *(f32x4 *)&part[wave][m * LD + d0] = y; });
            if (g == 0) {
                ptop[wave][m] = top[b];
                psum[wave][m] = sum[b];
                plargest[wave][m] = largest[b];
            }
            __syncthreads();
            for (int row = part_of * 4 + g; row < 16; row += 4 * WS) {
                const int r = r0 + 16 * b + row;
                if (r >= s1) continue;
                float to = ptop[mine][row], most = plargest[mine][row], total = 0.0f, f[WS];
#pragma unroll
                for (int w = 1; w < WS; ++w) {
                    to = fmaxf(to, ptop[w * WR + mine][row]);
                    most = fmaxf(most, plargest[w * WR + mine][row]);
                }
#pragma unroll
                for (int w = 0; w < WS; ++w) {
                    f[w] = __builtin_amdgcn_exp2f(ptop[w * WR + mine][row] - to);
                    total += f[w] * psum[w * WR + mine][row];
                }
                const float inv = 1.0f / total;
                float *dst = o.p + (int64_t)r * o.st + h * o.sh;
#pragma unroll
                for (int c = 0; c < (DP + 63) / 64; ++c) {
                    const int d0 = 64 * c + 4 * e;
                    if (d0 < p.d) {
                        f32x4 y = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                        for (int w = 0; w < WS; ++w) y += f[w] * *(const f32x4 *)&part[w * WR + mine][row * LD + d0];
                        *(f32x4 *)(dst + d0) = y * inv;
                    }
                }
                if (e == 0) lse[(int64_t)h * p.tokens + r] = lse_of(p, total, to, most);
            }
        }
    }
}

// Adds the results of 16 rows of the WS waves that share them, in order,
// times f, into rows [r, s1) of a head.  `part` holds 4 x 16 x (DP + 4) floats.
template <int DP, int WS>
__device__ __forceinline__ void join_rows(const Acc<DP> &acc, float *part, const Strided &to, int h, int r, int s1,
                                          int d, float f) {
    constexpr int LD = DP + 4, WR = 4 / WS;
    const int wave = threadIdx.x >> 6, g = (threadIdx.x & 63) >> 4, m = threadIdx.x & 15;
    __syncthreads();  // the buffer's last readers
    acc.each4([&](int d0, f32x4 y) { *(f32x4 *)&part[(wave * 16 + m) * LD + d0] = y; });
    __syncthreads();
    const int mine = wave % WR, e = threadIdx.x & 15;
    for (int row = wave / WR * 4 + g; row < 16; row += 4 * WS) {
        if (r + row >= s1) continue;
        float *dst = to.p + (int64_t)(r + row) * to.st + h * to.sh;
#pragma unroll
        for (int c = 0; c < (DP + 63) / 64; ++c) {
            const int d0 = 64 * c + 4 * e;
            if (d0 < d) {
                f32x4 y = *(const f32x4 *)&part[(mine * 16 + row) * LD + d0];
#pragma unroll
                for (int w = 1; w < WS; ++w) y += *(const f32x4 *)&part[((w * WR + mine) * 16 + row) * LD + d0];
                *(f32x4 *)(dst + d0) = y * f;
            }
        }
    }
}

// --- backward ---
//
// One launch forms all three: the first workgroups dk and dv of a tile of
// keys, the rest dq of a tile of rows, longest tiles first in both, so that
// the shorter dq tiles fill what the others leave of the chip.
//
// The slopes (kBias) come as [hq], or NULL, and the sums for their gradient go to
// slope_parts, [hq, tiles of rows, 4 waves], or NULL.
//
// delta = dout . out of every row is needed by both parts.  A kernel in front
// writes it to memory once, or, where a launch counts for more, each part
// forms it for itself (OWN), which costs the walk over rows a quarter more
// loads.
//
// Keys, queries and dout are needed both along the rows and across them.
// Heads of up to 64 are loaded once and turned in LDS, in a space of each
// wave's own (no barrier); with one block a wave the turned rows are read a
// product ahead of their own (EARLY), with two there are no registers for it.
// Wider heads are loaded twice, which was faster for them (8 heads of 128,
// 4096 rows: 1011 us against 1024; 12 heads of 64, 512 rows: 27.7 us loaded
// twice against 25.5).
constexpr int kStagedWidth = 64;

struct Backward {
    Strided dout, q, k, v, o, dq, dk, dv;
    const float *lse, *delta;
};

// dout . out of 16 rows: row m's in lanes (g, m).
template <int DP>
__device__ __forceinline__ float row_dots(const Rows<DP> &a, const Rows<DP> &b) {
    f32x4 dot = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int j = 0; j < DP / 16; ++j) dot += a.x[j] * b.x[j];
    return group_sum((dot[0] + dot[1]) + (dot[2] + dot[3]));
}

// delta [heads, tokens]: 16 lanes a row, which take the head's values in
// 16-byte pieces.
__global__ __launch_bounds__(256) void attention_delta(Problem p, Strided dout, Strided o, float *delta, int64_t first) {
    const int e = threadIdx.x & 15;
    const int64_t row = (first + blockIdx.x) * 16 + (threadIdx.x >> 4);
    if (row >= (int64_t)p.hq * p.tokens) return;
    const int t = (int)(row / p.hq), h = (int)(row - (int64_t)t * p.hq);
    const float *x = dout.p + t * dout.st + h * dout.sh, *y = o.p + t * o.st + h * o.sh;
    float sum = 0.0f;
    for (int d = 4 * e; d < p.d; d += 64) {
        const f32x4 u = *(const f32x4 *)(x + d) * *(const f32x4 *)(y + d);
        sum += (u[0] + u[1]) + (u[2] + u[3]);
    }
#pragma unroll
    for (int i = 1; i < 16; i <<= 1) sum += __shfl_xor(sum, i, 64);
    if (e == 0) delta[(int64_t)h * p.tokens + t] = sum;
}

template <int DP, bool EX, int RB, int WS, bool OWN, int FORM>
__device__ __forceinline__ void backward_dq(const Problem &p, const Backward &a, int id, float *shared, int tiles,
                                            const float *slopes, double *slope_parts) {
    const Strided &dout = a.dout, &q = a.q, &k = a.k, &v = a.v, &o = a.o, &dq = a.dq;
    const float *lse = a.lse;
    constexpr int WROWS = 16 * RB, WR = 4 / WS, TILE = WR * WROWS;
    const int lane = threadIdx.x & 63, g = lane >> 4, m = lane & 15;
    const int wave = uniform(threadIdx.x >> 6);
    int h, x;
    head_and_tile(id, p.hq, p.group, h, x);
    const Tile t = find_tile<TILE, FORM != 0>(p, x, p.causal);
    outside_rows<TILE>(p, t, x, [&](int r) { zero_row(dq.p + r * dq.st + h * dq.sh, p.d); });
    double *slope_part = (FORM & kBias) && slope_parts ? slope_parts + ((int64_t)h * tiles + x) * 4 + wave : nullptr;
    if ((FORM & kBias) && slope_part && lane == 0) *slope_part = 0.0;
    if (t.r0 < 0) return;
    const int s0 = t.s0, s1 = t.s1, t0 = t.r0, pe = prefix_end<FORM != 0>(p, t);
    const int part_of = wave / WR, r0 = t0 + wave % WR * WROWS;
    if (WS == 1 && r0 >= s1) return;
    const float slope = FORM & kBias ? slope_of(slopes, h) : 0.0f;
    double slope_sum = 0.0;
    const float *kp = k.p + (h / p.group) * k.sh, *vp = v.p + (h / p.group) * v.sh;

    Rows<DP> Q[RB], G[RB];
    Acc<DP> A[RB];
    float l[RB], del[RB];
#pragma unroll
    for (int b = 0; b < RB; ++b) {
        const int r = r0 + 16 * b;
        Q[b].template load<EX>(rows_rsrc(q.p + h * q.sh, q.st, r, s1, p.d), q.st, p.d);
        G[b].template load<EX>(rows_rsrc(dout.p + h * dout.sh, dout.st, r, s1, p.d), dout.st, p.d);
        const int64_t at = (int64_t)h * p.tokens + r + m;
        if (OWN) {
            Rows<DP> out;
            out.template load<EX>(rows_rsrc(o.p + h * o.sh, o.st, r, s1, p.d), o.st, p.d);
            del[b] = row_dots<DP>(G[b], out);
        } else {
            del[b] = r + m < s1 ? a.delta[at] : 0.0f;
        }
        l[b] = r + m < s1 ? lse[at] : 0.0f;
        A[b].clear();
    }
    const Range kr = keys_of<FORM != 0>(p, s0, s1, pe, r0, WROWS);
    const int step = 16 * WS;
    int kb = kr.lo + 16 * part_of;
    constexpr bool STAGED = DP <= kStagedWidth, EARLY = RB == 1;
    Rows<DP> K, V;
    Cols<DP> T;
    float *staged = shared + wave * 2 * 16 * (DP + 4);  // this wave's own
    K.template load<EX>(rows_rsrc(kp, k.st, kb, s1, p.d), k.st, p.d);
    V.template load<EX>(rows_rsrc(vp, v.st, kb, s1, p.d), v.st, p.d);
    if (!STAGED) T.template load<EX>(rows_rsrc(kp, k.st, kb, s1, p.d), k.st, p.d);
    for (; kb < kr.hi; kb += step) {
        f32x4 s[RB], dp[RB];
        if (STAGED) K.stage(staged);
#pragma unroll
        for (int b = 0; b < RB; ++b) s[b] = scores<DP, FORM>(K, Q[b]);
        K.template load<EX>(rows_rsrc(kp, k.st, kb + step, s1, p.d), k.st, p.d);
        if (STAGED && EARLY) T.take(staged);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int b = 0; b < RB; ++b) dp[b] = dots<DP>(V, G[b]);
        V.template load<EX>(rows_rsrc(vp, v.st, kb + step, s1, p.d), v.st, p.d);
        if (STAGED && !EARLY) T.take(staged);
        __builtin_amdgcn_sched_barrier(0);
        const bool whole = all_see<FORM != 0>(p, s1, pe, r0, WROWS, kb, 16);
        float away[RB];
        f32x4 steep[RB];
        if constexpr (FORM & (kBias | kCap)) {
#pragma unroll
            for (int b = 0; b < RB; ++b) away[b] = (float)(r0 + 16 * b + m - kb - 4 * g);
            bend_scores<FORM, RB, true>(p.bend, p.times, slope, away, s, steep);
        }
#pragma unroll
        for (int b = 0; b < RB; ++b) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                s[b][i] = probability<FORM>(p, s[b][i], l[b]) * (dp[b][i] - del[b]);
            const f32x4 ds = s[b];  // of the final scores
            if (FORM & kCap) s[b] *= steep[b];
            if (!whole) {
                const Range seen = keys_of<FORM != 0>(p, s0, s1, pe, r0 + 16 * b + m, 1);
#pragma unroll
                for (int i = 0; i < 4; ++i) s[b][i] = inside(seen, kb + 4 * g + i) ? s[b][i] : 0.0f;
            }
            if ((FORM & kBias) && slope_part) {
                const Range seen = keys_of<FORM != 0>(p, s0, s1, pe, r0 + 16 * b + m, 1);
                float sum = 0.0f;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    sum += whole || inside(seen, kb + 4 * g + i) ? ds[i] * fabsf(away[b] - (float)i) : 0.0f;
                slope_sum += r0 + 16 * b + m < s1 ? (double)sum : 0.0;  // rows past the sequence hold anything
            }
            A[b].add(T, s[b]);
        }
        if (!STAGED) {
            T.template load<EX>(rows_rsrc(kp, k.st, kb + step, s1, p.d), k.st, p.d);
            __builtin_amdgcn_sched_barrier(0);
        }
    }

    if ((FORM & kBias) && slope_part) {
#pragma unroll
        for (int i = 1; i < 64; i <<= 1) slope_sum += __shfl_xor(slope_sum, i, 64);
        if (lane == 0) *slope_part = slope_sum;
    }
    if (WS == 1) {
#pragma unroll
        for (int b = 0; b < RB; ++b) {
            const int r = r0 + 16 * b;
            if (r >= s1) break;
            const Rsrc ro = rows_rsrc(dq.p + h * dq.sh, dq.st, r, s1, p.d);
            A[b].each4([&](int d0, f32x4 y) {
                store4(ro, (EX || d0 < p.d) ? m * (int)dq.st * 4 + d0 * 4 : kOOB, y * p.factor);
            });
        }
    } else {
#pragma unroll
        for (int b = 0; b < RB; ++b) join_rows<DP, WS>(A[b], shared, dq, h, r0 + 16 * b, s1, p.d, p.factor);
    }
}

// dk and dv: the keys are held fixed and the blocks of 16 rows of every query
// head of the group are walked over.
template <int DP, bool EX, int RB, int WS, bool OWN, int FORM>
__device__ __forceinline__ void backward_dkv(const Problem &p, const Backward &a, int id, float *shared,
                                             const float *slopes) {
    const Strided &dout = a.dout, &q = a.q, &k = a.k, &v = a.v, &o = a.o, &dk = a.dk, &dv = a.dv;
    const float *lse = a.lse;
    constexpr int WROWS = 16 * RB, WR = 4 / WS, TILE = WR * WROWS;
    const int lane = threadIdx.x & 63, g = lane >> 4, m = lane & 15;
    const int wave = uniform(threadIdx.x >> 6);
    int h, x;
    head_and_tile(id, p.hq / p.group, 1, h, x);
    const Tile t = find_tile<TILE, FORM != 0>(p, x, false);
    outside_rows<TILE>(p, t, x, [&](int r) {
        zero_row(dk.p + r * dk.st + h * dk.sh, p.d);
        zero_row(dv.p + r * dv.st + h * dv.sh, p.d);
    });
    if (t.r0 < 0) return;
    const int s0 = t.s0, s1 = t.s1, t0 = t.r0, pe = prefix_end<FORM != 0>(p, t);
    const int part_of = wave / WR, k0 = t0 + wave % WR * WROWS;
    if (WS == 1 && k0 >= s1) return;

    Rows<DP> K[RB], V[RB];
    Acc<DP> DK[RB], DV[RB];
#pragma unroll
    for (int b = 0; b < RB; ++b) {
        K[b].template load<EX>(rows_rsrc(k.p + h * k.sh, k.st, k0 + 16 * b, s1, p.d), k.st, p.d);
        V[b].template load<EX>(rows_rsrc(v.p + h * v.sh, v.st, k0 + 16 * b, s1, p.d), v.st, p.d);
        DK[b].clear();
        DV[b].clear();
    }
    const Range rr = rows_of<FORM != 0>(p, s0, s1, pe, k0, WROWS);
    const int blocks = (rr.hi - rr.lo + 15) / 16, total = blocks * p.group;
    // Block n of the walk: head n % group of the group, and the n / group-th
    // block of rows from the last one on.  Workgroups that start together then
    // read the same rows of the same heads together, whatever their keys.
    int n = part_of, qh = n, qb = 0;
    const int step = WS;
    while (qh >= p.group) {
        qh -= p.group;
        ++qb;
    }
    Rows<DP> Q, G, out;
    Cols<DP> QT, GT;
    f32x4 l4, d4;
    const float *qp, *gp, *op;
    int r;
    auto at = [&]() {
        const int head = h * p.group + qh;
        const bool in = n < total;
        qp = q.p + head * q.sh;
        gp = dout.p + head * dout.sh;
        op = o.p + head * o.sh;
        r = in ? rr.lo + 16 * (blocks - 1 - qb) : s1;
    };
    auto stats = [&](const float *from) {
        const int left = r < s1 ? s1 - r : 0;
        return load4(__builtin_amdgcn_make_buffer_rsrc((void *)(from + (int64_t)(h * p.group + qh) * p.tokens + r),
                                                       (short)0, min(left, 16) * 4, 0x00020000),
                     16 * g);
    };
    at();
    Q.template load<EX>(rows_rsrc(qp, q.st, r, s1, p.d), q.st, p.d);
    G.template load<EX>(rows_rsrc(gp, dout.st, r, s1, p.d), dout.st, p.d);
    if (OWN) out.template load<EX>(rows_rsrc(op, o.st, r, s1, p.d), o.st, p.d);
    else d4 = stats(a.delta);
    l4 = stats(lse);
    constexpr bool STAGED = DP <= kStagedWidth, EARLY = RB == 1;
    float *staged = shared + wave * 2 * 16 * (DP + 4), *staged_g = staged + 16 * (DP + 4);  // this wave's own
    while (n < total) {
        const int row = r;
        const float *qc = qp, *gc = gp;
        const float slope = FORM & kBias ? slope_of(slopes, h * p.group + uniform(qh)) : 0.0f;
        if (STAGED) {
            Q.stage(staged);
            G.stage(staged_g);
        }
        n += step;
        qh += step;
        while (qh >= p.group) {
            qh -= p.group;
            ++qb;
        }
        at();
        f32x4 s[RB], dp[RB];
#pragma unroll
        for (int b = 0; b < RB; ++b) s[b] = scores<DP, FORM>(Q, K[b]);
        if (OWN) {
            const float del = row_dots<DP>(G, out);
#pragma unroll
            for (int i = 0; i < 4; ++i) d4[i] = __shfl(del, 4 * g + i, 64);
        }
        if (STAGED) {
            Q.template load<EX>(rows_rsrc(qp, q.st, r, s1, p.d), q.st, p.d);
            if (EARLY) GT.take(staged_g);
        } else {
            GT.template load<EX>(rows_rsrc(gc, dout.st, row, s1, p.d), dout.st, p.d);
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int b = 0; b < RB; ++b) dp[b] = dots<DP>(G, V[b]);
        if (STAGED) {
            G.template load<EX>(rows_rsrc(gp, dout.st, r, s1, p.d), dout.st, p.d);
            if (OWN) out.template load<EX>(rows_rsrc(op, o.st, r, s1, p.d), o.st, p.d);
            if (!EARLY) GT.take(staged_g);
        } else {
            QT.template load<EX>(rows_rsrc(qc, q.st, row, s1, p.d), q.st, p.d);
        }
        __builtin_amdgcn_sched_barrier(0);
        const bool whole = all_see<FORM != 0>(p, s1, pe, row, 16, k0, WROWS);
        f32x4 steep[RB];
        if constexpr (FORM & (kBias | kCap)) {
            float away[RB];
#pragma unroll
            for (int b = 0; b < RB; ++b) away[b] = (float)(k0 + 16 * b + m - row - 4 * g);
            bend_scores<FORM, RB, true>(p.bend, p.times, slope, away, s, steep);
        }
#pragma unroll
        for (int b = 0; b < RB; ++b) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                s[b][i] = probability<FORM>(p, s[b][i], l4[i]);
                dp[b][i] = s[b][i] * (dp[b][i] - d4[i]);
            }
            if (FORM & kCap) dp[b] *= steep[b];
            if (!whole) {
                const Range seen = rows_of<FORM != 0>(p, s0, s1, pe, k0 + 16 * b + m, 1);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const bool in = inside(seen, row + 4 * g + i);
                    s[b][i] = in ? s[b][i] : 0.0f;
                    dp[b][i] = in ? dp[b][i] : 0.0f;
                }
            }
        }
        l4 = stats(lse);
        if (!OWN) d4 = stats(a.delta);
        if (STAGED && EARLY) {
            QT.take(staged);
            __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int b = 0; b < RB; ++b) DV[b].add(GT, s[b]);
        if (STAGED) {
            if (!EARLY) QT.take(staged);
        } else {
            Q.template load<EX>(rows_rsrc(qp, q.st, r, s1, p.d), q.st, p.d);
            __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int b = 0; b < RB; ++b) DK[b].add(QT, dp[b]);
        if (!STAGED) {
            G.template load<EX>(rows_rsrc(gp, dout.st, r, s1, p.d), dout.st, p.d);
            if (OWN) out.template load<EX>(rows_rsrc(op, o.st, r, s1, p.d), o.st, p.d);
            __builtin_amdgcn_sched_barrier(0);
        }
    }

    if (WS == 1) {
#pragma unroll
        for (int b = 0; b < RB; ++b) {
            const int r1 = k0 + 16 * b;
            if (r1 >= s1) break;
            const Rsrc rk = rows_rsrc(dk.p + h * dk.sh, dk.st, r1, s1, p.d);
            const Rsrc rv = rows_rsrc(dv.p + h * dv.sh, dv.st, r1, s1, p.d);
            DK[b].each4([&](int d0, f32x4 y) {
                store4(rk, (EX || d0 < p.d) ? m * (int)dk.st * 4 + d0 * 4 : kOOB, y * p.factor);
            });
            DV[b].each4([&](int d0, f32x4 y) {
                store4(rv, (EX || d0 < p.d) ? m * (int)dv.st * 4 + d0 * 4 : kOOB, y);
            });
        }
    } else {
#pragma unroll
        for (int b = 0; b < RB; ++b) {
            join_rows<DP, WS>(DK[b], shared, dk, h, k0 + 16 * b, s1, p.d, p.factor);
            join_rows<DP, WS>(DV[b], shared, dv, h, k0 + 16 * b, s1, p.d, 1.0f);
        }
    }
}

template <int DP, bool EX, int RBQ, int RBK, int WS, bool OWN, int FORM>
__global__ __launch_bounds__(256, DP >= 96 && (RBQ == 2 || RBK == 2) ? 1 : 2) void attention_bwd(Problem p, Backward a,
                                                                                              int key_groups, int tiles, const float *slopes,
                                                                                              double *slope_parts) {
    // the waves' turned rows, and in the end what they join
    __shared__ __align__(16) float shared[(DP <= kStagedWidth ? 8 : 4) * 16 * (DP + 4)];
    const int id = p.first + (int)blockIdx.x;
    if (id < key_groups) backward_dkv<DP, EX, RBK, WS, OWN, FORM>(p, a, id, shared, slopes);
    else backward_dq<DP, EX, RBQ, WS, OWN, FORM>(p, a, id - key_groups, shared, tiles, slopes, slope_parts);
}

// The slopes' gradients: a workgroup adds a head's parts, a thread every 256th
// and then the threads in order of a tree.
__global__ __launch_bounds__(256) void attention_slopes(const double *parts, int64_t count, float *dslopes) {
    __shared__ double meet[256];
    const double *mine = parts + blockIdx.x * count;
    double sum = 0.0;
    for (int64_t i = threadIdx.x; i < count; i += 256) sum += mine[i];
    meet[threadIdx.x] = sum;
    for (int half = 128; half > 0; half >>= 1) {
        __syncthreads();
        if ((int)threadIdx.x < half) meet[threadIdx.x] += meet[threadIdx.x + half];
    }
    if (threadIdx.x == 0) dslopes[blockIdx.x] = (float)-meet[0];
}

// --- host ---

// Tokens stay so far below 2^30 that the tiles of 64 sequences, as find_tile
// counts them, sum to less than 2^31 whatever cu_seqlens holds: 64 bounds that
// go up and down rise by 32 times the tokens at most, in tiles of 16 rows or more.
constexpr int64_t kMaxTokens = ((int64_t)1 << 30) - 64, kMaxStride = (int64_t)1 << 22, kMaxHeadStride = (int64_t)1 << 40;

int check_tensor(const View &v, int64_t tokens, int64_t d) {
    if (v.t->data == nullptr) return GEMM_ERR_NULL;
    const int64_t st = v.t->token_stride, sh = v.t->head_stride;
    if (st < 0 || sh < 0 || sh > kMaxHeadStride) return GEMM_ERR_SHAPE;
    if (tokens > 1 && (st < d || st >= kMaxStride)) return GEMM_ERR_SHAPE;
    if (v.output && !rows_apart(v, tokens, d)) return GEMM_ERR_SHAPE;
    if (!aligned(v.t->data, 16) || (tokens > 1 && st % 4) || (v.heads > 1 && sh % 4)) return GEMM_ERR_ALIGN;
    return GEMM_OK;
}

// scale log2(e) as the forward pass folds it into its exponents: the largest
// scales would make it infinite, and a score of zero NaN.
float folded(double scale) { return (float)(scale * 1.44269504088896340736); }

int check_problem(const attn_problem &p) {
    if (p.tokens < 0 || p.tokens >= kMaxTokens || p.q_heads < 1 || p.q_heads > 65535 || p.kv_heads < 1 ||
        p.kv_heads > p.q_heads || p.q_heads % p.kv_heads || p.head_dim < 4 || p.head_dim > 128 || p.head_dim % 4 ||
        p.window < 0)
        return GEMM_ERR_SHAPE;
    if (p.cu_seqlens && (p.num_seqs < 0 || p.num_seqs >= ((int64_t)1 << 24))) return GEMM_ERR_SHAPE;
    if (!((float)p.scale > 0.0f) || !std::isfinite(folded(p.scale)) || (p.causal != 0 && p.causal != 1))
        return GEMM_ERR_DTYPE;
    if (!aligned(p.cu_seqlens, 4)) return GEMM_ERR_ALIGN;
    return GEMM_OK;
}

// No cap, bias or prefix.
constexpr attn_scores kPlain = {0.0, nullptr, nullptr};

int check_scores(const attn_problem &p, const attn_scores &s) {
    if (!(s.softcap == 0.0 || (s.softcap >= 1e-6 && s.softcap <= 1e6))) return GEMM_ERR_DTYPE;
    if (s.softcap > 0.0) {  // raw scores over the cap stay in fp32's normal range
        const float bend = (float)(p.scale / s.softcap);
        if (!(bend >= 0x1p-126f) || !std::isfinite(bend)) return GEMM_ERR_DTYPE;
    }
    if (s.prefix_lens && !p.causal) return GEMM_ERR_DTYPE;
    return aligned(s.slopes, 4) && aligned(s.prefix_lens, 4) ? GEMM_OK : GEMM_ERR_ALIGN;
}

// What all workgroups read: sequences, slopes and prefixes.
struct Shared {
    Span part[3];
    Shared(const attn_problem &p, const attn_scores &s)
        : part{{p.cu_seqlens, p.cu_seqlens ? (p.num_seqs + 1) * 4 : 0},
               {s.slopes, p.q_heads * 4},
               {s.prefix_lens, (p.cu_seqlens ? p.num_seqs : 1) * 4}} {}
    bool meets(const Span &x) const {
        for (const Span &s : part)
            if (spans_overlap(x, s)) return true;
        return false;
    }
    bool meets(const View &v, const attn_problem &p) const {
        for (const Span &s : part)
            if (s.bytes > 0 && in_range(v, s.p, s.bytes, p.tokens, p.head_dim)) return true;
        return false;
    }
};

Problem device_problem(const attn_problem &a, const attn_scores &s) {
    Problem p;
    p.cu = a.cu_seqlens;
    p.nseq = a.cu_seqlens ? (int)a.num_seqs : 1;
    p.tokens = (int)a.tokens;
    p.hq = (int)a.q_heads;
    p.group = (int)(a.q_heads / a.kv_heads);
    p.d = (int)a.head_dim;
    p.causal = (int)a.causal;
    p.window = a.window < a.tokens ? (int)a.window : 0;  // a wider window hides nothing
    p.first = 0;
    p.factor = (float)a.scale;
    const double times = s.softcap > 0.0 ? s.softcap : a.scale, scale = s.slopes ? 1.0 : times;
    p.scale = (float)scale;
    p.c = folded(scale);
    p.times = (float)times;
    p.prefix = s.prefix_lens;
    p.bend = s.softcap > 0.0 ? (float)(a.scale / s.softcap) : 0.0f;
    return p;
}

// Tiles of `tile` rows a head: every sequence's own, and enough for the rows of none.
int64_t tiles_of(const attn_problem &p, int64_t tile) {
    const int64_t whole = (p.tokens + tile - 1) / tile;
    return p.cu_seqlens ? std::max(whole, p.tokens / tile + p.num_seqs) : whole;
}

// How a kernel's rows (or keys) are dealt out: RB blocks of 16 a wave, WS
// waves of a workgroup to the same rows.  A second block a wave halves the
// loads of the other side for each product; joined waves (WS = 4) make the
// tiles short, so that the chip is full and evenly loaded, at the price of
// the joining.  Measured over 1 to 64 sequences of 64 to 8192 rows, 8 to 16
// heads of 32 to 128, causal and not:
//  * few rows: one block a wave, joined (512 rows, 12 heads of 64: forward
//    12.8 us against 13.7 with two blocks and 39.8 unjoined; backward 27.5
//    against 33.3);
//  * many rows: two blocks, joined (2 x 4096 rows: forward 403 us against 455
//    with one block and 506 unjoined; backward 1371 against 1733);
//  * many short sequences: two blocks, each wave its own rows (64 x 128 rows:
//    forward 26 us against 38 joined; backward 110 against 156; 16 x 512 rows:
//    backward 231 against 261).
// `many` is the number of 32-row tiles from which two blocks win, `most` the
// average sequence length (all that the host knows) that counts as short;
// from 512 tiles of 128 rows on unjoined waves fill the chip.  Both sides of
// each bound, causal, heads of 64 unless said otherwise, us:
//  * short sequences, forward, unjoined against joined: 64 x 128 rows with 4
//    heads (256 tiles) 14.9 to 14.9, with 8 (512) 22.0 to 27.5; 12 heads of 32 x
//    256 rows 42.2 to 51.4, of 16 x 512 72 to 74, of 8 x 1024 133 to 119.
//    Backward: 12 heads of 16 x 512 231 to 263, of 8 x 1024 396 to 423, and of
//    width 32 131 to 137 and 226 to 219.
struct Plan {
    int rb, ws;
    int64_t rows() const { return 16 * rb * (4 / ws); }
};
int64_t average_length(const attn_problem &p) {
    const int64_t length = p.cu_seqlens ? p.tokens / std::max<int64_t>(1, p.num_seqs) : p.tokens;
    return p.window > 0 ? std::min(length, p.window) : length;
}
Plan plan(const attn_problem &p, int64_t heads, int64_t many, int64_t most) {
    if (average_length(p) <= most && p.tokens / 128 * heads >= 512) return {2, 1};
    return {p.tokens / 32 * heads >= many ? 2 : 1, 4};
}
// 2048 rows of 8 heads (512 tiles) 51.3 us with one block, 53.2 with two; 4096
// of 8 (1024) 158 and 163, of 12 (1536) 234 and 208.  Heads of 128: 88 and 97,
// 308 and 273, 457 and 397; without a causal mask 8 heads of 64 gain from 512
// tiles on (80 and 72).
Plan plan_forward(const attn_problem &p) { return plan(p, p.q_heads, 1024, 256); }
// Keys of the backward pass: a tile of few keys takes all rows of the group's
// heads, so two blocks pay from fewer tiles where no mask makes tiles uneven.
// With 8 heads, one block and two, us:
//  * causal, 64 wide (320 tiles): 1024 rows (256 tiles) 47 and 63, 1280 (320)
//    70 and 69, 1536 (384) 98 and 84.  2 shared heads gain only from about
//    512: 5120 rows (320) 731 and 873, 4 of them at 4096 (512) 928 and 912;
//  * causal, 128 wide (256 tiles): 768 rows (192) 64 and 62, 1024 (256) 100 and
//    89; 2 shared heads 2816 rows (176) 525 and 728, 4096 (256) 1063 and 1057;
//  * no mask (192 tiles): 64 wide 768 rows (192) 45 and 50, 1024 (256) 84 and
//    64, 1280 107 and 140, 16 heads of 1024 (512) 136 and 124; 2 shared heads of
//    128 at 2816 rows (176) 975 and 1014, at 4096 (256) 1976 and 1871.
Plan plan_keys(const attn_problem &p) {
    return plan(p, p.kv_heads, !p.causal ? 192 : p.head_dim > 64 ? 256 : 320, 512);
}
// Rows of the backward pass: as the keys, but with shared heads two blocks
// throughout, as there are several times as many tiles of rows then (2048
// rows, 8 heads on 2 of 128: 299 us against 391).
Plan plan_rows(const attn_problem &p) {
    const Plan keys = plan_keys(p);
    return {p.q_heads > p.kv_heads ? 2 : keys.rb, keys.ws};
}

// Whether the backward pass forms delta in its own kernel: where that is
// short, so that a launch in front counts for more than the loads (256 rows,
// 12 heads of 64: 16.5 us a call against 20.6; 512 rows: 30.6 against 27.5;
// 256 rows, 8 heads of 128: 24.6 against 21.8).
bool own_delta(const attn_problem &p) {
    const double pairs = (double)p.tokens * (double)average_length(p) / (p.causal ? 2 : 1);
    return pairs * (double)(p.q_heads * (p.q_heads / p.kv_heads)) * (double)(p.head_dim * p.head_dim) <= 3.3e9;
}

#define ATTN_BY_DIM(LAUNCH)                                                     \
    do {                                                                        \
        const int64_t d_ = a.p.head_dim;                                        \
        if (d_ == 32) LAUNCH(32, true);                                         \
        else if (d_ < 32) LAUNCH(32, false);                                    \
        else if (d_ == 64) LAUNCH(64, true);                                    \
        else if (d_ < 64) LAUNCH(64, false);                                    \
        else if (d_ == 96) LAUNCH(96, true);                                    \
        else if (d_ < 96) LAUNCH(96, false);                                    \
        else if (d_ == 128) LAUNCH(128, true);                                  \
        else LAUNCH(128, false);                                                \
    } while (0)

// `a` has p, q, k, v, out and lse.
template <int FORM, class Args>
int forward(const Args &a, const attn_scores &scores, void *stream) {
    const int64_t T = a.p.tokens, D = a.p.head_dim;
    int st = check_problem(a.p);
    if (st == GEMM_OK && FORM) st = check_scores(a.p, scores);
    if (st != GEMM_OK) return st;
    if (T == 0) return GEMM_OK;
    const View q = {&a.q, a.p.q_heads, false}, k = {&a.k, a.p.kv_heads, false}, v = {&a.v, a.p.kv_heads, false},
               o = {&a.out, a.p.q_heads, true};
    for (const View *x : {&q, &k, &v, &o})
        if ((st = check_tensor(*x, T, D)) != GEMM_OK) return st;
    if (a.lse == nullptr) return GEMM_ERR_NULL;
    if (!aligned(a.lse, 4)) return GEMM_ERR_ALIGN;
    const bool in_place = same_tensor(a.out, a.q);
    const int64_t lse_bytes = a.p.q_heads * T * 4;
    const Shared shared(a.p, scores);
    if ((!in_place && overlap(o, q, T, D)) || overlap(o, k, T, D) || overlap(o, v, T, D) ||
        in_range(o, a.lse, lse_bytes, T, D) || in_range(q, a.lse, lse_bytes, T, D) ||
        in_range(k, a.lse, lse_bytes, T, D) || in_range(v, a.lse, lse_bytes, T, D) ||
        shared.meets(o, a.p) || shared.meets({a.lse, lse_bytes}))
        return GEMM_ERR_ALIAS;
    Problem p = device_problem(a.p, scores);
    const Plan how = plan_forward(a.p);
    const int64_t grid = tiles_of(a.p, how.rows()) * a.p.q_heads;
    if (grid >= ((int64_t)1 << 31)) return GEMM_ERR_SHAPE;
    const Strided sq = strided(a.q, T, a.p.q_heads), sk = strided(a.k, T, a.p.kv_heads),
                  sv = strided(a.v, T, a.p.kv_heads), so = strided(a.out, T, a.p.q_heads);
    hipStream_t hs = static_cast<hipStream_t>(stream);
    return in_slices(grid, 256, [&](int64_t first, unsigned count) {
        p.first = (int)first;
#define FWD_AS(DP, EX, RB, WS) \
    hipLaunchKernelGGL((attention_fwd<DP, EX, RB, WS, FORM>), dim3(count), dim3(256), 0, hs, p, sq, sk, sv, so, a.lse, \
                       scores.slopes)
#define FWD(DP, EX)                           \
    do {                                      \
        if (how.ws == 1) FWD_AS(DP, EX, 2, 1); \
        else if (how.rb == 2) FWD_AS(DP, EX, 2, 4); \
        else FWD_AS(DP, EX, 1, 4);            \
    } while (0)
        ATTN_BY_DIM(FWD);
#undef FWD
#undef FWD_AS
    });
}

// The backward pass's scratch: delta, and behind it the slopes' parts.
struct Scratch {
    int64_t delta_bytes, parts, bytes;  // parts: doubles of one head
};
Scratch scratch_of(const attn_problem &p, bool slopes) {
    Scratch s = {own_delta(p) ? 0 : p.q_heads * p.tokens * 4, 0, 0};
    s.bytes = s.delta_bytes;
    if (slopes) {
        const Plan rows = own_delta(p) ? Plan{1, 4} : plan_rows(p);
        s.parts = tiles_of(p, rows.rows()) * 4;
        s.delta_bytes = (s.delta_bytes + 7) / 8 * 8;
        s.bytes = s.delta_bytes + p.q_heads * s.parts * 8;
    }
    return s;
}

// `a` has p, dout, q, k, v, out, lse, dq, dk, dv, workspace and workspace_bytes.
template <int FORM, class Args>
int backward(const Args &a, const attn_scores &scores, float *dslopes, void *stream) {
    const int64_t T = a.p.tokens, D = a.p.head_dim, HQ = a.p.q_heads, HK = a.p.kv_heads;
    hipStream_t hs = static_cast<hipStream_t>(stream);
    int st = check_problem(a.p);
    if (st == GEMM_OK && FORM) st = check_scores(a.p, scores);
    if (st != GEMM_OK) return st;
    if (dslopes && !scores.slopes) return GEMM_ERR_NULL;
    if (!aligned(dslopes, 4)) return GEMM_ERR_ALIGN;
    const Shared shared(a.p, scores);
    if (shared.meets({dslopes, HQ * 4})) return GEMM_ERR_ALIAS;
    if (T == 0) {
        if (!dslopes) return GEMM_OK;
        hipLaunchKernelGGL(attention_slopes, dim3((unsigned)HQ), dim3(256), 0, hs, nullptr, (int64_t)0, dslopes);
        return hipGetLastError() == hipSuccess ? GEMM_OK : GEMM_ERR_LAUNCH;
    }
    const View in[5] = {{&a.dout, HQ, false}, {&a.q, HQ, false}, {&a.k, HK, false}, {&a.v, HK, false}, {&a.out, HQ, false}};
    const View res[3] = {{&a.dq, HQ, true}, {&a.dk, HK, true}, {&a.dv, HK, true}};
    for (const View &x : in)
        if ((st = check_tensor(x, T, D)) != GEMM_OK) return st;
    for (const View &x : res)
        if ((st = check_tensor(x, T, D)) != GEMM_OK) return st;
    if (a.lse == nullptr) return GEMM_ERR_NULL;
    if (!aligned(a.lse, 4)) return GEMM_ERR_ALIGN;
    const int64_t row_bytes = HQ * T * 4;
    const bool own = own_delta(a.p);
    const Scratch need = scratch_of(a.p, dslopes != nullptr);
    const Span scratch = {a.workspace, need.bytes}, rows_lse = {a.lse, row_bytes}, slopes = {dslopes, HQ * 4};
    if (need.bytes > 0) {
        if (a.workspace == nullptr || a.workspace_bytes < need.bytes) return GEMM_ERR_WORKSPACE;
        if (!aligned(a.workspace, need.parts > 0 ? 8 : 4)) return GEMM_ERR_ALIGN;
    }
    // the scratch and the slopes' gradient apart from one another and from everything else
    for (const Span &s : {scratch, slopes}) {
        if (s.p == nullptr || s.bytes == 0) continue;
        if (spans_overlap(s, rows_lse) || shared.meets(s)) return GEMM_ERR_ALIAS;
        for (const View &x : in)
            if (in_range(x, s.p, s.bytes, T, D)) return GEMM_ERR_ALIAS;
        for (const View &x : res)
            if (in_range(x, s.p, s.bytes, T, D)) return GEMM_ERR_ALIAS;
    }
    if (spans_overlap(scratch, slopes)) return GEMM_ERR_ALIAS;
    for (int i = 0; i < 3; ++i) {
        for (const View &x : in)
            if (overlap(res[i], x, T, D)) return GEMM_ERR_ALIAS;
        for (int j = 0; j < i; ++j)
            if (overlap(res[i], res[j], T, D)) return GEMM_ERR_ALIAS;
        if (in_range(res[i], a.lse, row_bytes, T, D) || shared.meets(res[i], a.p)) return GEMM_ERR_ALIAS;
    }
    Problem p = device_problem(a.p, scores);
    const Plan keys = own ? Plan{1, 4} : plan_keys(a.p), rows = own ? keys : plan_rows(a.p);
    // whole turns of the 8 XCDs, so that the second part's heads keep to theirs
    const int64_t nk = (tiles_of(a.p, keys.rows()) * HK + 7) / 8 * 8, tiles = tiles_of(a.p, rows.rows()),
                  grid = nk + tiles * HQ;
    if (grid >= ((int64_t)1 << 31) || (HQ * T + 15) / 16 >= ((int64_t)1 << 31)) return GEMM_ERR_SHAPE;
    const Backward b = {strided(a.dout, T, HQ), strided(a.q, T, HQ),  strided(a.k, T, HK),  strided(a.v, T, HK),
                        strided(a.out, T, HQ),  strided(a.dq, T, HQ), strided(a.dk, T, HK), strided(a.dv, T, HK),
                        a.lse, static_cast<const float *>(a.workspace)};
    double *parts = need.parts > 0 ? reinterpret_cast<double *>(static_cast<char *>(a.workspace) + need.delta_bytes)
                                   : nullptr;
    if (!own) {
        // the main kernel reads what this one writes
        st = in_slices((HQ * T + 15) / 16, 256, [&](int64_t first, unsigned count) {
            hipLaunchKernelGGL(attention_delta, dim3(count), dim3(256), 0, hs, p, b.dout, b.o,
                               static_cast<float *>(a.workspace), first);
        });
        if (st != GEMM_OK) return st;
    }
    st = in_slices(grid, 256, [&](int64_t first, unsigned count) {
        p.first = (int)first;
#define BWD_AS(DP, EX, RBQ, RBK, WS, OWN) \
    hipLaunchKernelGGL((attention_bwd<DP, EX, RBQ, RBK, WS, OWN, FORM>), dim3(count), dim3(256), 0, hs, p, b, (int)nk, (int)tiles, \
                       scores.slopes, parts)
#define BWD(DP, EX)                                              \
    do {                                                         \
        if (own) BWD_AS(DP, EX, 1, 1, 4, true);                  \
        else if (keys.ws == 1) BWD_AS(DP, EX, 2, 2, 1, false);   \
        else if (keys.rb == 2) BWD_AS(DP, EX, 2, 2, 4, false);   \
        else if (rows.rb == 2) BWD_AS(DP, EX, 2, 1, 4, false);   \
        else BWD_AS(DP, EX, 1, 1, 4, false);                     \
    } while (0)
        ATTN_BY_DIM(BWD);
#undef BWD
#undef BWD_AS
    });
    if (st != GEMM_OK || need.parts == 0) return st;
    hipLaunchKernelGGL(attention_slopes, dim3((unsigned)HQ), dim3(256), 0, hs, parts, need.parts, dslopes);
    return hipGetLastError() == hipSuccess ? GEMM_OK : GEMM_ERR_LAUNCH;
}

}  // namespace

#endif  // ATTENTION_KERNELS_H
