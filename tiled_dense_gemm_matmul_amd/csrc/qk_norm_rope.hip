// The norm of queries and keys for each head and the position rotation, in
// one pass over both, forward and backward, for MI355X (gfx950) (definitions
// in attention.h).
//
// The work is bound by memory: every value is read and written once (the
// backward pass reads dy and x and writes dx).  A wave takes one token and a
// group of G lanes one of its heads, each lane W rotated pairs (a, b), so
// that the sums over a head stay within the group and a lane turns its pairs
// by the same angles in every head of the token: each token's sines and
// cosines are formed once in a wave and kept in registers.
//  * W = 4 with 16-byte accesses where the pairs' layout and the arrays'
//    alignment allow it, else W = 1.
//  * The dimensions that are not rotated are paired in the same way and turned by
//    the angle zero, so a head is one kind of pair throughout.
//  * The angle pos * inv_freq is formed and reduced to a part of a turn in 64
//    bits, with the rounding errors of both products carried along.  Sine and
//    cosine are taken of that part rounded to fp32, and turned by what the
//    rounding left out (without that they were off by up to 1.1e-7, not
//    3e-8, and by far more than an ulp near their zeros), so they are good to
//    fp32 at any position up to 2^53.
//  * The weight's gradient sums over all tokens and heads: fp32 over a token's
//    heads in a lane, then 64 bits over tokens, lanes, waves and workgroups,
//    each in a fixed order; a second small kernel adds the workgroups' parts.

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

struct Norm {
    const void *pos;
    const float *inv_freq, *qw, *kw;
    int tokens, hq, hk, d, half;  // half: rotated pairs
    int wide, interleaved;
    float eps, inv_d;
};

// The W pairs from pair p on of a head, as (a, b).
template <int W>
struct Pairs {
    float a[W], b[W];
};

// Where pairs p .. p + W - 1 lie in a head: W consecutive values at `first`
// and W at `second` (2 W values from `first` on when interleaved).
struct Place {
    int first, second;
};
__device__ __forceinline__ Place place(const Norm &n, int p, int w) {
    if (n.interleaved) return {2 * p, 2 * p + w};
    if (p < n.half) return {p, p + n.half};
    const int rest = n.d / 2 - n.half;
    return {2 * n.half + p - n.half, 2 * n.half + p - n.half + rest};
}

template <int W>
__device__ __forceinline__ Pairs<W> read_pairs(const Norm &n, const float *head, Place at) {
    Pairs<W> r;
    if constexpr (W == 4) {
        const f32x4 u = *(const f32x4 *)(head + at.first), v = *(const f32x4 *)(head + at.second);
        if (n.interleaved) {
            r.a[0] = u[0]; r.b[0] = u[1]; r.a[1] = u[2]; r.b[1] = u[3];
            r.a[2] = v[0]; r.b[2] = v[1]; r.a[3] = v[2]; r.b[3] = v[3];
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) { r.a[i] = u[i]; r.b[i] = v[i]; }
        }
    } else {
        r.a[0] = head[at.first];
        r.b[0] = head[at.second];
    }
    return r;
}

template <int W>
__device__ __forceinline__ void write_pairs(const Norm &n, float *head, Place at, const Pairs<W> &r) {
    if constexpr (W == 4) {
        f32x4 u = {r.a[0], r.a[1], r.a[2], r.a[3]}, v = {r.b[0], r.b[1], r.b[2], r.b[3]};
        if (n.interleaved) {
            u = f32x4{r.a[0], r.b[0], r.a[1], r.b[1]};
            v = f32x4{r.a[2], r.b[2], r.a[3], r.b[3]};
        }
        *(f32x4 *)(head + at.first) = u;
        *(f32x4 *)(head + at.second) = v;
    } else {
        head[at.first] = r.a[0];
        head[at.second] = r.b[0];
    }
}

// Cosine and sine of the angle of pair p at a token (1 and 0 past the rotated pairs).
__device__ __forceinline__ void turn(const Norm &n, double pos, int p, float &c, float &s) {
#pragma clang fp contract(off)  // the products' roundings are taken as they are
    c = 1.0f;
    s = 0.0f;
    if (p < n.half) {
        // 1 / (2 pi) as the sum of two doubles
        constexpr double kTurn = 0x1.45f306dc9c883p-3, kTurnLow = -0x1.6b01ec5417056p-57;
        const double f = (double)n.inv_freq[p];
        const double angle = pos * f, angle_low = fma(pos, f, -angle);
        const double turns = angle * kTurn;
        const double low = fma(angle, kTurn, -turns) + (angle * kTurnLow + angle_low * kTurn);
        const double half_turns = 2.0 * ((turns - rint(turns)) + low);
        const float x = (float)half_turns, rest = (float)((half_turns - (double)x) * M_PI);
        sincospif(x, &s, &c);
        const float s0 = s;
        s = fmaf(c, rest, s);
        c = fmaf(-s0, rest, c);
    }
}
__device__ __forceinline__ double position(const Norm &n, int t) {
    return n.wide ? (double)((const int64_t *)n.pos)[t] : (double)((const int *)n.pos)[t];
}

template <int G>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
    for (int o = 1; o < G; o <<= 1) v += __shfl_xor(v, o, 64);
    return v;
}

// NP groups of W pairs a lane, G lanes a head; a wave takes token
// item / chunks and every (chunks * 64 / G)-th head from its chunk on; `first`
// workgroups lie in front of this launch's.
template <int W, int G, int NP>
__global__ __launch_bounds__(256) void qk_norm_rope_fwd(Norm n, Strided q, Strided k, Strided yq, Strided yk, int chunks,
                                                        int64_t first) {
    constexpr int HW = 64 / G;  // heads at a time
    const int lane = threadIdx.x & 63, part = lane % G, slot = lane / G;
    const int64_t item = (first + blockIdx.x) * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int t = (int)(item / chunks), chunk = (int)(item % chunks);
    if (t >= n.tokens) return;
    const double pos = position(n, t);
    Place at[NP];
    bool in[NP];
    float c[NP][W], s[NP][W];
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        const int p = (i * G + part) * W;
        in[i] = p < n.d / 2;
        at[i] = place(n, p, W);
#pragma unroll
        for (int e = 0; e < W; ++e) turn(n, pos, p + e, c[i][e], s[i][e]);
    }
    const int heads = n.hq + n.hk;
    for (int h = chunk * HW + slot; h < heads; h += chunks * HW) {
        const bool isq = h < n.hq;
        const float *x = isq ? q.p + t * q.st + h * q.sh : k.p + t * k.st + (h - n.hq) * k.sh;
        float *y = isq ? yq.p + t * yq.st + h * yq.sh : yk.p + t * yk.st + (h - n.hq) * yk.sh;
        const float *weight = isq ? n.qw : n.kw;
        Pairs<W> v[NP], w[NP];
        float sq = 0.0f;
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            if (in[i]) {
                v[i] = read_pairs<W>(n, x, at[i]);
                w[i] = read_pairs<W>(n, weight, at[i]);
#pragma unroll
                for (int e = 0; e < W; ++e) sq += v[i].a[e] * v[i].a[e] + v[i].b[e] * v[i].b[e];
            }
        }
        const float r = rsqrtf(lanes_sum<G>(sq) * n.inv_d + n.eps);
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            if (!in[i]) continue;
            Pairs<W> o;
#pragma unroll
            for (int e = 0; e < W; ++e) {
                const float a = v[i].a[e] * r * w[i].a[e];
                const float b = v[i].b[e] * r * w[i].b[e];
                o.a[e] = a * c[i][e] - b * s[i][e];
                o.b[e] = b * c[i][e] + a * s[i][e];
            }
            write_pairs<W>(n, y, at[i], o);
        }
    }
}

// Backward.  Workgroup b writes its part of the weights' gradients, 2 D
// doubles, to parts + 2 D b: each lane's sums, added over the lanes of one
// pair in lane order and over the waves in wave order.
constexpr int kWaves = 8;    // of a workgroup of the backward pass
constexpr int kParts = 512;  // workgroups of the backward pass at most: two a CU

template <int W, int G, int NP>
__global__ __launch_bounds__(64 * kWaves) void qk_norm_rope_bwd(Norm n, Strided gq, Strided gk, Strided q, Strided k, Strided dq,
                                                        Strided dk, double *parts, int chunks) {
    constexpr int HW = 64 / G;
    const int lane = threadIdx.x & 63, part = lane % G, slot = lane / G;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    Place at[NP];
    bool in[NP];
    double sums[2][NP][2 * W];
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        const int p = (i * G + part) * W;
        in[i] = p < n.d / 2;
        at[i] = place(n, p, W);
#pragma unroll
        for (int e = 0; e < 2 * W; ++e) sums[0][i][e] = sums[1][i][e] = 0.0;
    }
    const int heads = n.hq + n.hk;
    const int64_t items = (int64_t)n.tokens * chunks;
    for (int64_t item = (int64_t)blockIdx.x * kWaves + wave; item < items;
         item += (int64_t)gridDim.x * kWaves) {
        const int t = (int)(item / chunks), chunk = (int)(item % chunks);
        const double pos = position(n, t);
        float c[NP][W], s[NP][W];
        float dw[2][NP][2 * W];
#pragma unroll
        for (int i = 0; i < NP; ++i) {
#pragma unroll
            for (int e = 0; e < W; ++e) {
                turn(n, pos, (i * G + part) * W + e, c[i][e], s[i][e]);
                dw[0][i][e] = dw[0][i][W + e] = dw[1][i][e] = dw[1][i][W + e] = 0.0f;
            }
        }
        for (int h = chunk * HW + slot; h < heads; h += chunks * HW) {
            const bool isq = h < n.hq;
            const int hh = isq ? h : h - n.hq;
            const float *x = isq ? q.p + t * q.st + hh * q.sh : k.p + t * k.st + hh * k.sh;
            const float *g = isq ? gq.p + t * gq.st + hh * gq.sh : gk.p + t * gk.st + hh * gk.sh;
            float *d = isq ? dq.p + t * dq.st + hh * dq.sh : dk.p + t * dk.st + hh * dk.sh;
            const float *weight = isq ? n.qw : n.kw;
            Pairs<W> v[NP], dn[NP], w[NP];
            float sq = 0.0f, dot = 0.0f;
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                if (!in[i]) continue;
                v[i] = read_pairs<W>(n, x, at[i]);
                const Pairs<W> y = read_pairs<W>(n, g, at[i]);
                w[i] = read_pairs<W>(n, weight, at[i]);
#pragma unroll
                for (int e = 0; e < W; ++e) {
                    dn[i].a[e] = y.a[e] * c[i][e] + y.b[e] * s[i][e];
                    dn[i].b[e] = y.b[e] * c[i][e] - y.a[e] * s[i][e];
                    sq += v[i].a[e] * v[i].a[e] + v[i].b[e] * v[i].b[e];
                    dot += dn[i].a[e] * w[i].a[e] * v[i].a[e] +
                           dn[i].b[e] * w[i].b[e] * v[i].b[e];
                }
            }
            const float r = rsqrtf(lanes_sum<G>(sq) * n.inv_d + n.eps);
            const float f = lanes_sum<G>(dot) * n.inv_d * r * r;
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                if (!in[i]) continue;
                Pairs<W> o;
#pragma unroll
                for (int e = 0; e < W; ++e) {
                    o.a[e] = r * (dn[i].a[e] * w[i].a[e] - v[i].a[e] * f);
                    o.b[e] = r * (dn[i].b[e] * w[i].b[e] - v[i].b[e] * f);
                    const float pa = dn[i].a[e] * v[i].a[e] * r, pb = dn[i].b[e] * v[i].b[e] * r;
                    dw[0][i][e] += isq ? pa : 0.0f;
                    dw[0][i][W + e] += isq ? pb : 0.0f;
                    dw[1][i][e] += isq ? 0.0f : pa;
                    dw[1][i][W + e] += isq ? 0.0f : pb;
                }
                write_pairs<W>(n, d, at[i], o);
            }
        }
#pragma unroll
        for (int a = 0; a < 2; ++a)
#pragma unroll
            for (int i = 0; i < NP; ++i)
#pragma unroll
                for (int e = 0; e < 2 * W; ++e) sums[a][i][e] += (double)dw[a][i][e];
    }
    // lanes of one pair, then waves
    __shared__ double wsum[kWaves][2][2 * W * G * NP];
#pragma unroll
    for (int a = 0; a < 2; ++a)
#pragma unroll
        for (int i = 0; i < NP; ++i)
#pragma unroll
            for (int e = 0; e < 2 * W; ++e) {
                double v = sums[a][i][e];
#pragma unroll
                for (int o = G; o < 64; o <<= 1) v += __shfl_xor(v, o, 64);
                if (slot == 0) wsum[wave][a][((i * G + part) * 2 * W) + e] = v;
            }
    __syncthreads();
    for (int j = threadIdx.x; j < 2 * 2 * W * G * NP; j += 64 * kWaves) {
        const int a = j / (2 * W * G * NP), r = j % (2 * W * G * NP);
        const int p = r / (2 * W) * W, e = r % (2 * W);
        if (p >= n.d / 2) continue;
        double v = wsum[0][a][r];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) v += wsum[w][a][r];
        const Place w = place(n, p, W);
        const int d = n.interleaved ? w.first + 2 * (e % W) + e / W : (e < W ? w.first + e : w.second + e - W);
        parts[((int64_t)blockIdx.x * 2 + a) * n.d + d] = v;
    }
}

// The weights' gradients from the workgroups' parts: one workgroup takes 16
// values, each added over every 64th part by one thread and then over the 64
// threads in order.  Eight loads are in flight together, so the up to 512
// parts cost one trip to memory (a thread for every 16th part took 20 us for
// 1024 parts).
__global__ __launch_bounds__(1024) void weight_grads(const double *parts, int nparts, float *dqw, float *dkw, int d) {
    __shared__ double sum[64][16];
    const int c = threadIdx.x & 15, col = blockIdx.x * 16 + c, first = threadIdx.x >> 4;
    double part[kParts / 64];
#pragma unroll
    for (int i = 0; i < kParts / 64; ++i) {
        const int b = first + 64 * i;
        part[i] = col < 2 * d && b < nparts ? parts[(int64_t)b * 2 * d + col] : 0.0;
    }
    double v = 0.0;
#pragma unroll
    for (int i = 0; i < kParts / 64; ++i) v += part[i];
    sum[first][c] = v;
    __syncthreads();
    if (first == 0 && col < 2 * d) {
#pragma unroll
        for (int w = 1; w < 64; ++w) v += sum[w][c];
        (col < d ? dqw[col] : dkw[col - d]) = (float)v;
    }
}

bool vector_access(const attn_norm &n, const attn_tensor *const *t, int count) {
    const int64_t half = n.rotated / 2, rest = n.head_dim / 2 - half;
    if (n.head_dim % 8 || (!n.interleaved && (half % 4 || rest % 4))) return false;
    if (!aligned(n.q_weight, 16) || !aligned(n.k_weight, 16)) return false;
    for (int i = 0; i < count; ++i)
        if (!aligned(t[i]->data, 16) || (n.tokens > 1 && t[i]->token_stride % 4) || t[i]->head_stride % 4) return false;
    return true;
}

int check_norm(const attn_norm &n) {
    if (n.tokens < 0 || n.tokens >= ((int64_t)1 << 30) || n.q_heads < 1 || n.q_heads > 65535 || n.k_heads < 1 ||
        n.k_heads > 65535 || n.head_dim < 2 || n.head_dim > 256 || n.head_dim % 2 || n.rotated < 0 ||
        n.rotated > n.head_dim || n.rotated % 2)
        return GEMM_ERR_SHAPE;
    if ((n.positions64 != 0 && n.positions64 != 1) || (n.interleaved != 0 && n.interleaved != 1) || !(n.eps >= 0.0) ||
        !std::isfinite((float)n.eps))
        return GEMM_ERR_DTYPE;
    if (n.q_weight == nullptr || n.k_weight == nullptr || (n.rotated > 0 && n.inv_freq == nullptr) ||
        (n.tokens > 0 && n.positions == nullptr))
        return GEMM_ERR_NULL;
    if (!aligned(n.positions, n.positions64 ? 8 : 4) || !aligned(n.inv_freq, 4) || !aligned(n.q_weight, 4) ||
        !aligned(n.k_weight, 4))
        return GEMM_ERR_ALIGN;
    return GEMM_OK;
}

int check_view(const View &v, int64_t tokens, int64_t d) {
    if (v.t->data == nullptr) return GEMM_ERR_NULL;
    const int64_t most = (int64_t)1 << 56;  // elements from the first to the last
    if (v.t->token_stride < 0 || v.t->head_stride < 0 || v.t->token_stride > most / std::max<int64_t>(tokens, 1) ||
        v.t->head_stride > most / v.heads)
        return GEMM_ERR_SHAPE;
    if (v.output && !rows_apart(v, tokens, d)) return GEMM_ERR_SHAPE;
    if (!aligned(v.t->data, 4)) return GEMM_ERR_ALIGN;
    return GEMM_OK;
}

// Whether an output overlaps what every thread reads: weights, frequencies, positions.
bool covers_shared(const View &o, const attn_norm &n) {
    const int64_t T = n.tokens, D = n.head_dim;
    return in_range(o, n.q_weight, D * 4, T, D) || in_range(o, n.k_weight, D * 4, T, D) ||
           in_range(o, n.inv_freq, n.rotated * 2, T, D) || in_range(o, n.positions, T * (n.positions64 ? 8 : 4), T, D);
}

Norm device_norm(const attn_norm &a) {
    Norm n;
    n.pos = a.positions;
    n.inv_freq = a.inv_freq;
    n.qw = a.q_weight;
    n.kw = a.k_weight;
    n.tokens = (int)a.tokens;
    n.hq = (int)a.q_heads;
    n.hk = (int)a.k_heads;
    n.d = (int)a.head_dim;
    n.half = (int)a.rotated / 2;
    n.wide = (int)a.positions64;
    n.interleaved = (int)a.interleaved;
    n.eps = (float)a.eps;
    n.inv_d = 1.0f / (float)a.head_dim;
    return n;
}

// Lanes a head: the power of two that holds head_dim / 2 pairs at W a lane.
int lanes_of(int64_t d, int w) {
    int g = 1;
    while (g < 64 && g * w < d / 2) g *= 2;
    return g;
}

// Waves a token's heads are split over, so that a few tokens still fill the
// chip: one token of 40 heads of 128 would take one wave 10 rounds of loads.
int chunks_of(int64_t tokens, int64_t heads, int heads_a_wave) {
    const int64_t rounds = (heads + heads_a_wave - 1) / heads_a_wave;
    return (int)std::max<int64_t>(1, std::min<int64_t>(rounds, 4096 / tokens));
}

// Workgroups of the backward pass with every wave at work.
int64_t backward_groups(int64_t items) { return std::max<int64_t>(1, std::min<int64_t>((items + kWaves - 1) / kWaves, kParts)); }

#define NORM_BY_LANES(LAUNCH)                                                                                 \
    do {                                                                                                      \
        if (vec) {                                                                                            \
            switch (lanes_of(D, 4)) {                                                                         \
                case 1: LAUNCH(4, 1, 1); break;                                                               \
                case 2: LAUNCH(4, 2, 1); break;                                                               \
                case 4: LAUNCH(4, 4, 1); break;                                                               \
                case 8: LAUNCH(4, 8, 1); break;                                                               \
                case 16: LAUNCH(4, 16, 1); break;                                                             \
                default: LAUNCH(4, 32, 1); break;                                                             \
            }                                                                                                 \
        } else if (D <= 128) {                                                                                \
            LAUNCH(1, 64, 1);                                                                                 \
        } else {                                                                                              \
            LAUNCH(1, 64, 2);                                                                                 \
        }                                                                                                     \
    } while (0)

}  // namespace

extern "C" {

int attn_qk_norm_rope(const attn_qk_norm_rope_args *args, void *stream) {
    if (args == nullptr) return GEMM_ERR_NULL;
    const attn_qk_norm_rope_args &a = *args;
    const int64_t T = a.n.tokens, D = a.n.head_dim, HQ = a.n.q_heads, HK = a.n.k_heads;
    int st = check_norm(a.n);
    if (st != GEMM_OK) return st;
    if (T == 0) return GEMM_OK;
    const View q = {&a.q, HQ, false}, k = {&a.k, HK, false}, yq = {&a.q_out, HQ, true}, yk = {&a.k_out, HK, true};
    for (const View *x : {&q, &k, &yq, &yk})
        if ((st = check_view(*x, T, D)) != GEMM_OK) return st;
    if ((!same_tensor(a.q_out, a.q) && overlap(yq, q, T, D)) || (!same_tensor(a.k_out, a.k) && overlap(yk, k, T, D)) ||
        overlap(yq, k, T, D) || overlap(yk, q, T, D) || overlap(yq, yk, T, D) || covers_shared(yq, a.n) ||
        covers_shared(yk, a.n))
        return GEMM_ERR_ALIAS;
    const attn_tensor *all[4] = {&a.q, &a.k, &a.q_out, &a.k_out};
    const bool vec = vector_access(a.n, all, 4);
    const Norm n = device_norm(a.n);
    const Strided sq = strided(a.q, T, HQ), sk = strided(a.k, T, HK), oq = strided(a.q_out, T, HQ),
                  ok = strided(a.k_out, T, HK);
    hipStream_t hs = static_cast<hipStream_t>(stream);
#define FWD(W, G, NP)                                                                                              \
    do {                                                                                                            \
        const int chunks = chunks_of(T, HQ + HK, 64 / G);                                                           \
        st = in_slices((T * chunks + 3) / 4, 256, [&](int64_t first, unsigned count) {                              \
            hipLaunchKernelGGL((qk_norm_rope_fwd<W, G, NP>), dim3(count), dim3(256), 0, hs, n, sq, sk, oq, ok,      \
                               chunks, first);                                                                      \
        });                                                                                                         \
    } while (0)
    NORM_BY_LANES(FWD);
#undef FWD
    return st;
}

int64_t attn_qk_norm_rope_workspace_bytes(int64_t tokens, int64_t head_dim) {
    if (tokens < 0 || tokens >= ((int64_t)1 << 30) || head_dim < 2 || head_dim > 256) return -1;
    return kParts * 2 * head_dim * 8;
}

int attn_qk_norm_rope_backward(const attn_qk_norm_rope_backward_args *args, void *stream) {
    if (args == nullptr) return GEMM_ERR_NULL;
    const attn_qk_norm_rope_backward_args &a = *args;
    const int64_t T = a.n.tokens, D = a.n.head_dim, HQ = a.n.q_heads, HK = a.n.k_heads;
    int st = check_norm(a.n);
    if (st != GEMM_OK) return st;
    if (a.dq_weight == nullptr || a.dk_weight == nullptr || a.workspace == nullptr) return GEMM_ERR_NULL;
    if (!aligned(a.dq_weight, 4) || !aligned(a.dk_weight, 4) || !aligned(a.workspace, 8)) return GEMM_ERR_ALIGN;
    const int64_t need = attn_qk_norm_rope_workspace_bytes(T, D);
    if (a.workspace_bytes < need) return GEMM_ERR_WORKSPACE;
    const View gq = {&a.dq_out, HQ, false}, gk = {&a.dk_out, HK, false}, q = {&a.q, HQ, false}, k = {&a.k, HK, false},
               dq = {&a.dq, HQ, true}, dk = {&a.dk, HK, true};
    if (T > 0) {
        for (const View *x : {&gq, &gk, &q, &k, &dq, &dk})
            if ((st = check_view(*x, T, D)) != GEMM_OK) return st;
        for (const View *o : {&dq, &dk}) {
            for (const View *x : {&gq, &gk, &q, &k}) {
                const bool own = x->t != nullptr && same_tensor(*o->t, *x->t) &&
                                 ((o == &dq) == (x == &gq || x == &q));
                if (!own && overlap(*o, *x, T, D)) return GEMM_ERR_ALIAS;
            }
            if (covers_shared(*o, a.n)) return GEMM_ERR_ALIAS;
        }
        if (overlap(dq, dk, T, D)) return GEMM_ERR_ALIAS;
    }
    // the weights' gradients and the scratch apart from everything else
    const Span small[3] = {{a.dq_weight, D * 4}, {a.dk_weight, D * 4}, {a.workspace, need}};
    const Span shared[4] = {{a.n.q_weight, D * 4}, {a.n.k_weight, D * 4}, {a.n.inv_freq, a.n.rotated * 2},
                            {a.n.positions, T * (a.n.positions64 ? 8 : 4)}};
    for (int i = 0; i < 3; ++i) {
        for (int j = 0; j < i; ++j)
            if (spans_overlap(small[i], small[j])) return GEMM_ERR_ALIAS;
        for (const Span &x : shared)
            if (spans_overlap(small[i], x)) return GEMM_ERR_ALIAS;
        for (const View *x : {&gq, &gk, &q, &k, &dq, &dk})
            if (T > 0 && in_range(*x, small[i].p, small[i].bytes, T, D)) return GEMM_ERR_ALIAS;
    }
    const attn_tensor *all[6] = {&a.dq_out, &a.dk_out, &a.q, &a.k, &a.dq, &a.dk};
    const bool vec = vector_access(a.n, all, 6);
    const Norm n = device_norm(a.n);
    const Strided g0 = strided(a.dq_out, T, HQ), g1 = strided(a.dk_out, T, HK), sq = strided(a.q, T, HQ),
                  sk = strided(a.k, T, HK), o0 = strided(a.dq, T, HQ), o1 = strided(a.dk, T, HK);
    hipStream_t hs = static_cast<hipStream_t>(stream);
    double *parts = static_cast<double *>(a.workspace);
    int grid = 1;
#define BWD(W, G, NP)                                                                                                  \
    do {                                                                                                                \
        const int chunks = T > 0 ? chunks_of(T, HQ + HK, 64 / G) : 1;                                                   \
        grid = (int)backward_groups(T * chunks);                                                                        \
        hipLaunchKernelGGL((qk_norm_rope_bwd<W, G, NP>), dim3(grid), dim3(64 * kWaves), 0, hs, n, g0, g1, sq, sk, o0,  \
                           o1, parts, chunks);                                                                          \
    } while (0)
    NORM_BY_LANES(BWD);
#undef BWD
    hipLaunchKernelGGL(weight_grads, dim3((unsigned)((2 * D + 15) / 16)), dim3(1024), 0, hs, parts, grid, a.dq_weight,
                       a.dk_weight, (int)D);
    return hipGetLastError() == hipSuccess ? GEMM_OK : GEMM_ERR_LAUNCH;
}

}  // extern "C"
