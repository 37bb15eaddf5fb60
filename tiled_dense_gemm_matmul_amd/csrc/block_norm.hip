// The norms around a transformer block in one pass, forward and backward, for
// MI355X (gfx950) (definitions in block_norm.h).
//
// The work is bound by memory: every value is read and written once (forward:
// x and y in, x_out and h out; backward: dx_out, dh, x_out and y in, dx and dy
// out), and a row stays in registers between its sums.  With inputs in no cache
// 7992 rows of 4096 forward run at 5.3 TB/s, where a large copy on this card
// reaches 5.1, and 8192 rows of 768 backward take 36 us, 4.2 TB/s with the
// kernel behind it.  (Other times below are of calls repeated on the same
// arrays, part of which the last-level cache holds: 31 us, 4.9 TB/s, for
// these.)  LANES lanes own a row, each NV groups of 4 consecutive values: a
// wave rows of up to 1024 values, four rows a workgroup, and a workgroup of 256
// or 512 threads wider ones.
//  * Accesses are 16 bytes wide at any 4-byte alignment; where the width is no
//    multiple of 4, one lane takes a row's last values one by one (EX false),
//    behind the loads of all others (8192 rows of 1150 backward 49 us; 69 with
//    the choice inside every load).
//  * The backward pass sums over rows for the weights and the gate.  A
//    workgroup owns a run of rows and keeps its sums in registers (fp32, 64
//    rows a lane at most), the gate's until the sequence ends; it adds those of
//    its four waves, where each has rows of its own, in fp32 (one part a wave
//    would be four times the parts), writes them to parts of its own, and a
//    second kernel adds the parts in fp64.  Part w + b holds workgroup w's sum
//    over sequence b, which no other pair shares: b does not fall as w grows, so
//    w + b grows with every step of either.

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <algorithm>
#include <cmath>

#include "block_norm.h"
#include "gemm_fwd.h"
#include "launch.h"
#include "strided.h"

namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4u __attribute__((ext_vector_type(4), aligned(4)));  // at any 4-byte alignment

struct Matrix {
    float *p;  // NULL: not there
    int64_t st;
};

struct Problem {
    const float *pre, *post, *gate;
    const int *cu;
    int64_t gate_st;  // from one sequence's gate to the next
    int by_seq, nseq, tokens, width;
    float a, b, eps, inv_width;  // a, b: residual_scale, block_scale
};

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
    const int x = __builtin_bit_cast(int, v);
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(x, x, CTRL, 0xf, 0xf, true));
}
// Sum over the wave's lanes, the same in every lane: within quads and rows of
// 16 lanes by permutations of the operand, then across rows by swaps.
__device__ __forceinline__ float wave_sum(float v) {
    v += dpp<0xB1>(v);   // quad_perm 1, 0, 3, 2
    v += dpp<0x4E>(v);   // quad_perm 2, 3, 0, 1
    v += dpp<0x141>(v);  // row_half_mirror
    v += dpp<0x140>(v);  // row_mirror
    unsigned u = __builtin_bit_cast(unsigned, v);
    const auto a = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    v = __builtin_bit_cast(float, (unsigned)a[0]) + __builtin_bit_cast(float, (unsigned)a[1]);
    u = __builtin_bit_cast(unsigned, v);
    const auto b = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    return __builtin_bit_cast(float, (unsigned)b[0]) + __builtin_bit_cast(float, (unsigned)b[1]);
}

// Sums of N values over the lanes of a row.  Over several waves they meet in
// LDS, in one of two places in turn: a wave that is a whole sum ahead has
// passed the barrier that the others left their last reads before.
template <int LANES, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float (*meet)[LANES / 64][4], int &turn) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = wave_sum(v[i]);
    if constexpr (LANES > 64) {
        const int wave = threadIdx.x >> 6;
        if ((threadIdx.x & 63) == 0) {
#pragma unroll
            for (int i = 0; i < N; ++i) meet[turn][wave][i] = v[i];
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float s = meet[turn][0][i];
#pragma unroll
            for (int w = 1; w < LANES / 64; ++w) s += meet[turn][w][i];
            v[i] = s;
        }
        turn ^= 1;
    }
}

// A lane's values of a row, NV groups of 4.
template <int LANES, int NV, bool EX>
struct Row {
    f32x4 x[NV];

    static __device__ __forceinline__ int at(int i) { return 4 * (i * LANES + (int)(threadIdx.x & (LANES - 1))); }
    __device__ __forceinline__ void fill(float v) {
#pragma unroll
        for (int i = 0; i < NV; ++i) x[i] = f32x4{v, v, v, v};
    }
    // zeros past the row's end; a last group of 1 to 3 values (not EX) is
    // always one of the lanes' last groups, and is taken behind all others
    __device__ __forceinline__ void load(const float *row, int width) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            x[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
            if (at(i) + 4 <= width) x[i] = *(const f32x4u *)(row + at(i));
        }
        const int c = at(NV - 1);
        if (!EX && c < width && c + 4 > width) {
            x[NV - 1][0] = row[c];
            if (c + 1 < width) x[NV - 1][1] = row[c + 1];
            if (c + 2 < width) x[NV - 1][2] = row[c + 2];
        }
    }
    __device__ __forceinline__ void store(float *row, int width) const {
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (at(i) + 4 <= width) *(f32x4u *)(row + at(i)) = x[i];
        const int c = at(NV - 1);
        if (!EX && c < width && c + 4 > width) {
            row[c] = x[NV - 1][0];
            if (c + 1 < width) row[c + 1] = x[NV - 1][1];
            if (c + 2 < width) row[c + 2] = x[NV - 1][2];
        }
    }
};
template <int NV>
__device__ __forceinline__ float dot(const f32x4 (&a)[NV], const f32x4 (&b)[NV]) {
    f32x4 s = a[0] * b[0];
#pragma unroll
    for (int i = 1; i < NV; ++i) s += a[i] * b[i];
    return (s[0] + s[1]) + (s[2] + s[3]);
}

__device__ __forceinline__ int bound(const Problem &p, int b) { return min(max(p.cu[b], 0), p.tokens); }

// The last sequence that starts at row t or before, for a t inside
// [cu_seqlens[0], cu_seqlens[nseq]): the wave looks at 64 bounds at once.
__device__ __forceinline__ int sequence_of(const Problem &p, int t) {
    const int lane = threadIdx.x & 63;
    int lo = 0, hi = p.nseq, step;
    do {  // of [lo, hi), the last sequence that starts at t or before
        step = (hi - lo + 63) / 64;
        const int b = lo + lane * step;
        const int below = __popcll(__ballot(b < hi && bound(p, min(b, p.nseq)) <= t));
        lo += max(below - 1, 0) * step;
        hi = min(lo + step, hi);
    } while (step > 1);
    return uniform(lo);
}

// The sequences that a run of rows meets, one after the other: the wave holds
// the next 64 bounds, so that only every 64th sequence is searched for.
struct Sequences {
    int first = 0, bounds = 0x7fffffff;  // of sequence first + lane; none is known yet

    __device__ __forceinline__ void look(const Problem &p, int t) {
        first = sequence_of(p, t);
        bounds = bound(p, min(first + (int)(threadIdx.x & 63), p.nseq));
    }
    // The sequence of row t, which is no less than the last one's, and the row
    // behind it.
    __device__ __forceinline__ void find(const Problem &p, int t, int &seq, int &end) {
        auto below = [&]() {
            return __popcll(__ballot(first + (int)(threadIdx.x & 63) < p.nseq && bounds <= t));
        };
        int n = below();
        if (n == 0 || n == 64) {
            look(p, t);
            n = below();
        }
        seq = first + max(n - 1, 0);
        end = n < 64 ? __builtin_amdgcn_readlane(bounds, n) : uniform(bound(p, seq + 1));
    }
};

// The rows that belong to sequences.
struct Used {
    int first, last;
};
__device__ __forceinline__ Used used_rows(const Problem &p) {
    if (!p.cu) return {0, p.tokens};
    const int first = uniform(bound(p, 0));
    return {first, max(first, uniform(bound(p, p.nseq)))};
}

// --- forward ---

template <int LANES, int NV, bool EX>
__global__ __launch_bounds__(LANES < 256 ? 256 : LANES) void block_norm_fwd(Problem p, Matrix x, Matrix y, Matrix x_out,
                                                                          Matrix h, int64_t first) {
    constexpr int ROWS = LANES < 256 ? 256 / LANES : 1;  // of a workgroup
    typedef Row<LANES, NV, EX> R;
    __shared__ float meet[2][LANES / 64][4];
    int turn = 0;
    const int64_t t64 = (first + blockIdx.x) * ROWS + uniform(threadIdx.x / LANES);
    if (t64 >= p.tokens) return;
    const int t = (int)t64;
    const Used used = used_rows(p);
    if (t < used.first || t >= used.last) {
        R zero;
        zero.fill(0.0f);
        if (x_out.p) zero.store(x_out.p + t * x_out.st, p.width);
        if (h.p) zero.store(h.p + t * h.st, p.width);
        return;
    }
    R v;
    v.load(x.p + t * x.st, p.width);
    if (y.p) {
        R n, w;
        n.load(y.p + t * y.st, p.width);
        if (p.post) {
            w.load(p.post, p.width);
            float s[1] = {dot(n.x, n.x)};
            row_sums<LANES>(s, meet, turn);
            const float r = rsqrtf(s[0] * p.inv_width + p.eps);
#pragma unroll
            for (int i = 0; i < NV; ++i) n.x[i] = n.x[i] * r * w.x[i];
        }
        if (p.gate) {
            w.load(p.gate + (p.by_seq ? sequence_of(p, t) * p.gate_st : 0), p.width);
#pragma unroll
            for (int i = 0; i < NV; ++i) n.x[i] *= w.x[i];
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) v.x[i] = p.a * v.x[i] + p.b * n.x[i];
        v.store(x_out.p + t * x_out.st, p.width);
    }
    if (p.pre) {
        R w;
        w.load(p.pre, p.width);
        float s[1] = {dot(v.x, v.x)};
        row_sums<LANES>(s, meet, turn);
        const float r = rsqrtf(s[0] * p.inv_width + p.eps);
#pragma unroll
        for (int i = 0; i < NV; ++i) w.x[i] = v.x[i] * r * w.x[i];
        w.store(h.p + t * h.st, p.width);
    }
}

// --- backward ---

struct Backward {
    Matrix dx_out, dh, x_out, y, dx, dy;
    float *pre_parts, *post_parts, *gate_parts;  // rows of `pitch` floats
    int pitch;
};

// A lane's sums, added over the workgroup's rows in order, into row `part`.
template <int LANES, int NV, bool EX>
__device__ __forceinline__ void write_part(const Row<LANES, NV, EX> &sum, float *part, int pitch, f32x4 *meet) {
    if constexpr (LANES < 256) {
        constexpr int ROWS = 256 / LANES;
        __syncthreads();  // the buffer's last readers
#pragma unroll
        for (int i = 0; i < NV; ++i) meet[threadIdx.x / LANES * (NV * LANES) + i * LANES + threadIdx.x % LANES] = sum.x[i];
        __syncthreads();
        for (int j = threadIdx.x; j < NV * LANES; j += 256) {
            if (4 * j >= pitch) break;
            f32x4 s = meet[j];
#pragma unroll
            for (int r = 1; r < ROWS; ++r) s += meet[r * NV * LANES + j];
            *(f32x4 *)(part + 4 * j) = s;
        }
    } else {
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (sum.at(i) < pitch) *(f32x4 *)(part + sum.at(i)) = sum.x[i];
    }
}

template <int LANES, int NV, bool EX>
__global__ __launch_bounds__(LANES < 256 ? 256 : LANES, 2) void block_norm_bwd(Problem p, Backward a, int chunk,
                                                                             int64_t first) {
    constexpr int ROWS = LANES < 256 ? 256 / LANES : 1;
    typedef Row<LANES, NV, EX> R;
    __shared__ float meet[2][LANES / 64][4];
    __shared__ __align__(16) f32x4 joined[LANES < 256 ? NV * 256 : 1];
    int turn = 0;
    const int64_t group = first + blockIdx.x;
    const int t0 = (int)(group * chunk), t1 = min(t0 + chunk, p.tokens);
    const int mine = uniform(threadIdx.x / LANES);
    const Used used = used_rows(p);
    const bool by_seq = p.gate && p.by_seq;
    R pre, post, gate, dpre, dpost, dgate;
    dpre.fill(0.0f);
    dpost.fill(0.0f);
    dgate.fill(0.0f);
    pre.fill(1.0f);
    post.fill(1.0f);
    gate.fill(1.0f);
    if (p.pre) pre.load(p.pre, p.width);
    if (p.post) post.load(p.post, p.width);
    if (p.gate && !by_seq) gate.load(p.gate, p.width);
    Sequences sequences;
    for (int row = t0; row < t1;) {
        int end = t1, seq = 0;
        const bool in = row >= used.first && row < used.last;
        if (!in) {
            if (row < used.first) end = min(t1, used.first);
        } else {
            end = min(t1, used.last);
            if (by_seq) {
                int behind;
                sequences.find(p, row, seq, behind);
                end = min(end, max(row + 1, behind));
                gate.load(p.gate + seq * p.gate_st, p.width);
            }
        }
        // a workgroup's rows go to its waves in turn
        int t = row + (mine + ROWS - (row - t0) % ROWS) % ROWS;
        for (; t < end; t += ROWS) {
            if (!in) {
                R zero;
                zero.fill(0.0f);
                zero.store(a.dx.p + t * a.dx.st, p.width);
                if (a.dy.p) zero.store(a.dy.p + t * a.dy.st, p.width);
                continue;
            }
            R d, g, x, y;
            d.fill(0.0f);
            if (a.dx_out.p) d.load(a.dx_out.p + t * a.dx_out.st, p.width);
            if (p.pre) {
                x.load(a.x_out.p + t * a.x_out.st, p.width);
                g.load(a.dh.p + t * a.dh.st, p.width);
            }
            if (a.y.p) y.load(a.y.p + t * a.y.st, p.width);
            float s[3] = {0.0f, 0.0f, 0.0f};
            if (p.pre) {
                s[0] = dot(x.x, x.x);
                f32x4 w[NV];
#pragma unroll
                for (int i = 0; i < NV; ++i) w[i] = g.x[i] * pre.x[i];
                s[1] = dot(w, x.x);
            }
            if (p.post) s[2] = dot(y.x, y.x);
            row_sums<LANES>(s, meet, turn);
            if (p.pre) {
                const float r = rsqrtf(s[0] * p.inv_width + p.eps), f = s[1] * p.inv_width * r * r;
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    d.x[i] += r * (g.x[i] * pre.x[i] - x.x[i] * f);
                    dpre.x[i] += g.x[i] * x.x[i] * r;
                }
            }
#pragma unroll
            for (int i = 0; i < NV; ++i) g.x[i] = p.a * d.x[i];
            g.store(a.dx.p + t * a.dx.st, p.width);
            if (!a.y.p) continue;
#pragma unroll
            for (int i = 0; i < NV; ++i) d.x[i] *= p.b;
            const float r = p.post ? rsqrtf(s[2] * p.inv_width + p.eps) : 1.0f;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const f32x4 n = y.x[i] * r;
                if (p.gate) {
                    dgate.x[i] += d.x[i] * n * post.x[i];
                    d.x[i] *= gate.x[i];
                }
                if (p.post) {
                    dpost.x[i] += d.x[i] * n;
                    d.x[i] *= post.x[i];
                }
            }
            if (p.post) {
                float m[1] = {dot(d.x, y.x)};
                row_sums<LANES>(m, meet, turn);
                const float f = m[0] * p.inv_width * r * r;
#pragma unroll
                for (int i = 0; i < NV; ++i) d.x[i] = r * (d.x[i] - y.x[i] * f);
            }
            d.store(a.dy.p + t * a.dy.st, p.width);
        }
        if (in && by_seq) {
            write_part(dgate, a.gate_parts + (group + seq) * a.pitch, a.pitch, joined);
            dgate.fill(0.0f);
        }
        row = end;
    }
    if (p.pre) write_part(dpre, a.pre_parts + group * a.pitch, a.pitch, joined);
    if (p.post) write_part(dpost, a.post_parts + group * a.pitch, a.pitch, joined);
    if (p.gate && !by_seq) write_part(dgate, a.gate_parts + group * a.pitch, a.pitch, joined);
}

// The parts' sums: a workgroup takes 64 columns of one result, a thread 4 of
// them over every EACH-th part, joined in order.  Results are numbered dpre_weight,
// dpost_weight, then the gate's rows, those that the call has.
struct Sums {
    const float *pre_parts, *post_parts, *gate_parts;
    float *dpre, *dpost, *dgate;
    int64_t dgate_st;
    int pitch, groups, chunk;
};
template <int EACH>
__global__ __launch_bounds__(16 * EACH) void block_norm_sums(Problem p, Sums a, int tiles, int64_t first) {
    const int64_t id = first + blockIdx.x;
    int64_t job = id / tiles;
    const int c = (int)(id % tiles) * 64 + 4 * (threadIdx.x & 15), part = threadIdx.x >> 4;
    const float *parts;
    float *to;
    int64_t lo = 0, hi = a.groups;
    if (p.pre && job-- == 0) {
        parts = a.pre_parts;
        to = a.dpre;
    } else if (p.post && job-- == 0) {
        parts = a.post_parts;
        to = a.dpost;
    } else {
        parts = a.gate_parts;
        to = a.dgate + job * a.dgate_st;
        if (p.by_seq) {
            const int s0 = max(bound(p, (int)job), bound(p, 0)), s1 = min(bound(p, (int)job + 1), bound(p, p.nseq));
            lo = s0 / a.chunk + job;
            hi = s1 > s0 ? (s1 - 1) / a.chunk + job + 1 : lo;
        }
    }
    double s[4] = {0.0, 0.0, 0.0, 0.0};
    if (c < p.width) {
#pragma unroll EACH == 64 ? 8 : 4
        for (int64_t i = lo + part; i < hi; i += EACH) {
            const f32x4 v = *(const f32x4 *)(parts + i * a.pitch + c);
#pragma unroll
            for (int e = 0; e < 4; ++e) s[e] += (double)v[e];
        }
    }
    __shared__ double meet[EACH][64];
#pragma unroll
    for (int e = 0; e < 4; ++e) meet[part][4 * (threadIdx.x & 15) + e] = s[e];
    __syncthreads();
    const int mine = threadIdx.x, col = (int)(id % tiles) * 64 + mine;
    if (mine < 64 && col < p.width) {
        double v = meet[0][mine];
#pragma unroll
        for (int w = 1; w < EACH; ++w) v += meet[w][mine];
        to[col] = (float)v;
    }
}

// --- host ---

constexpr int64_t kMost = (int64_t)1 << 56;  // elements from the first to the last
constexpr int64_t kMaxTokens = (int64_t)1 << 30, kMaxWidth = 8192, kMaxSeqs = (int64_t)1 << 24;

int check_problem(const block_norm_problem &p) {
    if (p.tokens < 0 || p.tokens >= kMaxTokens || p.width < 1 || p.width > kMaxWidth) return GEMM_ERR_SHAPE;
    if (p.cu_seqlens && (p.num_seqs < 0 || p.num_seqs >= kMaxSeqs)) return GEMM_ERR_SHAPE;
    if ((p.gate_by_sequence != 0 && p.gate_by_sequence != 1) || !std::isfinite((float)p.residual_scale) ||
        !std::isfinite((float)p.block_scale) || !(p.eps >= 0.0) || !std::isfinite((float)p.eps))
        return GEMM_ERR_DTYPE;
    if (p.gate && p.gate_by_sequence && !p.cu_seqlens) return GEMM_ERR_NULL;
    if (p.gate && p.gate_by_sequence && p.num_seqs > 1 && (p.gate_stride < 0 || p.gate_stride > kMost / p.num_seqs))
        return GEMM_ERR_SHAPE;
    if (!aligned(p.pre_weight, 4) || !aligned(p.post_weight, 4) || !aligned(p.gate, 4) || !aligned(p.cu_seqlens, 4))
        return GEMM_ERR_ALIGN;
    return GEMM_OK;
}

// A matrix as the checks of strided.h take it: one head of `width` values a token.
struct Rows {
    attn_tensor t;
    bool output;
    explicit Rows(const block_rows &r, bool out = false) : t{r.data, r.row_stride, 0}, output(out) {}
    View view() const { return {&t, 1, output}; }
    bool there() const { return t.data != nullptr; }
};

int check_rows(const Rows &r, int64_t tokens, int64_t width) {
    if (r.t.token_stride < 0 || r.t.token_stride > kMost / std::max<int64_t>(tokens, 1)) return GEMM_ERR_SHAPE;
    if (r.output && !rows_apart(r.view(), tokens, width)) return GEMM_ERR_SHAPE;
    return aligned(r.t.data, 4) ? GEMM_OK : GEMM_ERR_ALIGN;
}

int64_t cu_bytes(const block_norm_problem &p) { return p.cu_seqlens ? (p.num_seqs + 1) * 4 : 0; }
// Rows of the gate, and what they span `stride` elements apart.
int64_t gate_rows(const block_norm_problem &p) { return !p.gate ? 0 : p.gate_by_sequence ? p.num_seqs : 1; }
int64_t gate_bytes(const block_norm_problem &p, int64_t stride) {
    const int64_t rows = gate_rows(p);
    return rows > 0 ? ((rows - 1) * stride + p.width) * 4 : 0;
}

// Whether an output overlaps what all rows share.
bool covers_shared(const Rows &o, const block_norm_problem &p) {
    const View v = o.view();
    const int64_t T = p.tokens, W = p.width;
    return in_range(v, p.pre_weight, W * 4, T, W) || in_range(v, p.post_weight, W * 4, T, W) ||
           in_range(v, p.gate, gate_bytes(p, p.gate_stride), T, W) || in_range(v, p.cu_seqlens, cu_bytes(p), T, W);
}

// Whether an output overlaps an input without being the very same matrix.
bool clash(const Rows &o, const Rows &in, const block_norm_problem &p) {
    if (!o.there() || !in.there()) return false;
    const bool same = o.t.data == in.t.data && (p.tokens <= 1 || o.t.token_stride == in.t.token_stride);
    return !same && overlap(o.view(), in.view(), p.tokens, p.width);
}

Matrix matrix(const block_rows &r) { return {static_cast<float *>(r.data), r.row_stride}; }

Problem device_problem(const block_norm_problem &a) {
    Problem p;
    p.pre = a.pre_weight;
    p.post = a.post_weight;
    p.gate = a.gate;
    p.cu = a.cu_seqlens;
    p.by_seq = (int)a.gate_by_sequence;
    p.gate_st = a.gate_stride;
    p.nseq = a.cu_seqlens ? (int)a.num_seqs : 1;
    p.tokens = (int)a.tokens;
    p.width = (int)a.width;
    p.a = (float)a.residual_scale;
    p.b = (float)a.block_scale;
    p.eps = (float)a.eps;
    p.inv_width = 1.0f / (float)a.width;
    return p;
}

// Lanes of a row: as few as hold it, 16 values each.  More values a lane were
// a little faster over many rows and slower over few (a wave of 5 or 6 groups
// a lane against 256 lanes of 2, us: 8192 rows of 1152 forward 23.3 and 24.4,
// backward 42.5 and 43.3; 1001 rows of 1150 forward 6.8 and 5.9; 2000 rows of
// 1536 backward 29.4 and 21.4).
int lanes_of(int64_t width) { return width <= 1024 ? 64 : width <= 4096 ? 256 : 512; }

// Rows of a workgroup of the backward pass.  Enough workgroups to fill the
// chip, but no more than that, as each writes parts that are read again; and
// 64 rows a lane at most, which bounds the fp32 sums.  Narrow rows take more of
// them, wide ones, of 512 threads, fewer: us with 256, 512 and 1024, 16384 rows
// of 128: -, 18.5, 16.6 (2048: 20.0); 8192 rows of 768: -, 30.2, 32.8; 4096
// rows of 2048: 43.5, 38.7, -; of 4096: 89.1, 93.1, -; of 4100: 94.5, 99.4, -;
// of 8192: 172, 181, -.
int64_t chunk_of(const block_norm_problem &p) {
    const int64_t rows = std::max<int64_t>(1, 256 / lanes_of(p.width));
    const int64_t most = p.width <= 256 ? 1024 : p.width <= 4096 ? 512 : 256;
    const int64_t each = (p.tokens + most * rows - 1) / (most * rows);
    return rows * std::min<int64_t>(std::max<int64_t>(each, 1), 64);
}

struct Parts {
    int64_t pitch, chunk, groups, gate_rows;
    int64_t bytes(const block_norm_problem &p) const {
        return ((p.pre_weight ? groups : 0) + (p.post_weight ? groups : 0) + gate_rows) * pitch * 4;
    }
};
Parts parts_of(const block_norm_problem &p) {
    Parts r;
    r.pitch = (p.width + 3) / 4 * 4;
    r.chunk = chunk_of(p);
    r.groups = (p.tokens + r.chunk - 1) / r.chunk;
    r.gate_rows = p.gate ? r.groups + (p.gate_by_sequence ? p.num_seqs : 0) : 0;
    return r;
}

// Groups of 4 values a lane: 1 to 4 of 64 lanes, and as many as the widths of
// more lanes, which begin where fewer are full, need.
#define BLOCK_BY_WIDTH(LAUNCH)                                      \
    do {                                                            \
        const int lanes_ = lanes_of(W);                             \
        const int nv_ = (int)((W + 4 * lanes_ - 1) / (4 * lanes_)); \
        if (lanes_ == 64) {                                         \
            if (nv_ == 1) BLOCK_BY_ODD(LAUNCH, 64, 1);              \
            else if (nv_ == 2) BLOCK_BY_ODD(LAUNCH, 64, 2);         \
            else if (nv_ == 3) BLOCK_BY_ODD(LAUNCH, 64, 3);         \
            else BLOCK_BY_ODD(LAUNCH, 64, 4);                       \
        } else if (lanes_ == 256) {                                 \
            if (nv_ == 2) BLOCK_BY_ODD(LAUNCH, 256, 2);             \
            else if (nv_ == 3) BLOCK_BY_ODD(LAUNCH, 256, 3);        \
            else BLOCK_BY_ODD(LAUNCH, 256, 4);                      \
        } else {                                                    \
            if (nv_ == 3) BLOCK_BY_ODD(LAUNCH, 512, 3);             \
            else BLOCK_BY_ODD(LAUNCH, 512, 4);                      \
        }                                                           \
    } while (0)
#define BLOCK_BY_ODD(LAUNCH, LANES, NV)             \
    do {                                            \
        if (W % 4 == 0) LAUNCH(LANES, NV, true);    \
        else LAUNCH(LANES, NV, false);              \
    } while (0)

}  // namespace

extern "C" {

int block_norm(const block_norm_args *args, void *stream) {
    if (args == nullptr) return GEMM_ERR_NULL;
    const block_norm_args &a = *args;
    const int64_t T = a.p.tokens, W = a.p.width;
    int st = check_problem(a.p);
    if (st != GEMM_OK) return st;
    const Rows x(a.x), y(a.y), xo(a.x_out, true), h(a.h, true);
    if (T == 0) return GEMM_OK;
    if (!y.there() && (xo.there() || a.p.post_weight || a.p.gate)) return GEMM_ERR_SHAPE;
    if (!a.p.pre_weight && h.there()) return GEMM_ERR_SHAPE;
    if (!y.there() && (a.p.residual_scale != 1.0 || a.p.block_scale != 1.0)) return GEMM_ERR_DTYPE;
    if (!y.there() && !a.p.pre_weight) return GEMM_ERR_NULL;
    if (!x.there() || (y.there() && !xo.there()) || (a.p.pre_weight && !h.there())) return GEMM_ERR_NULL;
    for (const Rows *r : {&x, &y, &xo, &h})
        if (r->there() && (st = check_rows(*r, T, W)) != GEMM_OK) return st;
    if (xo.there() && h.there() && overlap(xo.view(), h.view(), T, W)) return GEMM_ERR_ALIAS;
    for (const Rows *o : {&xo, &h})
        if (o->there() && (clash(*o, x, a.p) || clash(*o, y, a.p) || covers_shared(*o, a.p))) return GEMM_ERR_ALIAS;
    const Problem p = device_problem(a.p);
    const Matrix mx = matrix(a.x), my = matrix(a.y), mxo = matrix(a.x_out), mh = matrix(a.h);
    hipStream_t hs = static_cast<hipStream_t>(stream);
#define FWD(LANES, NV, EX)                                                                                          \
    do {                                                                                                             \
        constexpr int threads = LANES < 256 ? 256 : LANES, rows = threads / LANES;                                   \
        st = in_slices((T + rows - 1) / rows, threads, [&](int64_t first, unsigned count) {                          \
            hipLaunchKernelGGL((block_norm_fwd<LANES, NV, EX>), dim3(count), dim3(threads), 0, hs, p, mx, my, mxo,   \
                               mh, first);                                                                           \
        });                                                                                                          \
    } while (0)
    BLOCK_BY_WIDTH(FWD);
#undef FWD
    return st;
}

int64_t block_norm_backward_workspace_bytes(const block_norm_problem *problem) {
    if (problem == nullptr || check_problem(*problem) != GEMM_OK) return -1;
    return parts_of(*problem).bytes(*problem);
}

int block_norm_backward(const block_norm_backward_args *args, void *stream) {
    if (args == nullptr) return GEMM_ERR_NULL;
    const block_norm_backward_args &a = *args;
    const int64_t T = a.p.tokens, W = a.p.width;
    int st = check_problem(a.p);
    if (st != GEMM_OK) return st;
    const Rows dxo(a.dx_out), dh(a.dh), xo(a.x_out), y(a.y), dx(a.dx, true), dy(a.dy, true);
    if (!y.there() && T > 0 && (dy.there() || a.p.post_weight || a.p.gate)) return GEMM_ERR_SHAPE;
    if ((!a.p.pre_weight && (dh.there() || a.dpre_weight)) || (!a.p.post_weight && a.dpost_weight) ||
        (!a.p.gate && a.dgate))
        return GEMM_ERR_SHAPE;
    if (!y.there() && T > 0 && (a.p.residual_scale != 1.0 || a.p.block_scale != 1.0)) return GEMM_ERR_DTYPE;
    const int64_t gates = gate_rows(a.p);
    if (gates > 1 && (a.dgate_stride < W || a.dgate_stride > kMost / gates)) return GEMM_ERR_SHAPE;
    if ((a.p.pre_weight && !a.dpre_weight) || (a.p.post_weight && !a.dpost_weight) || (gates > 0 && !a.dgate))
        return GEMM_ERR_NULL;
    if (T > 0 && (!dx.there() || (y.there() && !dy.there()) || (a.p.pre_weight && (!dh.there() || !xo.there())) ||
                  (!a.p.pre_weight && (!dxo.there() || !y.there()))))
        return GEMM_ERR_NULL;
    if (!aligned(a.dpre_weight, 4) || !aligned(a.dpost_weight, 4) || !aligned(a.dgate, 4)) return GEMM_ERR_ALIGN;
    const Parts parts = parts_of(a.p);
    const int64_t need = parts.bytes(a.p);
    if (need > 0 && (a.workspace == nullptr || a.workspace_bytes < need)) return GEMM_ERR_WORKSPACE;
    if (!aligned(a.workspace, 16)) return GEMM_ERR_ALIGN;
    // the sums and the scratch apart from one another and from everything else
    const Span sums[4] = {{a.dpre_weight, W * 4}, {a.dpost_weight, W * 4}, {a.dgate, gate_bytes(a.p, a.dgate_stride)}, {a.workspace, need}};
    const Span shared[4] = {{a.p.pre_weight, W * 4}, {a.p.post_weight, W * 4}, {a.p.gate, gate_bytes(a.p, a.p.gate_stride)},
                            {a.p.cu_seqlens, cu_bytes(a.p)}};
    const Rows *all[6] = {&dxo, &dh, &xo, &y, &dx, &dy};
    if (T > 0) {
        for (const Rows *r : all)
            if (r->there() && (st = check_rows(*r, T, W)) != GEMM_OK) return st;
        if (dy.there() && overlap(dx.view(), dy.view(), T, W)) return GEMM_ERR_ALIAS;
        for (const Rows *o : {&dx, &dy}) {
            if (!o->there()) continue;
            for (const Rows *in : {&dxo, &dh, &xo, &y})
                if (clash(*o, *in, a.p)) return GEMM_ERR_ALIAS;
            if (covers_shared(*o, a.p)) return GEMM_ERR_ALIAS;
        }
    }
    for (int i = 0; i < 4; ++i) {
        for (int j = 0; j < i; ++j)
            if (spans_overlap(sums[i], sums[j])) return GEMM_ERR_ALIAS;
        for (const Span &s : shared)
            if (spans_overlap(sums[i], s)) return GEMM_ERR_ALIAS;
        for (const Rows *r : all)
            if (T > 0 && r->there() && sums[i].bytes > 0 && in_range(r->view(), sums[i].p, sums[i].bytes, T, W))
                return GEMM_ERR_ALIAS;
    }
    const Problem p = device_problem(a.p);
    float *ws = static_cast<float *>(a.workspace);
    Backward b = {matrix(a.dx_out), matrix(a.dh), matrix(a.x_out), matrix(a.y), matrix(a.dx), matrix(a.dy), ws, ws, ws,
                  (int)parts.pitch};
    if (p.pre) b.post_parts = b.gate_parts = ws + parts.groups * parts.pitch;
    if (p.post) b.gate_parts = b.post_parts + parts.groups * parts.pitch;
    hipStream_t hs = static_cast<hipStream_t>(stream);
#define BWD(LANES, NV, EX)                                                                                           \
    do {                                                                                                              \
        constexpr int threads = LANES < 256 ? 256 : LANES;                                                            \
        st = in_slices(parts.groups, threads, [&](int64_t first, unsigned count) {                                    \
            hipLaunchKernelGGL((block_norm_bwd<LANES, NV, EX>), dim3(count), dim3(threads), 0, hs, p, b,              \
                               (int)parts.chunk, first);                                                              \
        });                                                                                                           \
    } while (0)
    BLOCK_BY_WIDTH(BWD);
#undef BWD
    if (st != GEMM_OK) return st;
    const Sums s = {b.pre_parts, b.post_parts, b.gate_parts, a.dpre_weight, a.dpost_weight, a.dgate,
                    a.dgate_stride, (int)parts.pitch, (int)parts.groups, (int)parts.chunk};
    const int64_t jobs = (p.pre ? 1 : 0) + (p.post ? 1 : 0) + gates, tiles = (W + 63) / 64;
    // Many parts of few results: four times the threads, each with its loads in
    // flight at once (8192 rows of 768: 30.2 us for the whole pass and 31.3; 512
    // rows, 128 parts: 9.0 and 8.5; gates of 2048 sequences: 132 and 56).
    if (parts.groups >= 256 && jobs * tiles <= 512)
        return in_slices(jobs * tiles, 1024, [&](int64_t first, unsigned count) {
            hipLaunchKernelGGL(block_norm_sums<64>, dim3(count), dim3(1024), 0, hs, p, s, (int)tiles, first);
        });
    return in_slices(jobs * tiles, 256, [&](int64_t first, unsigned count) {
        hipLaunchKernelGGL(block_norm_sums<16>, dim3(count), dim3(256), 0, hs, p, s, (int)tiles, first);
    });
}

}  // extern "C"
