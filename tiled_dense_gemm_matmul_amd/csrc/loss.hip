// Fused loss kernels for MI355X (gfx950): cross_entropy (loss + in-place
// dLogits, label smoothing and z-loss) and sum_losses, as defined on the page
// "cross_entropy ve sum_losses — Fused Loss + dLogits"
// (https://llm.istanbul/learn/tr/07_loss), sections "Ne Yapar?" and "Satır
// Satır".
//
// The work is HBM-bound: every logit is read and its gradient written, so
// the ideal is one read and one write of the [S x V] array.  The page reads
// each row three times (max, sum, gradient); here a workgroup of 256 to 1024
// threads keeps its whole row in registers (16 to 64 values per thread: rows
// of up to 65536 logits with 16-byte accesses, 16384 with 4-byte ones), so
// the row is read from memory once.  With 16-byte accesses the workgroup is
// sized to the row: 256 x 16 up to 4096 logits, 512 x 16 up to 8192,
// 512 x 32 up to 16384, 1024 x 32 up to 32768, 1024 x 64 beyond (the fewer
// idle register slots, the more rows in flight per CU: 512 x 16384 logits in
// 10.1 against 12.2 us on 256 x 64, 2048 x 4096 in 10.1 against 21.0).
// Longer rows fall back to the page's streaming order.
//  * Loads are 16-byte buffer loads when V % 4 == 0 and the array is 16-byte
//    aligned, else 4-byte loads; both coalesced along the row.  Elements past
//    V come back as zeros from the buffer's range check and are masked out of
//    the reductions by their index.
//  * Reductions: a butterfly over the 64 lanes of a wave, then the waves'
//    partials in a fixed order from LDS.  Each reduction has its own LDS
//    slots, so consecutive reductions need no trailing barrier.
//  * exp(l - max) is computed once per element and kept for the gradient.
//  * Logit arrays of 256 MiB or more (past the Infinity Cache) are read and
//    written with the non-temporal cache policy; smaller ones, which the cache
//    can hold, keep the default.

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <cmath>
#include <initializer_list>
#include <type_traits>
#include <utility>

#include "distill.h"
#include "gemm_fwd.h"
#include "launch.h"
#include "loss.h"

namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int u32x4v __attribute__((vector_size(16)));
typedef __amdgpu_buffer_rsrc_t Rsrc;
constexpr int kOOB = (int)0x80000000u;
constexpr int kNonTemporal = 2;                       // buffer-access cache policy: nt
constexpr int64_t kStreamBytes = (int64_t)256 << 20;  // arrays past the Infinity Cache

__device__ __forceinline__ Rsrc row_rsrc(const void *base, int bytes) {
    const uint64_t b = reinterpret_cast<uint64_t>(base);
    const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(b));
    const uint32_t hi = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(b >> 32));
    void *ub = reinterpret_cast<void *>((static_cast<uint64_t>(hi) << 32) | lo);
    return __builtin_amdgcn_make_buffer_rsrc(ub, (short)0, __builtin_amdgcn_readfirstlane(bytes), 0x00020000);
}

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor(v, o, 64));
    return v;
}
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
    return v;
}

// Workgroup reduction into every thread: wave butterflies, then the NW wave
// partials added (or maxed) in wave order from `slots`.
template <int NW, bool MAX>
__device__ __forceinline__ float block_reduce(float v, float *slots) {
    v = MAX ? wave_max(v) : wave_sum(v);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    if (lane == 0) slots[wave] = v;
    __syncthreads();
    float r = slots[0];
#pragma unroll
    for (int w = 1; w < NW; ++w) r = MAX ? fmaxf(r, slots[w]) : r + slots[w];
    return r;
}

// The loss of one row from its reductions (the page's phase 3).
__device__ __forceinline__ float row_loss(float lse, float l_t, float mean_l, float alpha, float beta) {
    return (lse - (1.0f - alpha) * l_t - alpha * mean_l) + beta * lse * lse;
}

// One workgroup per row, the row held in registers: CAP values per thread,
// in groups of W consecutive elements (W = 4 with 16-byte accesses).  Group
// j of thread t covers elements [(j NT + t) W, +W); a group past the row end
// is fetched and stored at an offset past the buffer's range, so its loads
// return zeros and its stores are dropped, and it is left out of the
// reductions by comparing j with the thread's count of valid groups.
template <int NT, int CAP, bool VEC, bool STREAM>
__global__ __launch_bounds__(NT) void cross_entropy_resident(float *logits, const uint32_t *tgts, float *losses,
                                                             int V, float alpha, float beta, float inv_norm) {
    constexpr int NW = NT / 64;
    constexpr int W = VEC ? 4 : 1;
    constexpr int G = CAP / W;
    constexpr int POL = STREAM ? kNonTemporal : 0;  // cache policy of the row's loads and stores
    __shared__ float red[3][NW];
    const int tid = threadIdx.x;
    const int s = blockIdx.x;
    float *row = logits + (size_t)s * V;
    const Rsrc rr = row_rsrc(row, V * 4);
    const uint32_t tgt = tgts[s];
    auto off = [&](int j) { return (j * NT + tid) * (W * 4); };
    if (tgt >= (uint32_t)V) {
        // ignored row: zero loss, zero gradient (nothing to read)
        if (tid == 0) losses[s] = 0.0f;
#pragma unroll
        for (int j = 0; j < G; ++j) {
            if (VEC) __builtin_amdgcn_raw_buffer_store_b128(u32x4v{0u, 0u, 0u, 0u}, rr, off(j), 0, POL);
            else __builtin_amdgcn_raw_buffer_store_b32(0u, rr, off(j), 0, POL);
        }
        return;
    }
    const int ng = V / W;                                   // groups in the row
    const int nv = ng > tid ? min(G, (ng - tid + NT - 1) / NT) : 0;  // this thread's valid groups
    float x[CAP];
#pragma unroll
    for (int j = 0; j < G; ++j) {
        if (VEC) {
            const f32x4 q = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(rr, off(j), 0, POL));
            x[4 * j] = q.x; x[4 * j + 1] = q.y; x[4 * j + 2] = q.z; x[4 * j + 3] = q.w;
        } else {
            x[j] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(rr, off(j), 0, POL));
        }
    }
    // phase 1: row max (and the plain sum for label smoothing)
    float m = -INFINITY, sl = 0.0f;
#pragma unroll
    for (int j = 0; j < G; ++j) {
        if (j < nv) {
#pragma unroll
            for (int c = 0; c < W; ++c) {
                m = fmaxf(m, x[W * j + c]);
                sl += x[W * j + c];
            }
        }
    }
    const float row_max = block_reduce<NW, true>(m, red[0]);
    // phase 2: denominator; keep exp(l - max) for the gradient
    float se = 0.0f;
#pragma unroll
    for (int j = 0; j < G; ++j) {
#pragma unroll
        for (int c = 0; c < W; ++c) {
            const float e = j < nv ? __expf(x[W * j + c] - row_max) : 0.0f;
            se += e;
            x[W * j + c] = e;
        }
    }
    const float denom = fmaxf(block_reduce<NW, false>(se, red[1]), 1e-30f);
    const float sum_l = alpha > 0.0f ? block_reduce<NW, false>(sl, red[2]) : 0.0f;
    const float inv_denom = 1.0f / denom;
    const float lse = row_max + __logf(denom);
    if (tid == 0) {
        const float l_t = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(rr, (int)tgt * 4, 0, 0));
        losses[s] = row_loss(lse, l_t, sum_l / (float)V, alpha, beta);
    }
    // Thread 0 has read the target's logit (its value is used above); the
    // thread that owns that element overwrites it only after this barrier.
    __syncthreads();
    // phase 4: the gradient, in place.  The target's register slot in the
    // thread that holds it (-1 elsewhere).
    const int tg = (int)tgt / W;
    const int tslot = (tg % NT == tid) ? (tg / NT) * W + (int)tgt % W : -1;
    const float zf = 2.0f * beta * lse;
    const float smooth = alpha / (float)V;
    const float hit = 1.0f - alpha;
#pragma unroll
    for (int j = 0; j < G; ++j) {
        float g[W];
#pragma unroll
        for (int c = 0; c < W; ++c) {
            const int i = W * j + c;
            const float p = x[i] * inv_denom;
            const float t = (i == tslot ? hit : 0.0f) + smooth;
            g[c] = ((p - t) + zf * p) * inv_norm;
        }
        if (VEC) {
            const f32x4 q = f32x4{g[0], g[W > 1 ? 1 : 0], g[W > 2 ? 2 : 0], g[W > 3 ? 3 : 0]};
            __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4v, q), rr, off(j), 0, POL);
        } else {
            __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(unsigned, g[0]), rr, off(j), 0, POL);
        }
    }
}

// Rows too long for the registers: the page's order, reading the row three
// times (max and plain sum, exp sum, gradient).
template <int NT>
__global__ __launch_bounds__(NT) void cross_entropy_stream(float *logits, const uint32_t *tgts, float *losses, int V,
                                                           float alpha, float beta, float inv_norm) {
    constexpr int NW = NT / 64;
    __shared__ float red[3][NW];
    const int tid = threadIdx.x;
    const int s = blockIdx.x;
    float *row = logits + (size_t)s * V;
    const uint32_t tgt = tgts[s];
    if (tgt >= (uint32_t)V) {
        if (tid == 0) losses[s] = 0.0f;
        for (int v = tid; v < V; v += NT) row[v] = 0.0f;
        return;
    }
    float m = -INFINITY, sl = 0.0f;
    for (int v = tid; v < V; v += NT) {
        const float l = row[v];
        m = fmaxf(m, l);
        sl += l;
    }
    const float row_max = block_reduce<NW, true>(m, red[0]);
    float se = 0.0f;
    for (int v = tid; v < V; v += NT) se += __expf(row[v] - row_max);
    const float denom = fmaxf(block_reduce<NW, false>(se, red[1]), 1e-30f);
    const float sum_l = alpha > 0.0f ? block_reduce<NW, false>(sl, red[2]) : 0.0f;
    const float inv_denom = 1.0f / denom;
    const float lse = row_max + __logf(denom);
    if (tid == 0) losses[s] = row_loss(lse, row[tgt], sum_l / (float)V, alpha, beta);
    __syncthreads();
    const float zf = 2.0f * beta * lse;
    const float smooth = alpha / (float)V;
    for (int v = tid; v < V; v += NT) {
        const float p = __expf(row[v] - row_max) * inv_denom;
        const float t = (v == (int)tgt ? 1.0f - alpha : 0.0f) + smooth;
        row[v] = ((p - t) + zf * p) * inv_norm;
    }
}

// sum_losses: one workgroup; thread t adds t, t + NT, ... in order, then the
// fixed-order workgroup reduction.
template <int NT>
__global__ __launch_bounds__(NT) void sum_losses_kernel(const float *losses, float *out, int S) {
    __shared__ float red[NT / 64];
    float acc = 0.0f;
    for (int i = threadIdx.x; i < S; i += NT) acc += losses[i];
    const float total = block_reduce<NT / 64, false>(acc, red);
    if (threadIdx.x == 0) out[0] = total;
}

// --- distillation ---
//
// One workgroup per row again.  The gradient of both terms is a function of
// the logit alone, A e^(l - max) + B e^((l - max) / tau) + C, but for the
// target's column and the teacher's: those few are written once more, with
// their subtractions, after the row.  Bound by memory like cross_entropy:
// each logit is read once and its gradient written once while the row fits in
// the registers (65536 logits); longer rows are read twice, the maximum and
// the sums being formed in one pass over the row.
//
//  * 16-byte accesses start at the row's first 16-byte boundary, so rows of
//    any length and any 4-byte alignment take them; the up to three logits in
//    front of the boundary and behind the last whole group go to one thread
//    each.
//  * Between its loads and its stores a row meets two barriers: one for the
//    maximum (and the teacher's entries, in LDS), one for all sums together.
//    The last wave, whose share of the row is the smallest, forms the
//    teacher's statistics between the two, and all threads together look for
//    columns that several entries name: K^2 comparisons by K threads alone
//    took as long as half of a 4096-logit row.
//  * Rows of 16385 to 51200 logits take 512 threads with 64 or 100 logits
//    each, so that two rows share a CU and one's loads run under the other's
//    reductions and stores: 4096 x 32000 in 184 us (5.7 TB/s) against 230
//    with 1024 threads of 32, 4093 x 50257 in 322 us (5.1 TB/s) against 343
//    with 1024 of 64.  The bound of four waves a SIMD that this needs costs the
//    100-logit kernel 20 to 68 bytes of spilled registers a thread; without
//    it one row would have the CU to itself (354 us).
//  * tau = 1 (T1) makes both exponentials one, which is then kept in place of
//    the logit, as in cross_entropy.
//  * The exponentials over the row are __expf, as in cross_entropy: x log2(e) is
//    rounded once, so a probability e^x is off by about |x| 2^-24 of itself
//    (e^-20 by 1.2e-6).  It is a product and one instruction; only small
//    probabilities lose by it, which weigh little in the sums.  The teacher's few
//    are expf.
constexpr int kMaxTop = 1024;  // teacher entries a row

struct Distill {
    const float *logits;
    float *grad;
    const void *targets, *ids, *teacher;
    float *losses;
    int S, V, K;
    int targets64, ids64, half;
    float inv_tau, tau, mix, alpha, beta, inv_norm;
};

// A column of a 32- or 64-bit index array, -1 for one outside [0, V).
__device__ __forceinline__ int column(const void *p, int wide, int64_t i, int V) {
    const int64_t v = wide ? ((const int64_t *)p)[i] : (int64_t)((const int *)p)[i];
    return v >= 0 && v < V ? (int)v : -1;
}
__device__ __forceinline__ float teacher_logit(const Distill &a, int64_t i) {
    return a.half ? (float)((const _Float16 *)a.teacher)[i] : ((const float *)a.teacher)[i];
}

// Sum or maximum over the wave's lanes, the same in every lane: shifts within
// rows of 16 lanes, then broadcasts into the next rows (a butterfly through
// LDS takes several times as long).
template <bool MAX>
__device__ __forceinline__ float lanes_reduce(float v) {
    const int none = MAX ? __builtin_bit_cast(int, -INFINITY) : 0;
    auto step = [&](auto ctrl, auto rows) {
        const float u = __builtin_bit_cast(
            float, __builtin_amdgcn_update_dpp(none, __builtin_bit_cast(int, v), ctrl.value, rows.value, 0xf, false));
        v = MAX ? fmaxf(v, u) : v + u;
    };
    using std::integral_constant;
    step(integral_constant<int, 0x111>(), integral_constant<int, 0xf>());  // row_shr:1
    step(integral_constant<int, 0x112>(), integral_constant<int, 0xf>());  // row_shr:2
    step(integral_constant<int, 0x114>(), integral_constant<int, 0xf>());  // row_shr:4
    step(integral_constant<int, 0x118>(), integral_constant<int, 0xf>());  // row_shr:8
    step(integral_constant<int, 0x142>(), integral_constant<int, 0xa>());  // row_bcast:15
    step(integral_constant<int, 0x143>(), integral_constant<int, 0xc>());  // row_bcast:31
    return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), 63));
}

// The teacher's distribution over a row's used entries: mass j =
// exp(z[j] - ref) inv, its logarithm z[j] - ref - log_sum.
struct Masses {
    float ref, inv, log_sum;
    int any;  // some entry has mass (or is NaN, which is passed on)
};

// A row's teacher entries in LDS: columns (-1: not used), the teacher's
// logits over tau, the student's logits there, and whether another entry
// names the same column.
struct Teacher {
    __align__(16) int id[kMaxTop];
    float z[kMaxTop], l[kMaxTop];
    unsigned char twice[kMaxTop];
    float target;  // the student's logit at the target
    Masses mass;
};

__device__ __forceinline__ Masses masses(const Teacher &t, int K) {
    const int lane = threadIdx.x & 63;
    float m = -INFINITY, se = 0.0f;
    for (int j = lane; j < K; j += 64)
        if (t.id[j] >= 0) m = fmaxf(m, t.z[j]);
    m = lanes_reduce<true>(m);
    Masses r;
    r.ref = m == -INFINITY ? 0.0f : m;
    for (int j = lane; j < K; j += 64)
        if (t.id[j] >= 0) se += expf(t.z[j] - r.ref);
    se = lanes_reduce<false>(se);
    r.any = se != 0.0f;
    r.inv = r.any ? 1.0f / se : 0.0f;
    r.log_sum = r.any ? logf(se) : 0.0f;
    return r;
}
__device__ __forceinline__ float mass_of(const Teacher &t, const Masses &r, int j) {
    return r.any && t.id[j] >= 0 ? expf(t.z[j] - r.ref) * r.inv : 0.0f;
}

// Marks the entries whose column another entry names too.  Entries are dealt
// to the threads, and with fewer entries than threads so are the entries that
// each is compared with, four at a time.
template <int NT>
__device__ __forceinline__ void mark_repeats(Teacher &t, int K) {
    int span = 64;  // threads for one entry each: a power of two
    while (span < K && span < NT) span *= 2;
    const int parts = NT / span, part = threadIdx.x / span;
    for (int j = threadIdx.x & (span - 1); j < K; j += span) {
        const int id = t.id[j];
        if (id < 0) continue;
        bool twice = false;
        for (int q = 4 * part; q < K; q += 4 * parts) {
            const int4 u = *(const int4 *)&t.id[q];
            twice |= (u.x == id && q != j) | (u.y == id && q + 1 != j) | (u.z == id && q + 2 != j) |
                     (u.w == id && q + 3 != j);
        }
        if (twice) t.twice[j] = 1;
    }
}

// What a row's losses and gradient are made of.
struct RowSums {
    float top, lse, log_soft, sum_l;
    float A, B, C;  // the gradient's factors
};
__device__ __forceinline__ RowSums row_sums(const Distill &a, int tgt, bool taught, float top, float hard, float soft,
                                            float sum_l) {
    RowSums r;
    r.top = top;
    r.lse = top + logf(hard);
    r.log_soft = logf(soft);
    r.sum_l = a.alpha > 0.0f ? sum_l : 0.0f;  // logits of minus infinity take part in it only when it is asked for
    const float weight = tgt >= 0 ? (1.0f - a.mix) * a.inv_norm : 0.0f;
    r.A = weight * (1.0f + 2.0f * a.beta * r.lse) / hard;
    r.B = taught ? a.mix * a.tau * a.inv_norm / soft : 0.0f;
    r.C = -weight * (a.alpha / (float)a.V);
    return r;
}

// e^x of x <= 0 for both terms' gradients and sums.
template <bool T1>
__device__ __forceinline__ float gradient(const Distill &a, const RowSums &r, float l) {
    const float d = l - r.top;
    if (T1) return (r.A + r.B) * __expf(d) + r.C;
    return r.A * __expf(d) + r.B * __expf(d * a.inv_tau) + r.C;
}

// Sums three values over the workgroup at once, in wave order.
template <int NW>
__device__ __forceinline__ void block_sum3(float &x, float &y, float &z, float (*slots)[NW]) {
    x = lanes_reduce<false>(x);
    y = lanes_reduce<false>(y);
    z = lanes_reduce<false>(z);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    if (lane == 0) {
        slots[0][wave] = x;
        slots[1][wave] = y;
        slots[2][wave] = z;
    }
    __syncthreads();
    x = slots[0][0];
    y = slots[1][0];
    z = slots[2][0];
#pragma unroll
    for (int w = 1; w < NW; ++w) {
        x += slots[0][w];
        y += slots[1][w];
        z += slots[2][w];
    }
}

// Puts entries first, first + NT, ... of a row's teacher into LDS.
template <int NT>
__device__ __forceinline__ void load_teacher(const Distill &a, int s, const float *row, Teacher &t, int first) {
    for (int j = first; j < a.K; j += NT) {
        const int64_t i = (int64_t)s * a.K + j;
        const int id = column(a.ids, a.ids64, i, a.V);
        t.id[j] = id;
        t.twice[j] = 0;
        t.z[j] = teacher_logit(a, i) * a.inv_tau;
        t.l[j] = id >= 0 ? row[id] : 0.0f;
    }
    // whole groups of four for the comparisons
    if (threadIdx.x < 3 && a.K + (int)threadIdx.x < kMaxTop) t.id[a.K + threadIdx.x] = -1;
}

// The row's losses, and the columns whose gradient differs from the rest's.
// Called once the stores of the row's gradient have been issued; waits for
// them before any such column is written again.
template <int NT, bool T1>
__device__ __forceinline__ void finish_row(const Distill &a, int s, int tgt, const RowSums &r,
                                           const Masses &mass, const Teacher &t, float *grad) {
    const int tid = threadIdx.x;
    const float hit = (1.0f - a.mix) * (1.0f - a.alpha) * a.inv_norm, soft = a.mix * a.tau * a.inv_norm;
    // Entry j of a thread is j = tid + NT i.  The first entry of a column
    // writes it, with the masses of all of that column's entries in their order.
    constexpr int EACH = (kMaxTop + NT - 1) / NT;
    float value[EACH];
    bool mine[EACH], target_named = false;
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
        const int j = tid + NT * i;
        mine[i] = false;
        const int id = j < a.K ? t.id[j] : -1;
        if (id < 0) continue;
        bool first = true;
        float m = mass_of(t, mass, j);
        if (t.twice[j]) {
            m = 0.0f;
            for (int e = 0; e < a.K; ++e) {
                if (t.id[e] != id) continue;
                first = first && e >= j;
                m += mass_of(t, mass, e);
            }
        }
        target_named = target_named || id == tgt;
        mine[i] = first;
        value[i] = gradient<T1>(a, r, t.l[j]) - soft * m - (id == tgt ? hit : 0.0f);
    }
    if (tid >= NT - 64) {
        float kd = 0.0f;
        for (int j = tid - (NT - 64); j < a.K; j += 64) {
            const float m = mass_of(t, mass, j);
            if (m != 0.0f)
                kd += m * ((t.z[j] - mass.ref - mass.log_sum) - ((t.l[j] - r.top) * a.inv_tau - r.log_soft));
        }
        kd = lanes_reduce<false>(kd);
        if (tid == NT - 1) {
            a.losses[s] = tgt >= 0 ? row_loss(r.lse, t.target, r.sum_l / (float)a.V, a.alpha, a.beta) : 0.0f;
            a.losses[(size_t)a.S + s] = mass.any ? a.tau * a.tau * kd : 0.0f;
        }
    }
    __builtin_amdgcn_s_waitcnt(0);  // this wave's stores of the row are complete
    const bool named = __syncthreads_or(target_named);
#pragma unroll
    for (int i = 0; i < EACH; ++i)
        if (mine[i]) grad[t.id[tid + NT * i]] = value[i];
    if (!named && tid == 0 && tgt >= 0) grad[tgt] = gradient<T1>(a, r, t.target) - hit;
}

// The row's layout for 16-byte accesses: `head` logits in front of the first
// boundary, `groups` whole groups, `tail` logits behind them.
struct RowShape {
    int head, groups, tail;
};
__device__ __forceinline__ RowShape row_shape(const float *row, int V) {
    RowShape r;
    r.head = min((int)((16 - (reinterpret_cast<uintptr_t>(row) & 15)) & 15) / 4, V);
    r.groups = (V - r.head) / 4;
    r.tail = V - r.head - 4 * r.groups;
    return r;
}
// The column of the edge logit that this thread holds, or -1.
__device__ __forceinline__ int edge_column(const RowShape &r) {
    const int t = threadIdx.x;
    if (t < r.head) return t;
    if (t < r.head + r.tail) return t + 4 * r.groups;
    return -1;
}

template <int NT, int CAP, bool STREAM, bool T1>
__global__ __launch_bounds__(NT, CAP == 100 ? 4 : 1) void distill_resident(Distill a) {
    constexpr int NW = NT / 64, G = CAP / 4, POL = STREAM ? kNonTemporal : 0;
    __shared__ float red[4][NW];
    __shared__ Teacher teacher;
    const int tid = threadIdx.x, s = blockIdx.x;
    const float *row = a.logits + (size_t)s * a.V;
    float *grad = a.grad + (size_t)s * a.V;
    const RowShape shape = row_shape(row, a.V);
    const int edge = edge_column(shape);
    const Rsrc rr = row_rsrc(row + shape.head, shape.groups * 16), rg = row_rsrc(grad + shape.head, shape.groups * 16);
    auto off = [&](int j) { return (j * NT + tid) * 16; };
    const int tgt = a.targets ? column(a.targets, a.targets64, s, a.V) : -1;
    if (a.targets && tgt < 0) {
        // padding: zero losses, zero gradient
        if (tid < 2) a.losses[(size_t)tid * a.S + s] = 0.0f;
#pragma unroll
        for (int j = 0; j < G; ++j) __builtin_amdgcn_raw_buffer_store_b128(u32x4v{0u, 0u, 0u, 0u}, rg, off(j), 0, POL);
        if (edge >= 0) grad[edge] = 0.0f;
        return;
    }
    f32x4 x[G];
#pragma unroll
    for (int j = 0; j < G; ++j)
        x[j] = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(rr, off(j), 0, POL));
    const float xe = edge >= 0 ? row[edge] : -INFINITY;
    if (tid == 0) teacher.target = tgt >= 0 ? row[tgt] : 0.0f;
    load_teacher<NT>(a, s, row, teacher, tid);
    const int nv = shape.groups > tid ? min(G, (shape.groups - tid + NT - 1) / NT) : 0;  // this thread's groups
    float m = xe, sl = edge >= 0 ? xe : 0.0f;
#pragma unroll
    for (int j = 0; j < G; ++j) {
        if (j < nv) {
            m = fmaxf(m, fmaxf(fmaxf(x[j][0], x[j][1]), fmaxf(x[j][2], x[j][3])));
            sl += (x[j][0] + x[j][1]) + (x[j][2] + x[j][3]);
        }
    }
    // The barrier in here also makes the teacher's entries visible, and all
    // reads of the row are complete before it: what they gave has been used,
    // or written to LDS.
    const float top = block_reduce<NW, true>(m, red[0]);
    float hard = 0.0f, soft = 0.0f;
    if (edge >= 0) {
        hard = __expf(xe - top);
        if (!T1) soft = __expf((xe - top) * a.inv_tau);
    }
#pragma unroll
    for (int j = 0; j < G; ++j) {
        if (j < nv) {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const float d = x[j][c] - top, e = __expf(d);
                hard += e;
                if (T1) x[j][c] = e;
                else soft += __expf(d * a.inv_tau);
            }
        }
    }
    mark_repeats<NT>(teacher, a.K);
    if (tid >= NT - 64) {
        const Masses of = masses(teacher, a.K);
        if (tid == NT - 1) teacher.mass = of;
    }
    block_sum3<NW>(hard, soft, sl, &red[1]);
    const Masses mass = teacher.mass;
    const RowSums r = row_sums(a, tgt, mass.any, top, hard, T1 ? hard : soft, sl);
#pragma unroll
    for (int j = 0; j < G; ++j) {
        f32x4 g;
#pragma unroll
        for (int c = 0; c < 4; ++c) g[c] = T1 ? (r.A + r.B) * x[j][c] + r.C : gradient<false>(a, r, x[j][c]);
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4v, g), rg, off(j), 0, POL);
    }
    if (edge >= 0) grad[edge] = gradient<T1>(a, r, xe);
    finish_row<NT, T1>(a, s, tgt, r, mass, teacher, grad);
}

// Rows too long for the registers, or whose gradient lies at another
// alignment than the row (VEC false: 4-byte accesses): one pass for the
// maximum and the sums, each thread moving its own reference when it meets a
// larger logit, one for the gradient.
template <int NT, bool VEC>
__global__ __launch_bounds__(NT) void distill_stream(Distill a) {
    constexpr int NW = NT / 64;
    __shared__ float red[4][NW];
    __shared__ Teacher teacher;
    const int tid = threadIdx.x, s = blockIdx.x;
    const float *row = a.logits + (size_t)s * a.V;
    float *grad = a.grad + (size_t)s * a.V;
    const RowShape shape = VEC ? row_shape(row, a.V) : RowShape{0, 0, 0};
    const int edge = VEC ? edge_column(shape) : -1;
    const f32x4 *groups = (const f32x4 *)(row + shape.head);
    f32x4 *out = (f32x4 *)(grad + shape.head);
    const int tgt = a.targets ? column(a.targets, a.targets64, s, a.V) : -1;
    if (a.targets && tgt < 0) {
        if (tid < 2) a.losses[(size_t)tid * a.S + s] = 0.0f;
        for (int v = tid; v < a.V; v += NT) grad[v] = 0.0f;
        return;
    }
    if (tid == 0) teacher.target = tgt >= 0 ? row[tgt] : 0.0f;
    load_teacher<NT>(a, s, row, teacher, tid);
    float m = -INFINITY, ref = 0.0f, hard = 0.0f, soft = 0.0f, sl = 0.0f;
    auto raise = [&](float l) {  // to a larger reference
        if (l > m) {
            if (m != -INFINITY) {
                hard *= __expf(m - l);
                soft *= __expf((m - l) * a.inv_tau);
            }
            m = ref = l;
        }
    };
    auto add = [&](float l) {
        sl += l;
        hard += __expf(l - ref);
        soft += __expf((l - ref) * a.inv_tau);
    };
    if (VEC) {
        for (int i = tid; i < shape.groups; i += NT) {
            const f32x4 l = groups[i];
            raise(fmaxf(fmaxf(l[0], l[1]), fmaxf(l[2], l[3])));
#pragma unroll
            for (int c = 0; c < 4; ++c) add(l[c]);
        }
        if (edge >= 0) {
            raise(row[edge]);
            add(row[edge]);
        }
    } else {
        for (int v = tid; v < a.V; v += NT) {
            const float l = row[v];
            raise(l);
            add(l);
        }
    }
    const float top = block_reduce<NW, true>(m, red[0]);
    if (m == -INFINITY) {  // nothing above minus infinity here
        // a NaN's sums stay NaN
    } else {
        hard *= __expf(m - top);
        soft *= __expf((m - top) * a.inv_tau);
    }
    mark_repeats<NT>(teacher, a.K);
    if (tid >= NT - 64) {
        const Masses of = masses(teacher, a.K);
        if (tid == NT - 1) teacher.mass = of;
    }
    block_sum3<NW>(hard, soft, sl, &red[1]);
    const Masses mass = teacher.mass;
    const RowSums r = row_sums(a, tgt, mass.any, top, hard, soft, sl);
    if (VEC) {
        for (int i = tid; i < shape.groups; i += NT) {
            const f32x4 l = groups[i];
            f32x4 g;
#pragma unroll
            for (int c = 0; c < 4; ++c) g[c] = gradient<false>(a, r, l[c]);
            out[i] = g;
        }
        if (edge >= 0) grad[edge] = gradient<false>(a, r, row[edge]);
    } else {
        for (int v = tid; v < a.V; v += NT) grad[v] = gradient<false>(a, r, row[v]);
    }
    finish_row<NT, false>(a, s, tgt, r, mass, teacher, grad);
}

bool overlaps(const void *a, size_t abytes, const void *b, size_t bbytes) {
    if (a == nullptr || b == nullptr || abytes == 0 || bbytes == 0) return false;
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
    return a0 < b0 + bbytes && b0 < a0 + abytes;
}

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

}  // namespace

extern "C" {

int loss_cross_entropy(float *logits, const uint32_t *targets, float *losses, int64_t S, int64_t V, float alpha,
                       float beta, float inv_norm, void *stream) {
    if (S < 0 || V < 0 || S >= ((int64_t)1 << 31) || V >= ((int64_t)1 << 29)) return GEMM_ERR_SHAPE;
    if (S > 0 && (targets == nullptr || losses == nullptr || (V > 0 && logits == nullptr))) return GEMM_ERR_NULL;
    if (!aligned(logits, 4) || !aligned(targets, 4) || !aligned(losses, 4)) return GEMM_ERR_ALIGN;
    if (!(alpha >= 0.0f && alpha <= 1.0f) || !(beta >= 0.0f) || !std::isfinite(beta) || !std::isfinite(inv_norm))
        return GEMM_ERR_DTYPE;
    if (overlaps(losses, (size_t)S * 4, logits, (size_t)S * V * 4) || overlaps(losses, (size_t)S * 4, targets, (size_t)S * 4))
        return GEMM_ERR_ALIAS;
    if (S == 0) return GEMM_OK;
    hipStream_t st = static_cast<hipStream_t>(stream);
    const int v = (int)V;
    const bool vec = V % 4 == 0 && aligned(logits, 16);
    const bool stream_hint = S * V * 4 >= kStreamBytes;
    // a workgroup of `threads` threads a row
    auto launch = [&](void (*kernel)(float *, const uint32_t *, float *, int, float, float, float), int threads) {
        return in_slices(S, threads, [&](int64_t first, unsigned count) {
            hipLaunchKernelGGL(kernel, dim3(count), dim3(threads), 0, st, logits + first * V, targets + first,
                               losses + first, v, alpha, beta, inv_norm);
        });
    };
    // a resident launch of NT threads holding CAP logits each
#define LOSS_RESIDENT(NT, CAP) \
    launch(stream_hint ? cross_entropy_resident<NT, CAP, true, true> : cross_entropy_resident<NT, CAP, true, false>, NT)
    if (vec && V <= 256 * 16) return LOSS_RESIDENT(256, 16);
    if (vec && V <= 512 * 16) return LOSS_RESIDENT(512, 16);
    if (vec && V <= 512 * 32) return LOSS_RESIDENT(512, 32);
    if (vec && V <= 1024 * 32) return LOSS_RESIDENT(1024, 32);
    if (V <= 256 * 64 && !vec) return launch(cross_entropy_resident<256, 64, false, false>, 256);
    if (V <= 1024 * 64 && vec) return LOSS_RESIDENT(1024, 64);
    return launch(cross_entropy_stream<1024>, 1024);
#undef LOSS_RESIDENT
}

int loss_sum_losses(const float *losses, float *out, int64_t S, void *stream) {
    if (S < 0 || S >= ((int64_t)1 << 31)) return GEMM_ERR_SHAPE;
    if (out == nullptr || (S > 0 && losses == nullptr)) return GEMM_ERR_NULL;
    if (!aligned(losses, 4) || !aligned(out, 4)) return GEMM_ERR_ALIGN;
    if (overlaps(out, 4, losses, (size_t)S * 4)) return GEMM_ERR_ALIAS;
    hipLaunchKernelGGL((sum_losses_kernel<1024>), dim3(1), dim3(1024), 0, static_cast<hipStream_t>(stream), losses, out,
                       (int)S);
    return hipGetLastError() == hipSuccess ? GEMM_OK : GEMM_ERR_LAUNCH;
}

int loss_distill_cross_entropy(const loss_distill_args *args, void *stream) {
    if (args == nullptr) return GEMM_ERR_NULL;
    const loss_distill_args &p = *args;
    const int64_t S = p.S, V = p.V, K = p.K;
    if (S < 0 || V < 0 || K < 0 || S >= ((int64_t)1 << 31) || V >= ((int64_t)1 << 29) || K > kMaxTop)
        return GEMM_ERR_SHAPE;
    if (S > 0 && (p.losses == nullptr || (V > 0 && (p.logits == nullptr || p.dlogits == nullptr)) ||
                  (K > 0 && (p.teacher_ids == nullptr || p.teacher_logits == nullptr))))
        return GEMM_ERR_NULL;
    const float tau = (float)p.temperature, mix = (float)p.mix, alpha = (float)p.alpha, beta = (float)p.beta;
    if ((p.targets64 != 0 && p.targets64 != 1) || (p.ids64 != 0 && p.ids64 != 1) ||
        (p.teacher_f16 != 0 && p.teacher_f16 != 1) || !(tau > 0.0f) || !std::isfinite(tau) ||
        !std::isfinite(1.0f / tau) || !std::isfinite(tau * tau) || !(mix >= 0.0f && mix <= 1.0f) ||
        !(alpha >= 0.0f && alpha <= 1.0f) || !(beta >= 0.0f) || !std::isfinite(beta) ||
        !std::isfinite((float)p.inv_norm))
        return GEMM_ERR_DTYPE;
    if (p.targets == nullptr && mix != 1.0f && S > 0) return GEMM_ERR_NULL;  // the hard term needs targets
    if (!aligned(p.logits, 4) || !aligned(p.dlogits, 4) || !aligned(p.losses, 4) ||
        !aligned(p.targets, p.targets64 ? 8 : 4) || !aligned(p.teacher_ids, p.ids64 ? 8 : 4) ||
        !aligned(p.teacher_logits, p.teacher_f16 ? 2 : 4))
        return GEMM_ERR_ALIGN;
    const size_t rows = (size_t)S * V * 4, lb = (size_t)S * 8, tb = (size_t)S * (p.targets64 ? 8 : 4),
                 ib = (size_t)S * K * (p.ids64 ? 8 : 4), zb = (size_t)S * K * (p.teacher_f16 ? 2 : 4);
    if ((p.dlogits != p.logits && overlaps(p.dlogits, rows, p.logits, rows)) ||
        overlaps(p.dlogits, rows, p.losses, lb) || overlaps(p.logits, rows, p.losses, lb))
        return GEMM_ERR_ALIAS;
    for (const auto &out : {std::make_pair((const void *)p.dlogits, rows), std::make_pair((const void *)p.losses, lb)})
        if (overlaps(out.first, out.second, p.targets, tb) || overlaps(out.first, out.second, p.teacher_ids, ib) ||
            overlaps(out.first, out.second, p.teacher_logits, zb))
            return GEMM_ERR_ALIAS;
    if (S == 0) return GEMM_OK;
    Distill a;
    a.logits = p.logits;
    a.grad = p.dlogits;
    a.targets = p.targets;
    a.ids = p.teacher_ids;
    a.teacher = p.teacher_logits;
    a.losses = p.losses;
    a.S = (int)S;
    a.V = (int)V;
    a.K = (int)K;
    a.targets64 = (int)p.targets64;
    a.ids64 = (int)p.ids64;
    a.half = (int)p.teacher_f16;
    a.tau = tau;
    a.inv_tau = 1.0f / tau;
    a.mix = mix;
    a.alpha = alpha;
    a.beta = beta;
    a.inv_norm = (float)p.inv_norm;
    hipStream_t st = static_cast<hipStream_t>(stream);
    const bool nt = S * V * 4 >= kStreamBytes;
    const bool same_phase = ((reinterpret_cast<uintptr_t>(p.logits) ^ reinterpret_cast<uintptr_t>(p.dlogits)) & 15) == 0;
    // a workgroup of `threads` threads a row; S stays the distance between the two rows of losses
    auto launch = [&](void (*kernel)(Distill), int threads) {
        return in_slices(S, threads, [&](int64_t first, unsigned count) {
            Distill b = a;
            b.logits += first * V;
            b.grad += first * V;
            if (p.targets) b.targets = static_cast<const char *>(p.targets) + first * (p.targets64 ? 8 : 4);
            b.ids = static_cast<const char *>(p.teacher_ids) + first * K * (p.ids64 ? 8 : 4);
            b.teacher = static_cast<const char *>(p.teacher_logits) + first * K * (p.teacher_f16 ? 2 : 4);
            b.losses += first;
            hipLaunchKernelGGL(kernel, dim3(count), dim3(threads), 0, st, b);
        });
    };
#define DISTILL(NT, CAP)                                                                                              \
    (tau == 1.0f ? launch(nt ? distill_resident<NT, CAP, true, true> : distill_resident<NT, CAP, false, true>, NT)    \
                 : launch(nt ? distill_resident<NT, CAP, true, false> : distill_resident<NT, CAP, false, false>, NT))
    if (!same_phase) return launch(distill_stream<1024, false>, 1024);
    if (V > 1024 * 64) return launch(distill_stream<1024, true>, 1024);
    if (V <= 256 * 16) return DISTILL(256, 16);
    if (V <= 512 * 16) return DISTILL(512, 16);
    if (V <= 512 * 32) return DISTILL(512, 32);
    if (V <= 512 * 64) return DISTILL(512, 64);
    if (V <= 512 * 100) return DISTILL(512, 100);
    return DISTILL(1024, 64);
#undef DISTILL
}

}  // extern "C"
