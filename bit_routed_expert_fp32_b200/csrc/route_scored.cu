// Scored router: softmax or sigmoid scores, a balance bias that steers the choice but not
// the weights, groups of experts of which the best are kept, top-k, renormalised and scaled
// weights (the routing of DeepSeek-style layers whose load is balanced by a bias).
//   L = fp32(x Wr^T + b),  s = sigmoid(L) or softmax(L),  c = s + balance
//   group score = the sum of its one or two largest c; the top_groups best groups stay
//   ids = the k largest c of those groups, w = s[ids] (/ sum of them) * scale
// The logits are fp32 as in moe_route; scores and choice are formed from them in fp64: the
// sigmoid's upper end leaves fp32 scores equal whose logits differ, and a sum of score and
// bias loses what separates two of them.
#include <float.h>

#include "operands.cuh"
#include "route_common.cuh"
#include "tc5.cuh"

namespace moe {
namespace {

using namespace tc5;

__device__ inline double shfl_xor_d(double v, int o) { return __shfl_xor_sync(0xffffffffu, v, o); }

// Order-preserving key of c (larger c, larger key; 0 is below every key): -0 equals +0, and
// NaN (only non-finite inputs make one) counts as -infinity.
__device__ inline unsigned long long score_key(double c) {
    if (c != c) c = -INFINITY;
    const unsigned long long b = (unsigned long long)__double_as_longlong(c + 0.0);
    return (b >> 63) ? ~b : (b | (1ull << 63));
}
__device__ inline double unkey(unsigned long long k) {
    return __longlong_as_double((long long)((k >> 63) ? (k & ~(1ull << 63)) : ~k));
}

// e^x in fp64 for |x| <= 708, to about one ulp and without branches, so that a lane's eight
// interleave: x = n ln 2 + r with ln 2 in two parts (the first of 42 bits: n times it is
// exact; Cody and Waite's reduction), Taylor's series of e^r to r^13 (|r| <= ln 2 / 2: the
// rest is below 2^-57), and n added to the exponent.
__device__ __forceinline__ double exp_d(double x) {
    constexpr double kRound = 6755399441055744.0;          // 1.5 * 2^52: adding it rounds to an integer
    const double t = fma(x, 1.4426950408889634, kRound), n = t - kRound;
    double r = fma(n, -0x1.62e42fefa38p-1, x);
    r = fma(n, -0x1.ef35793c76730p-45, r);
    double e = 1.0 / 6227020800.0;
    e = fma(e, r, 1.0 / 479001600.0);
    e = fma(e, r, 1.0 / 39916800.0);
    e = fma(e, r, 1.0 / 3628800.0);
    e = fma(e, r, 1.0 / 362880.0);
    e = fma(e, r, 1.0 / 40320.0);
    e = fma(e, r, 1.0 / 5040.0);
    e = fma(e, r, 1.0 / 720.0);
    e = fma(e, r, 1.0 / 120.0);
    e = fma(e, r, 1.0 / 24.0);
    e = fma(e, r, 1.0 / 6.0);
    e = fma(e, r, 0.5);
    e = fma(e, r, 1.0);
    e = fma(e, r, 1.0);
    return __hiloint2double(__double2hiint(e) + (__double2loint(t) << 20), __double2loint(e));
}
// 1 / y for normal y > 0 whose reciprocal is normal, to an ulp: the hardware's approximation
// (about 20 bits) and two steps of Newton's iteration.
__device__ __forceinline__ double recip_d(double y) {
    double r;
    asm("rcp.approx.ftz.f64 %0, %1;" : "=d"(r) : "d"(y));
    r = fma(fma(-y, r, 1.0), r, r);
    return fma(fma(-y, r, 1.0), r, r);
}
// The scores in fp64: sigmoid(l) (zero below -708, as the reciprocal of an overflowing sum),
// and e^(l - m) of a softmax (zero below -708).
__device__ __forceinline__ double sigmoid_d(float l) {
    const double e = exp_d(fmin(fmax(-(double)l, -708.0), 708.0));
    return l < -708.f ? 0.0 : l == l ? recip_d(1.0 + e) : (double)l;
}
__device__ __forceinline__ double softmax_term_d(float l, float m) {
    const double d = (double)l - (double)m;
    return d < -708.0 ? 0.0 : d == d ? exp_d(fmin(d, 708.0)) : d;
}

// Scratch of a warp that chooses: its token's logits, and the values by which it chooses (as
// fp32 where groups do not align with lanes, as keys on the careful path).
struct Scratch {
    float L[256];
    union {
        float c[256];
        unsigned long long key[256];
    };
};

// One token's choice by one warp, in fp64 throughout, for the few tokens that fp32 does not
// decide.  Each round takes the largest key over the warp in two 32-bit reductions (high words,
// then the low words of those that tie), the lowest expert among equals.  Returns the expert of
// slot n in lane n < k.  The loops stay rolled: a token that comes here pays mostly for
// fetching the instructions (unrolled, 13 us of a 20 us kernel at 8192 tokens).  Tokens whose
// scores tie come here, a padding row of zeros without a balance among them: 4 to 6 us more for a
// call of up to 130 tokens, 12 to 20 % for 8192 that all do.
__device__ __noinline__ int choose_careful(const ScoreArgs& r, int E, int k, Scratch& S, int lane) {
    float m = 0.f;
    double iz = 1.0;
    __syncwarp();
    if (!r.sigmoid) {
        m = -INFINITY;
#pragma unroll 1
        for (int e = lane; e < E; e += 32) m = fmaxf(m, S.L[e]);
#pragma unroll 1
        for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        double z = 0.0;
#pragma unroll 1
        for (int e = lane; e < E; e += 32) z += softmax_term_d(S.L[e], m);
#pragma unroll 1
        for (int o = 16; o; o >>= 1) z += shfl_xor_d(z, o);
        iz = recip_d(z);
    }
#pragma unroll 1
    for (int e = lane; e < 256; e += 32) {
        unsigned long long key = 0;
        if (e < E) {
            double c = r.sigmoid ? sigmoid_d(S.L[e]) : softmax_term_d(S.L[e], m) * iz;
            if (r.balance) c += (double)__ldg(r.balance + e);
            key = score_key(c);
        }
        S.key[e] = key;
    }
    __syncwarp();
    if (r.top_groups < r.n_groups) {
        const int gs = E / r.n_groups;
        // lane g: the group's two largest; the lanes start at different experts of their
        // groups (bank conflicts)
        double sc = -INFINITY;
        if (lane < r.n_groups) {
            unsigned long long t1 = 0, t2 = 0;
            int i = lane % gs;
#pragma unroll 2
            for (int n = 0; n < gs; ++n) {
                const unsigned long long c = S.key[lane * gs + i];
                t2 = max(t2, min(t1, c));
                t1 = max(t1, c);
                if (++i == gs) i = 0;
            }
            sc = r.group_top == 2 ? unkey(t1) + unkey(t2) : unkey(t1);
            if (sc != sc) sc = -INFINITY;
        }
        __syncwarp();
        int rank = 0;
#pragma unroll 1
        for (int g = 0; g < r.n_groups; ++g) {
            const double o = __shfl_sync(0xffffffffu, sc, g);
            rank += o > sc || (o == sc && g < lane);
        }
        const unsigned kept = __ballot_sync(0xffffffffu, lane < r.n_groups && rank < r.top_groups);
#pragma unroll 1
        for (int e = lane; e < E; e += 32)
            if (!((kept >> (e / gs)) & 1u)) S.key[e] = 0;
        __syncwarp();
    }
    int my_id = 0;
#pragma unroll 1
    for (int n = 0; n < k; ++n) {
        unsigned long long bk = 0;
        int be = lane;
#pragma unroll 2
        for (int e = lane; e < 256; e += 32) {
            const unsigned long long c = S.key[e];
            if (c > bk) {                   // strict: an equal key keeps the lower expert
                bk = c;
                be = e;
            }
        }
        const uint32_t hi = (uint32_t)(bk >> 32), lo = (uint32_t)bk;
        const uint32_t mh = __reduce_max_sync(0xffffffffu, hi);
        const uint32_t ml = __reduce_max_sync(0xffffffffu, hi == mh ? lo : 0u);
        const int e = (int)__reduce_min_sync(0xffffffffu, hi == mh && lo == ml ? (uint32_t)be : 0xFFFFu);
        if (lane == n) my_id = e;
        if (lane == (e & 31)) S.key[e] = 0;
        __syncwarp();
    }
    return my_id;
}

// Order-preserving 32-bit key of a value that is not NaN (0 is below every key) and back.
__device__ inline uint32_t key32(float f) {
    const uint32_t b = __float_as_uint(f + 0.f);
    return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ inline float unkey32(uint32_t k) { return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k); }

// The choice in fp32 where fp32 decides it.  Sigmoid scores from the fast exponential (its
// documented error of 2 + 1.17 |x| ulp counts in proportion to s (1 - s): 8e-8 at most), one
// rounding and the fast quotient (two ulp) are off by at most 2.7e-7; softmax scores by at
// most 2.6e-6 of the largest (ten ulp of the sum's terms on average, its thirteen additions,
// the terms' own few ulp).  Adding the balance rounds once more, relative to the value
// it gives.  So where neighbours among the k + 1 largest values (and the scores of the kept
// groups and of the others) lie further apart than both can be off, their order is the exact
// one; otherwise, and where NaN or infinities meet, false is returned and the careful path
// decides.  A softmax without balance has the order of its logits (as long as fp64 scores would
// not vanish).  A key gives its low three bits to the expert's place in the lane; a lane's eight
// are sorted once and then only popped.
__device__ __forceinline__ bool choose_fast(const ScoreArgs& r, int E, int k, const float (&L)[8], const float (&b)[8],
                                            Scratch& scratch, int lane, int& my_id) {
    // what two scores can be off together, and, relative to their sum of sizes, what the
    // rounding and eight steps of a key come to (2^-20 of either)
    constexpr float kRel = 6e-7f;
    float abs_err = 6e-7f;
    const bool grouped = r.top_groups < r.n_groups, by_logit = !r.sigmoid && !r.balance;
    float c[8], m = 0.f;
    if (r.sigmoid) {
#pragma unroll
        for (int j = 0; j < 8; ++j) c[j] = __fdividef(1.f, 1.f + __expf(-L[j])) + b[j];
    } else {
        m = L[0];
#pragma unroll
        for (int j = 1; j < 8; ++j) m = fmaxf(m, L[j]);
        m = unkey32(__reduce_max_sync(0xffffffffu, m == m ? key32(m) : 0u));
        if (!by_logit || grouped) {
            float z = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                c[j] = __expf(L[j] - m);
                z += c[j];
            }
            z = warp_sum(z);
            const float iz = __fdividef(1.f, z);          // also the largest score
            abs_err = 6e-6f * iz;
#pragma unroll
            for (int j = 0; j < 8; ++j) c[j] = c[j] * iz + b[j];
        }
    }
    // NaN anywhere, or opposite infinities in a lane, make a lane's sum NaN
    float sum = 0.f;
    uint32_t key[8];
    const int live = E - 8 * lane;                         // experts of this lane (or more)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float v = by_logit ? L[j] : c[j];
        const bool in = j < live;
        if (in) sum += by_logit && grouped ? v + c[j] : v;
        key[j] = in ? (key32(v) & ~7u) | (7u - j) : 0u;
    }
    if (__any_sync(0xffffffffu, sum != sum)) return false;
    if (grouped) {
        const int gs = E / r.n_groups, lpg = gs >> 3;
        float t1, t2;
        int leader;                                       // lanes apart that groups lie
        if ((gs & 7) == 0 && (lpg & (lpg - 1)) == 0) {
            // a group is a power of two of lanes: top two of eight, then across them
            t1 = fmaxf(c[0], c[1]);
            t2 = fminf(c[0], c[1]);
#pragma unroll
            for (int j = 2; j < 8; ++j) {
                t2 = fmaxf(t2, fminf(t1, c[j]));
                t1 = fmaxf(t1, c[j]);
            }
            for (int o = 1; o < lpg; o <<= 1) {
                const float a1 = __shfl_xor_sync(0xffffffffu, t1, o), a2 = __shfl_xor_sync(0xffffffffu, t2, o);
                t2 = fmaxf(fminf(t1, a1), fmaxf(t2, a2));
                t1 = fmaxf(t1, a1);
            }
            leader = lpg;
        } else {
            __syncwarp();
#pragma unroll
            for (int j = 0; j < 8; ++j) scratch.c[8 * lane + j] = c[j];
            __syncwarp();
            t1 = t2 = -INFINITY;
            if (lane < r.n_groups) {
                int i = lane % gs;
                for (int n = 0; n < gs; ++n) {
                    const float v = scratch.c[lane * gs + i];
                    t2 = fmaxf(t2, fminf(t1, v));
                    t1 = fmaxf(t1, v);
                    if (++i == gs) i = 0;
                }
            }
            leader = 1;
        }
        // the best groups one by one; lanes past the last group hold none
        const bool pair = r.group_top == 2, group = lane < r.n_groups * leader;
        const float sc = pair ? t1 + t2 : t1;
        uint32_t rest = group ? key32(sc) : 0u;
        if (__any_sync(0xffffffffu, group && sc != sc)) return false;
        unsigned lanes = 0;
        for (int n = 0; n < r.top_groups; ++n) {
            const uint32_t top = __reduce_max_sync(0xffffffffu, rest);
            const bool hit = rest == top;
            lanes |= __ballot_sync(0xffffffffu, hit);
            if (hit) rest = 0;
        }
        // What a group's score can be off goes with its terms: a sum that cancels keeps what
        // rounding them has lost.  (An infinite term makes the sum exact; a finite sum past the
        // type's range counts as its end.)  No kept group may reach down to what another can reach.
        const bool exact = fabsf(t1) == INFINITY || (pair && fabsf(t2) == INFINITY);
        const float mid = exact ? sc : fminf(fmaxf(sc, -FLT_MAX), FLT_MAX);
        const float off = exact ? 0.f : abs_err + kRel * fabsf(t1) + (pair ? kRel * fabsf(t2) : 0.f);
        const bool kept = (lanes >> lane) & 1u;
        const uint32_t lo = __reduce_min_sync(0xffffffffu, kept ? key32(mid - off) : 0xffffffffu);
        const uint32_t hi = __reduce_max_sync(0xffffffffu, group && !kept ? key32(mid + off) : 0u);
        // groups that tie, and infinities that meet, are left to fp64
        if (__popc(lanes) != r.top_groups * leader || lo <= hi) return false;
        if (leader > 1 || gs == 8) {                       // a lane's experts are of one group
            if (!((lanes >> lane) & 1u))
#pragma unroll
                for (int j = 0; j < 8; ++j) key[j] = 0;
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (j < live && !((lanes >> ((8 * lane + j) / gs)) & 1u)) key[j] = 0;
        }
    }
    // descending, by the 19 comparators of Batcher's odd-even merge sort
#pragma unroll
    for (int q = 0; q < 19; ++q) {
        constexpr int A[19] = {0, 2, 4, 6, 0, 1, 4, 5, 1, 5, 0, 1, 2, 3, 2, 3, 1, 3, 5};
        constexpr int B[19] = {1, 3, 5, 7, 2, 3, 6, 7, 2, 6, 4, 5, 6, 7, 4, 5, 2, 4, 6};
        const uint32_t x = key[A[q]], y = key[B[q]];
        key[A[q]] = max(x, y);
        key[B[q]] = min(x, y);
    }
    uint32_t mine = 0;                                     // lane n: the n-th largest key
    int from = 0;                                          // and the lane it was in
    for (int n = 0; n <= k; ++n) {
        const uint32_t top = __reduce_max_sync(0xffffffffu, key[0]);
        const int wl = __ffs(__ballot_sync(0xffffffffu, key[0] == top)) - 1;
        if (lane == wl) {
#pragma unroll
            for (int j = 0; j < 7; ++j) key[j] = key[j + 1];
            key[7] = 0;
        }
        if (lane == n) {
            mine = top;
            from = wl;
        }
    }
    my_id = 8 * from + 7 - (int)(mine & 7u);
    const float v = unkey32(mine & ~7u);
    const uint32_t next = __shfl_down_sync(0xffffffffu, mine, 1);
    bool ok = true;
    if (lane < k) {
        const float w = unkey32(next & ~7u);
        ok = next == 0 || v - w > (by_logit ? 0.f : abs_err) + kRel * (fabsf(v) + fabsf(w));
        if (by_logit) ok &= v - m > -700.f;
    }
    return __all_sync(0xffffffffu, ok);
}

// One token: choice, weights, output of slots < k.  b: the lane's eight balance values.
__device__ void select_scored(const ScoreArgs& r, int E, int k, const float* row, const float (&b)[8], Scratch& scratch,
                              int lane, int32_t* ids_out, float* w_out, int32_t* s_ids) {
    float L[8];
    if ((E & 3) == 0 && 8 * lane + 8 <= E) {
        const float4 u = __ldcg(reinterpret_cast<const float4*>(row) + 2 * lane);
        const float4 v = __ldcg(reinterpret_cast<const float4*>(row) + 2 * lane + 1);
        L[0] = u.x; L[1] = u.y; L[2] = u.z; L[3] = u.w;
        L[4] = v.x; L[5] = v.y; L[6] = v.z; L[7] = v.w;
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) L[j] = 8 * lane + j < E ? ldcg_f32(row + 8 * lane + j) : -INFINITY;
    }
    __syncwarp();
    *reinterpret_cast<float4*>(scratch.L + 8 * lane) = make_float4(L[0], L[1], L[2], L[3]);
    *reinterpret_cast<float4*>(scratch.L + 8 * lane + 4) = make_float4(L[4], L[5], L[6], L[7]);
    __syncwarp();
    int my_id = 0;
    if (!choose_fast(r, E, k, L, b, scratch, lane, my_id)) my_id = choose_careful(r, E, k, scratch, lane);
    // the chosen scores in fp64, one a lane; softmax scores relative to the largest logit, over
    // the sum of all only where they are not renormalised
    const float l = lane < k ? scratch.L[my_id] : 0.f;
    double s;
    if (r.sigmoid) {
        s = sigmoid_d(l);
    } else {
        float m = L[0];
#pragma unroll
        for (int j = 1; j < 8; ++j) m = fmaxf(m, L[j]);
#pragma unroll
        for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        s = softmax_term_d(l, m);
        if (!r.renormalise) {
            double z = 0.0;
#pragma unroll
            for (int j = 0; j < 8; ++j) z += softmax_term_d(L[j], m);
#pragma unroll
            for (int o = 16; o; o >>= 1) z += shfl_xor_d(z, o);
            s *= recip_d(z);
        }
    }
    double w = lane < k ? s : 0.0;
    if (r.renormalise) {
        double sum = w;                                   // of lanes 0 .. 15 (k <= 16)
#pragma unroll
        for (int o = 8; o; o >>= 1) sum += shfl_xor_d(sum, o);
        w = sum > 1e-280 ? w * recip_d(sum) : sum > 0.0 ? w / sum : 0.0;
    }
    if (lane < k) {
        ids_out[lane] = my_id;
        w_out[lane] = (float)(w * (double)r.scale);
        if (s_ids) s_ids[lane] = my_id;
    }
}

// The lane's eight balance values (0 without one).
__device__ inline void load_balance(const ScoreArgs& r, int E, int lane, float (&b)[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) b[j] = r.balance && 8 * lane + j < E ? __ldg(r.balance + 8 * lane + j) : 0.f;
}

// ---------------------------------------------------------------- up to kSmallT tokens
// The router's fp32 rows are read once, straight into MMA fragments: a CTA takes 16 experts
// and a part of K (the CTAs of a cluster share the experts), its warps 32-wide steps in turn.
// A weight is split exactly into three bf16 pieces (each the upper bits of what is left), so
// that x w1 + x w2 + x w3 on mma.sync has fp32-level products.  The order of K inside a
// step is free as long as both operands follow it: lane (g, t) takes elements 8t .. 8t+7 of
// its rows, 32 contiguous bytes, as the fragments of two MMAs.  A warp's sum is short (its
// few steps, the small pieces in an accumulator of their own); warps and CTAs are added in
// double-float.  Up to 8 tokens the last CTA to finish (a ticket) chooses, a warp per token,
// and permutes, while the others form the decode operands; above, a kernel of its own does that
// (16 tokens: 17.7 us with a last CTA of 16 warps, 12.7 us so).
constexpr int kSmExperts = 16, kSmStep = 32, kSmParts = 8, kTailT = 8;

template <int NTL, int NW>   // 8-token MMA columns, warps
struct SmallSmem {
    union {
        float part[NW][kSmExperts][8 * NTL];
        Scratch scratch[NW];
    };
    Df sum[kSmExperts][8 * NTL];
    int32_t ids[kTailT * 16];
    float bal[256];
    int cnt[256];
    int off[257];
    int last;
};

template <int NTL, int NW>
__global__ void __launch_bounds__(32 * NW, 2)
    scored_small_kernel(RouteArgs p, ScoreArgs r, int parts) {
    constexpr int kThreads = 32 * NW, U = NTL == 1 ? 4 : NTL <= 4 ? 2 : 1;
    constexpr bool kTail = 8 * NTL <= kTailT;
    extern __shared__ __align__(16) uint8_t smem_raw[];
    SmallSmem<NTL, NW>& S = *reinterpret_cast<SmallSmem<NTL, NW>*>(smem_raw);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
    const int part = (int)cluster_rank(), e0 = (int)(blockIdx.x / parts) * kSmExperts;
    const int steps = p.H / kSmStep;
    float hi[NTL][4], lo[NTL][4];
#pragma unroll
    for (int n = 0; n < NTL; ++n)
#pragma unroll
        for (int c = 0; c < 4; ++c) hi[n][c] = lo[n][c] = 0.f;
    const bool rows[2] = {e0 + g < p.E, e0 + g + 8 < p.E};
    const float* w0 = p.Wr + (size_t)(e0 + g) * p.H + 8 * t4;
    griddep_wait();
    griddep_launch_dependents();
    if (blockIdx.x == 0 && threadIdx.x == 0) {              // no expert pass of this workspace runs now
        p.ctrl->work[0] = 0;
        p.ctrl->work[1] = 0;
    }
    if (kTail)                                             // for the choice: a late first read of it would wait for HBM
        for (int i = threadIdx.x; i < 256; i += kThreads) S.bal[i] = r.balance && i < p.E ? __ldg(r.balance + i) : 0.f;
    // U steps at a time: up to 8 tokens all of a warp's loads are on their way at once on the
    // usual sizes
    for (int st = part * NW + warp; st < steps; st += U * parts * NW) {
        float w[U][2][8];
        uint4 xv[U][NTL];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int su = st + u * parts * NW, k0 = su * kSmStep;
            const bool in = su < steps;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float4* src = reinterpret_cast<const float4*>(w0 + (size_t)8 * h * p.H + k0);
                const float4 z = make_float4(0.f, 0.f, 0.f, 0.f);
                const float4 a = in && rows[h] ? __ldg(src) : z, b = in && rows[h] ? __ldg(src + 1) : z;
                w[u][h][0] = a.x; w[u][h][1] = a.y; w[u][h][2] = a.z; w[u][h][3] = a.w;
                w[u][h][4] = b.x; w[u][h][5] = b.y; w[u][h][6] = b.z; w[u][h][7] = b.w;
            }
#pragma unroll
            for (int n = 0; n < NTL; ++n) {
                const int t = 8 * n + g;
                xv[u][n] = in && t < p.T
                               ? *reinterpret_cast<const uint4*>(p.x + (size_t)t * p.H + k0 + 8 * t4)
                               : make_uint4(0, 0, 0, 0);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int pl = 0; pl < 3; ++pl) {
                uint32_t a[2][4];               // [row half][pair]
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int q = 0; q < 4; ++q) a[h][q] = next_plane(w[u][h][2 * q], w[u][h][2 * q + 1]);
#pragma unroll
                for (int n = 0; n < NTL; ++n) {
                    float(&d)[4] = pl == 0 ? hi[n] : lo[n];
                    mma_bf16_16816(d[0], d[1], d[2], d[3], a[0][0], a[1][0], a[0][1], a[1][1], xv[u][n].x, xv[u][n].y);
                    mma_bf16_16816(d[0], d[1], d[2], d[3], a[0][2], a[1][2], a[0][3], a[1][3], xv[u][n].z, xv[u][n].w);
                }
            }
    }
#pragma unroll
    for (int n = 0; n < NTL; ++n)
#pragma unroll
        for (int c = 0; c < 4; ++c) S.part[warp][g + 8 * (c >> 1)][8 * n + 2 * t4 + (c & 1)] = hi[n][c] + lo[n][c];
    __syncthreads();
    for (int i = threadIdx.x; i < kSmExperts * 8 * NTL; i += kThreads) {
        const int e = i / (8 * NTL), t = i % (8 * NTL);
        Df v = Df{S.part[0][e][t], 0.f};
#pragma unroll
        for (int u = 1; u < NW; ++u) v = df_add(v, Df{S.part[u][e][t], 0.f});
        S.sum[e][t] = v;
    }
    __syncthreads();
    cluster_sync();
    for (int i = part * kThreads + threadIdx.x; i < kSmExperts * p.T; i += parts * kThreads) {
        const int t = i / kSmExperts, e = i % kSmExperts;
        if (e0 + e >= p.E) continue;
        const uint32_t at = smem_u32(&S.sum[e][t]);
        Df w[kSmParts];
#pragma unroll
        for (int q = 0; q < kSmParts; ++q)
            if (q < parts)
                asm volatile("ld.shared::cluster.v2.f32 {%0,%1}, [%2];"
                             : "=f"(w[q].hi), "=f"(w[q].lo)
                             : "r"(map_peer(at, q))
                             : "memory");
        Df v = w[0];
#pragma unroll
        for (int q = 1; q < kSmParts; ++q)
            if (q < parts) v = df_add(v, w[q]);
        if (p.bias) v = df_add(v, Df{__ldg(p.bias + e0 + e), 0.f});
        p.logits[(size_t)t * p.E + e0 + e] = v.hi + v.lo;      // the one rounding
    }
    __syncwarp();
    cluster_arrive();                   // a CTA leaves only when its sums have been read
    if (kTail) {
        __threadfence();
        __syncthreads();
        if (threadIdx.x == 0) S.last = atomicAdd(&p.ctrl->route_ticket, 1u) == gridDim.x - 1;
        __syncthreads();
    }
    const bool last = kTail && S.last;
    if (last) {
        __threadfence();
        for (int i = threadIdx.x; i < 256; i += kThreads) S.cnt[i] = 0;
        __syncthreads();
        if (warp < p.T) {
            float bal[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) bal[j] = S.bal[8 * lane + j];
            for (int t = warp; t < p.T; t += NW) {
                select_scored(r, p.E, p.k, p.logits + (size_t)t * p.E, bal, S.scratch[warp], lane,
                              p.r.topk_ids + (size_t)t * p.k, p.r.topk_w + (size_t)t * p.k, S.ids + t * p.k);
                __syncwarp();
                if (lane < p.k) atomicAdd(&S.cnt[S.ids[t * p.k + lane]], 1);
            }
        }
        __syncthreads();
        if (warp == 0) {
            warp_scan_counts(S.cnt, S.off, p.E, lane);
            __syncwarp();
            for (int i = lane; i < p.E; i += 32) {
                p.r.counts[i] = S.cnt[i];
                p.r.offsets[i] = S.off[i];
            }
            if (lane == 0) p.r.offsets[p.E] = S.off[p.E];
            __syncwarp();
            // off doubles as the running position per expert
            warp_scatter(S.ids, 0, p.T * p.k, S.off, p.r.perm, p.r.inv_perm, lane, p.E);
            if (lane == 0) p.ctrl->route_ticket = 0;
        } else if (warp == 1) {
            warp_active(S.cnt, p.E, p.S, p.active, p.ctrl, p.T, lane);
        }
    }
    // the decode operands of (token, group) pairs, one per warp
    if (kTail && p.ops && !(last && warp < 2)) {
        const int G8 = 8 * ((p.H / 64 + 7) / 8);
        const OperandArgs o{p.T, p.H, p.x, p.zx, p.iq, p.ctrl};
        // the last CTA's share falls to its warps past the permutation's two
        const int w = last ? warp - 2 : warp, nw = last ? NW - 2 : NW;
        for (int base = blockIdx.x * NW; base < p.T * G8; base += gridDim.x * NW)
            for (int v = w; v < NW; v += nw) {
                const int pr = base + v;
                if (pr >= p.T * G8) break;
                compute_z(o, pr / G8, pr % G8, lane);
                if (p.iq) compute_iq(o, pr / G8, pr % G8, lane);
            }
    }
    __syncwarp();
    cluster_wait();
}

// The choice and the permutation of up to kSmallT tokens: a cluster of eight CTAs takes a
// contiguous part of the tokens each, a warp per token, counts its experts in shared memory,
// forms its bases from the others' counts, and permutes.  The other clusters form the decode
// operands of (token, group) pairs meanwhile, one per warp.  (Whole call, one CTA of 32 warps,
// whose choice its SM's instruction rate bounds, against the cluster: full-size layer 16 tokens
// 13.3 / 12.7 us, 32 16.9 / 14.8, 64 25.8 / 18.8; H 2048, 64 experts 8.7 / 9.0, 10.9 / 9.4,
// 15.6 / 10.9.)
constexpr int kChooseCtas = 8, kChooseWarps = kSmallT / kChooseCtas;
struct ChooseSmem {
    union {
        Scratch scratch[kChooseWarps];
        int run[kChooseWarps][256];
    };
    int32_t ids[kChooseWarps * 16];
    int cnt[256], total[256], base[256];
    int off[257];
};

__global__ void __launch_bounds__(32 * kChooseWarps) scored_choose_kernel(RouteArgs p, ScoreArgs r) {
    static_assert(32 * kChooseWarps == 256, "a thread per expert");
    __shared__ ChooseSmem S;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, e = threadIdx.x;
    S.cnt[e] = 0;
    griddep_wait();
    griddep_launch_dependents();
    if (blockIdx.x >= kChooseCtas) {
        const int G8 = 8 * ((p.H / 64 + 7) / 8), pr = (int)(blockIdx.x - kChooseCtas) * kChooseWarps + warp;
        if (pr < p.T * G8) {
            const OperandArgs o{p.T, p.H, p.x, p.zx, p.iq, p.ctrl};
            compute_z(o, pr / G8, pr % G8, lane);
            if (p.iq) compute_iq(o, pr / G8, pr % G8, lane);
        }
        return;
    }
    const int rank = (int)cluster_rank(), per = (p.T + kChooseCtas - 1) / kChooseCtas;
    const int t0 = min(p.T, rank * per), t1 = min(p.T, t0 + per), n = (t1 - t0) * p.k, t = t0 + warp;
    float bal[8];
    load_balance(r, p.E, lane, bal);
    __syncthreads();
    if (t < t1) {
        int32_t* ids = S.ids + warp * p.k;
        select_scored(r, p.E, p.k, p.logits + (size_t)t * p.E, bal, S.scratch[warp], lane, p.r.topk_ids + (size_t)t * p.k,
                      p.r.topk_w + (size_t)t * p.k, ids);
        __syncwarp();
        if (lane < p.k) atomicAdd(&S.cnt[ids[lane]], 1);
    }
    __syncwarp();
    cluster_sync();                     // every CTA's counts are there; scratch is free
    {
        const uint32_t at = smem_u32(&S.cnt[e]);
        int c[kChooseCtas], base = 0, total = 0;
#pragma unroll
        for (int q = 0; q < kChooseCtas; ++q)
            asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(c[q]) : "r"(map_peer(at, q)) : "memory");
#pragma unroll
        for (int q = 0; q < kChooseCtas; ++q) {
            base += q < rank ? c[q] : 0;
            total += c[q];
        }
        S.base[e] = base;
        S.total[e] = total;
#pragma unroll
        for (int w = 0; w < kChooseWarps; ++w) S.run[w][e] = 0;
    }
    cluster_arrive();                   // this CTA has read the others' counts
    __syncthreads();
    // each warp counts and then ranks 32 of the pairs (8 x 16 at most: four warps)
    const int b0 = min(n, warp * 32), b1 = min(n, b0 + 32);
    if (b0 + lane < b1) atomicAdd(&S.run[warp][S.ids[b0 + lane]], 1);
    if (warp == kChooseWarps - 1) warp_scan_counts(S.total, S.off, p.E, lane);
    if (warp == kChooseWarps - 2 && rank == 0) warp_active(S.total, p.E, p.S, p.active, p.ctrl, p.T, lane);
    __syncthreads();
    if (e < p.E) {
        int run = S.off[e] + S.base[e];
        if (rank == 0) {
            p.r.counts[e] = S.total[e];
            p.r.offsets[e] = S.off[e];
        }
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const int v = S.run[w][e];
            S.run[w][e] = run;
            run += v;
        }
    }
    if (e == 0 && rank == 0) p.r.offsets[p.E] = S.off[p.E];
    __syncthreads();
    if (b0 < b1) warp_scatter(S.ids + b0, t0 * p.k + b0, b1 - b0, S.run[warp], p.r.perm, p.r.inv_perm, lane, p.E);
    __syncwarp();
    cluster_wait();                     // a CTA leaves only when its counts have been read
}

// ---------------------------------------------------------------- above kSmallT tokens
// The router's rows as three bf16 planes [3][E][H] (w = w1 + w2 + w3 exactly, each the
// upper bits of what is left), for the logits kernel's operand loads; zeroes the histograms
// that the top-k kernel adds to.
__global__ void __launch_bounds__(256) scored_split_kernel(RouteArgs p, uint16_t* planes, int32_t* sums, int n_sums) {
    griddep_wait();
    griddep_launch_dependents();
    const size_t n8 = (size_t)p.E * p.H / 8, plane = (size_t)p.E * p.H;
    const size_t i0 = (size_t)blockIdx.x * blockDim.x + threadIdx.x, step = (size_t)gridDim.x * blockDim.x;
    for (size_t i = i0; i < (size_t)n_sums; i += step) sums[i] = 0;
    const size_t n_hist = (size_t)((p.T + kChunk - 1) / kChunk) * p.E;
    for (size_t i = i0; i < n_hist; i += step) p.hist[i] = 0;
    for (size_t i = i0; i < n8; i += step) {
        const float4 a = __ldg(reinterpret_cast<const float4*>(p.Wr) + 2 * i);
        const float4 b = __ldg(reinterpret_cast<const float4*>(p.Wr) + 2 * i + 1);
        float w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int pl = 0; pl < 3; ++pl) {
            uint32_t o[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) o[q] = next_plane(w[2 * q], w[2 * q + 1]);
            *reinterpret_cast<uint4*>(planes + pl * plane + 8 * i) = make_uint4(o[0], o[1], o[2], o[3]);
        }
    }
}

// Top-k: a warp per token.  Adds to the histograms of the token's chunk (p.hist) and of its
// span of kSpan chunks (integer atomics: the sums do not depend on their order), from which
// the scatter kernel's CTAs form their bases by themselves.
constexpr int kTopWarps = 4, kSpan = 16;

__global__ void __launch_bounds__(32 * kTopWarps, 6) scored_topk_kernel(RouteArgs p, ScoreArgs r, int32_t* sums) {
    __shared__ Scratch s_scratch[kTopWarps];
    griddep_wait();
    griddep_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int t = blockIdx.x * kTopWarps + warp, c = t / kChunk;
    if (t >= p.T) return;
    float bal[8];
    load_balance(r, p.E, lane, bal);
    int32_t* ids = p.r.topk_ids + (size_t)t * p.k;
    select_scored(r, p.E, p.k, p.logits + (size_t)t * p.E, bal, s_scratch[warp], lane, ids, p.r.topk_w + (size_t)t * p.k,
                  nullptr);
    if (lane < p.k) {
        const int e = ids[lane];                               // the lane's own write
        atomicAdd(p.hist + (size_t)c * p.E + e, 1);
        atomicAdd(sums + (size_t)(c / kSpan) * p.E + e, 1);
    }
}

// Permutation: one CTA per chunk.  Thread e adds up its expert's rows in the spans and chunks
// before this one and, over all spans, its total; the warps then take a contiguous share of
// the chunk's pairs each, count it, and rank its pairs from where the warps before end.
__global__ void __launch_bounds__(256) scored_scatter_kernel(RouteArgs p, const int32_t* sums) {
    __shared__ int s_cnt[256];
    __shared__ int s_off[257];
    __shared__ int s_run[8][256];
    griddep_wait();
    griddep_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, e = threadIdx.x;
    const int c = blockIdx.x, span = c / kSpan, n_spans = ((int)gridDim.x + kSpan - 1) / kSpan;
    int base = 0, total = 0;
    if (e < p.E) {
#pragma unroll 8
        for (int q = 0; q < n_spans; ++q) {
            const int v = __ldcg(sums + (size_t)q * p.E + e);
            total += v;
            if (q < span) base += v;
        }
#pragma unroll 8
        for (int q = span * kSpan; q < c; ++q) base += __ldcg(p.hist + (size_t)q * p.E + e);
    }
    s_cnt[e] = total;
#pragma unroll
    for (int w = 0; w < 8; ++w) s_run[w][e] = 0;
    __syncthreads();
    const int t0 = c * kChunk, pair0 = t0 * p.k, n = (min(p.T, t0 + kChunk) - t0) * p.k;
    const int share = (n + 255) / 256 * 32, b0 = min(n, warp * share), b1 = min(n, b0 + share);
    const int32_t* ids = p.r.topk_ids + pair0;
    for (int i = b0 + lane; i < b1; i += 32) atomicAdd(&s_run[warp][ids[i]], 1);
    if (warp == 0) warp_scan_counts(s_cnt, s_off, p.E, lane);
    __syncthreads();
    if (e < p.E) {
        int run = s_off[e] + base;
#pragma unroll
        for (int w = 0; w < 8; ++w) {
            const int v = s_run[w][e];
            s_run[w][e] = run;
            run += v;
        }
    }
    __syncthreads();
    warp_scatter(ids + b0, pair0 + b0, b1 - b0, s_run[warp], p.r.perm, p.r.inv_perm, lane, p.E);
    if (c != 0) return;
    if (e < p.E) {
        p.r.counts[e] = total;
        p.r.offsets[e] = s_off[e];
    }
    if (e == 0) {
        p.r.offsets[p.E] = s_off[p.E];
        p.ctrl->work[0] = 0;                              // no expert pass of this workspace runs now
        p.ctrl->work[1] = 0;
    }
    if (warp == 1) warp_active(s_cnt, p.E, p.S, p.active, p.ctrl, p.T, lane);
}

template <int NTL, int NW>
cudaError_t launch_small(const RouteArgs& a, const ScoreArgs& r, cudaStream_t s) {
    const size_t smem = sizeof(SmallSmem<NTL, NW>);
    const cudaError_t err = set_smem_limit(scored_small_kernel<NTL, NW>, smem);
    if (err != cudaSuccess) return err;
    // K parts: up to eight CTAs of a cluster, each warp of them with at least one step
    int parts = kSmParts;
    while (parts > 1 && parts * NW > a.H / kSmStep) parts /= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((a.E + kSmExperts - 1) / kSmExperts * parts);
    cfg.blockDim = dim3(32 * NW);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = parts;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, scored_small_kernel<NTL, NW>, a, r, parts);
}

}  // namespace

cudaError_t launch_route_scored(const RouteArgs& a, const ScoreArgs& r, int num_ctas, cudaStream_t s) {
    cudaError_t err;
    if (a.T <= kSmallT) {
        if (a.T <= kTailT) return launch_small<1, 8>(a, r, s);
        err = a.T <= 16 ? launch_small<2, 8>(a, r, s) : a.T <= 32 ? launch_small<4, 8>(a, r, s) : launch_small<8, 8>(a, r, s);
        if (err != cudaSuccess) return err;
        const int pairs = a.ops ? a.T * 8 * ((a.H / 64 + 7) / 8) : 0, ctas = (pairs + kChooseWarps - 1) / kChooseWarps;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((1 + (ctas + kChooseCtas - 1) / kChooseCtas) * kChooseCtas);
        cfg.blockDim = dim3(32 * kChooseWarps);
        cfg.stream = s;
        cudaLaunchAttribute attr[2];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = kChooseCtas;
        attr[1].val.clusterDim.y = 1;
        attr[1].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 2;
        return cudaLaunchKernelEx(&cfg, scored_choose_kernel, a, r);
    }
    // the spans' sums and the planes take regions of the workspace that only moe_forward uses
    const int nchunks = (a.T + kChunk - 1) / kChunk, n_sums = (nchunks + kSpan - 1) / kSpan * a.E;
    int32_t* sums = reinterpret_cast<int32_t*>(a.zx);
    const LogitPlan plan = plan_scored_logits(a, num_ctas);
    if (!plan.few) {
        err = launch_pdl(scored_split_kernel, dim3(4 * num_ctas), dim3(256), 0, s, a, a.planes, sums, n_sums);
        if (err != cudaSuccess) return err;
    }
    if ((err = launch_scored_logits(a, plan, sums, n_sums, s)) != cudaSuccess) return err;
    const int top = (a.T + kTopWarps - 1) / kTopWarps;
    if ((err = launch_pdl(scored_topk_kernel, dim3(top), dim3(32 * kTopWarps), 0, s, a, r, sums)) != cudaSuccess)
        return err;
    return launch_pdl(scored_scatter_kernel, dim3(nchunks), dim3(256), 0, s, a, (const int32_t*)sums);
}

}  // namespace moe
