// Pieces the routers share: double-float sums, the scan over experts, the permutation of the
// (token, slot) pairs and the active-expert list.
#pragma once
#include "kernels.h"

namespace moe {

__device__ inline float bf16lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ inline float bf16hi(uint32_t v) { return __uint_as_float(v & 0xFFFF0000u); }

// Double-float sums (a value is hi + lo, two fp32 numbers) with the exact two-sum
// (Knuth: s = a + b and the rounding error of that addition, both in fp32): the
// relative error of a sum of n terms is about n 2^-48 of the sum of their magnitudes.
// The decode router forms each thread's share of a logit (28 products of an fp32
// weight and a bf16 token) with fp32 fmas and adds the shares across the CTA in
// double-float, so the logit carries the rounding of 28-term partial sums only, at
// fp32 arithmetic rates (the fp64 units of this part are a small fraction of its fp32
// ones, and a double-float product costs a dozen fp32 operations).
struct Df {
    float hi, lo;
};
// (explicitly rounded operations: the compiler must not fuse or reorder them)
__device__ __forceinline__ void two_sum(float a, float b, float& s, float& err) {
    s = __fadd_rn(a, b);
    const float bp = __fsub_rn(s, a);
    err = __fadd_rn(__fsub_rn(a, __fsub_rn(s, bp)), __fsub_rn(b, bp));
}
__device__ __forceinline__ Df df_add(Df a, Df b) {
    Df r;
    float err;
    two_sum(a.hi, b.hi, r.hi, err);
    r.lo = __fadd_rn(__fadd_rn(a.lo, b.lo), err);
    return r;
}
// every lane ends with the same sum (the exact two-sum is symmetric in its arguments)
__device__ inline Df warp_sum_df(Df v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        Df w;
        w.hi = __shfl_xor_sync(0xffffffffu, v.hi, o);
        w.lo = __shfl_xor_sync(0xffffffffu, v.lo, o);
        v = df_add(v, w);
    }
    return v;
}

__device__ inline float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// The leading bf16 pieces (the upper 16 bits) of two weights as a pair; the weights keep the
// rest, exactly.  The 24 bits of a weight are used up by three of them.
__device__ inline uint32_t next_plane(float& a, float& b) {
    const uint32_t ua = __float_as_uint(a), ub = __float_as_uint(b);
    a -= __uint_as_float(ua & 0xFFFF0000u);
    b -= __uint_as_float(ub & 0xFFFF0000u);
    return __byte_perm(ua, ub, 0x7632);
}

// Exclusive scan of s_cnt[0..E) into s_off[0..E] by one warp (E <= 256).
__device__ inline void warp_scan_counts(const int* s_cnt, int* s_off, int E, int lane) {
    int loc[8];
    int sum = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        int e = lane * 8 + j;
        loc[j] = e < E ? s_cnt[e] : 0;
        sum += loc[j];
    }
    int incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        int n = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += n;
    }
    int run = incl - sum;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        int e = lane * 8 + j;
        if (e < E) s_off[e] = run;
        run += loc[j];
    }
    if (lane == 31) s_off[E] = incl;
}

// Ranks the flattened pairs [0, n) (ids in s_ids) into positions starting at
// s_run[e]; writes perm / inv_perm.  One warp; pair order = (token, slot) order.
// An id outside [0, E) (only possible with caller-given routing, which reports it) takes
// no position; its pair's inv_perm entry is set to 0 so that readers stay in bounds.
// dedup_k > 0 (caller-given routing, k = dedup_k): an id that an earlier slot of the same
// token already holds is left out as an invalid one is (the range starts on a token).
__device__ inline void warp_scatter(const int32_t* ids, int pair0, int n, int* s_run, int32_t* perm, int32_t* inv_perm,
                             int lane, int E, int dedup_k = 0) {
    const unsigned lt = (1u << lane) - 1u;
    for (int base = 0; base < n; base += 32) {
        int i = base + lane;
        int e = i < n ? ids[i] : -1;
        bool valid = i < n && e >= 0 && e < E;
        if (valid && dedup_k > 1) {
            const int sl = (pair0 + i) % dedup_k;
            for (int j = 0; j < sl; ++j)
                if (ids[i - sl + j] == e) valid = false;
        }
        if (i < n && !valid) inv_perm[pair0 + i] = 0;
        if (!valid) e = -1 - lane;
        unsigned mask = __match_any_sync(0xffffffffu, e);
        int rank = __popc(mask & lt);
        int first = valid ? s_run[e] : 0;
        __syncwarp();
        if (valid && rank == 0) s_run[e] = first + __popc(mask);
        __syncwarp();
        if (valid) {
            int pos = first + rank;
            perm[pos] = pair0 + i;
            inv_perm[pair0 + i] = pos;
        }
    }
}

// Active expert list: experts with a nonzero count (ascending), then shared experts.
__device__ inline void warp_active(const int* s_cnt, int E, int S, int32_t* active, Ctrl* ctrl, int T, int lane) {
    int n = 0;
    for (int base = 0; base < E; base += 32) {
        int e = base + lane;
        bool on = e < E && s_cnt[e] > 0;
        unsigned m = __ballot_sync(0xffffffffu, on);
        if (on) active[n + __popc(m & ((1u << lane) - 1u))] = e;
        n += __popc(m);
    }
    if (lane < S) active[n + lane] = E + lane;
    if (lane == 0) {
        ctrl->n_active = n + S;
        ctrl->routed_T = T;
    }
}

// The last CTA of a top-k kernel over chunks of kChunk tokens (all its threads): per-expert
// totals over the chunks, the exclusive scan over experts, then each chunk's base in each expert's range (offset + the expert's rows in earlier
// chunks).  A thread reads its expert's column 16 chunks at a time (independent
// loads, one L2 round trip per 16 chunks).
__device__ inline void chunk_scan(const RouteArgs& p, int* s_cnt, int* s_off, int nchunks) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int e = threadIdx.x; e < p.E; e += blockDim.x) {
        int run = 0;
        for (int q0 = 0; q0 < nchunks; q0 += 16) {
            int v[16];
#pragma unroll
            for (int u = 0; u < 16; ++u) v[u] = q0 + u < nchunks ? __ldcg(p.hist + (size_t)(q0 + u) * p.E + e) : 0;
#pragma unroll
            for (int u = 0; u < 16; ++u) run += v[u];
        }
        s_cnt[e] = run;
    }
    __syncthreads();
    if (warp == 0) warp_scan_counts(s_cnt, s_off, p.E, lane);
    __syncthreads();
    for (int e = threadIdx.x; e < p.E; e += blockDim.x) {
        p.r.counts[e] = s_cnt[e];
        p.r.offsets[e] = s_off[e];
        int run = s_off[e];
        for (int q0 = 0; q0 < nchunks; q0 += 16) {
            int v[16];
#pragma unroll
            for (int u = 0; u < 16; ++u) v[u] = q0 + u < nchunks ? __ldcg(p.hist + (size_t)(q0 + u) * p.E + e) : 0;
#pragma unroll
            for (int u = 0; u < 16; ++u) {
                if (q0 + u < nchunks) p.hist[(size_t)(q0 + u) * p.E + e] = run;
                run += v[u];
            }
        }
    }
    if (threadIdx.x == 0) p.r.offsets[p.E] = s_off[p.E];
    if (warp == 0) {
        warp_active(s_cnt, p.E, p.S, p.active, p.ctrl, p.T, lane);
        if (lane == 0) p.ctrl->topk_ticket = 0;
    }
}

}  // namespace moe
