// Scored router: softmax or sigmoid scores, a balance bias that steers the choice but not
// the weights, groups of experts of which the best are kept, top-k, renormalised and scaled
// weights (the routing of DeepSeek-style layers whose load is balanced by a bias).
//   L = fp32(x Wr^T + b),  s = sigmoid(L) or softmax(L),  c = s + balance
//   group score = the sum of its one or two largest c; the top_groups best groups stay
//   ids = the k largest c of those groups, w = s[ids] (/ sum of them) * scale
// The logits are fp32 as in moe_route; scores and choice are formed from them in fp64: the
// sigmoid's upper end leaves fp32 scores equal whose logits differ, and a sum of score and
// bias loses what separates two of them.
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

// One token's choice by one warp: lane l holds experts 8l .. 8l+7.  `scratch` (256 doubles of
// this warp) serves the group scores.  Each round takes the largest key over the warp in two
// 32-bit reductions (high words, then the low words of those that tie), the lowest lane and
// the lowest expert inside it first.  Writes ids and weights of slots < k.
__device__ void select_scored(const ScoreArgs& r, int E, int k, const float* row, double* scratch, int lane,
                              int32_t* ids_out, float* w_out, int32_t* s_ids) {
    float L[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) L[j] = 8 * lane + j < E ? ldcg_f32(row + 8 * lane + j) : -INFINITY;
    double s[8];
    if (r.sigmoid) {
#pragma unroll
        for (int j = 0; j < 8; ++j) s[j] = 1.0 / (1.0 + exp(-(double)L[j]));
    } else {
        float m = L[0];
#pragma unroll
        for (int j = 1; j < 8; ++j) m = fmaxf(m, L[j]);
#pragma unroll
        for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        double z = 0.0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            s[j] = exp((double)L[j] - (double)m);
            z += s[j];
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) z += shfl_xor_d(z, o);
#pragma unroll
        for (int j = 0; j < 8; ++j) s[j] /= z;
    }
    unsigned long long key[8];
    const bool grouped = r.top_groups < r.n_groups;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int e = 8 * lane + j;
        key[j] = 0;
        if (e < E) {
            const double c = r.balance ? s[j] + (double)__ldg(r.balance + e) : s[j];
            key[j] = score_key(c);
            if (grouped) scratch[e] = c == c ? c : -INFINITY;
        }
    }
    if (grouped) {
        const int gs = E / r.n_groups;
        __syncwarp();
        double sc = -INFINITY;
        if (lane < r.n_groups) {
            // the lanes start at different experts of their groups (bank conflicts)
            double t1 = -INFINITY, t2 = -INFINITY;
            int i = lane % gs;
            for (int n = 0; n < gs; ++n) {
                const double c = scratch[lane * gs + i];
                if (c > t1) {
                    t2 = t1;
                    t1 = c;
                } else if (c > t2) {
                    t2 = c;
                }
                if (++i == gs) i = 0;
            }
            sc = r.group_top == 2 ? t1 + t2 : t1;
            if (sc != sc) sc = -INFINITY;
        }
        __syncwarp();
        int rank = 0;
        for (int g = 0; g < r.n_groups; ++g) {
            const double o = __shfl_sync(0xffffffffu, sc, g);
            rank += o > sc || (o == sc && g < lane);
        }
        const unsigned kept = __ballot_sync(0xffffffffu, lane < r.n_groups && rank < r.top_groups);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (8 * lane + j < E && !((kept >> ((8 * lane + j) / gs)) & 1u)) key[j] = 0;
    }
    double my_s = 0.0;
    int my_id = 0;
    for (int n = 0; n < k; ++n) {
        unsigned long long bk = key[0];
        int bj = 0;
#pragma unroll
        for (int j = 1; j < 8; ++j)
            if (key[j] > bk) {              // strict: an equal key keeps the lower expert
                bk = key[j];
                bj = j;
            }
        const uint32_t hi = (uint32_t)(bk >> 32), lo = (uint32_t)bk;
        const uint32_t mh = __reduce_max_sync(0xffffffffu, hi);
        const uint32_t ml = __reduce_max_sync(0xffffffffu, hi == mh ? lo : 0u);
        const int wl = __ffs(__ballot_sync(0xffffffffu, hi == mh && lo == ml)) - 1;
        const int wj = __shfl_sync(0xffffffffu, bj, wl);
        double v = 0.0;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j == wj) v = s[j];
        v = __shfl_sync(0xffffffffu, v, wl);
        if (lane == n) {
            my_s = v;
            my_id = 8 * wl + wj;
        }
        if (lane == wl) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (j == wj) key[j] = 0;
        }
    }
    double w = lane < k ? my_s : 0.0;
    if (r.renormalise) {
        double sum = w;
#pragma unroll
        for (int o = 16; o; o >>= 1) sum += shfl_xor_d(sum, o);
        w = sum > 0.0 ? w / sum : 0.0;
    }
    if (lane < k) {
        ids_out[lane] = my_id;
        w_out[lane] = (float)(w * (double)r.scale);
        if (s_ids) s_ids[lane] = my_id;
    }
}

// ---------------------------------------------------------------- up to kSmallT tokens
// The router's fp32 rows are read once, straight into MMA fragments: a CTA takes 16 experts
// and a part of K (the CTAs of a cluster share the experts), a warp every 64th 32-wide step.
// A weight is split exactly into three bf16 pieces (each the rounding of what is left), so
// that x w1 + x w2 + x w3 on mma.sync has fp32-level products.  The order of K inside a
// step is free as long as both operands follow it: lane (g, t) takes elements 8t .. 8t+7 of
// its rows, 32 contiguous bytes, as the fragments of two MMAs.  A warp's sum is short (its
// few steps, the small pieces in an accumulator of their own); warps and CTAs are added in
// double-float.  The last CTA to finish (a ticket) chooses the experts and permutes.
constexpr int kSmThreads = 256, kSmWarps = 8, kSmExperts = 16, kSmStep = 32;

template <int NTL>   // 8-token MMA columns
struct SmallSmem {
    union {
        float part[kSmWarps][kSmExperts][8 * NTL];
        double scratch[kSmWarps][256];
    };
    Df sum[kSmExperts][8 * NTL];
    int32_t ids[kSmallT * 16];
    int cnt[256];
    int off[257];
    int last;
};

__device__ inline uint32_t pack_bf16x2(float lo, float hi) {
    return (uint32_t)f32_to_bf16_bits(lo) | ((uint32_t)f32_to_bf16_bits(hi) << 16);
}
__device__ inline float bf16_part(float w) { return __uint_as_float((uint32_t)f32_to_bf16_bits(w) << 16); }

template <int NTL>
__global__ void __launch_bounds__(kSmThreads) scored_small_kernel(RouteArgs p, ScoreArgs r, int parts) {
    extern __shared__ __align__(16) uint8_t smem_raw[];
    SmallSmem<NTL>& S = *reinterpret_cast<SmallSmem<NTL>*>(smem_raw);
    if (blockIdx.x == 0 && threadIdx.x == 0) {          // no expert pass of this workspace runs now
        p.ctrl->work[0] = 0;
        p.ctrl->work[1] = 0;
    }
    griddep_launch_dependents();        // one wave of CTAs: the expert pass may start launching
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
    const int part = (int)cluster_rank(), e0 = (int)(blockIdx.x / parts) * kSmExperts;
    const int steps = p.H / kSmStep;
    float hi[NTL][4], lo[NTL][4];
#pragma unroll
    for (int n = 0; n < NTL; ++n)
#pragma unroll
        for (int c = 0; c < 4; ++c) hi[n][c] = lo[n][c] = 0.f;
    const bool r0 = e0 + g < p.E, r1 = e0 + g + 8 < p.E;
    const float* w0 = p.Wr + (size_t)(e0 + g) * p.H + 8 * t4;
    const float* w1 = w0 + (size_t)8 * p.H;
#pragma unroll 2
    for (int st = part * kSmWarps + warp; st < steps; st += parts * kSmWarps) {
        const int k0 = st * kSmStep;
        float w[2][8];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float4* src = reinterpret_cast<const float4*>((h ? w1 : w0) + k0);
            const float4 z = make_float4(0.f, 0.f, 0.f, 0.f);
            const float4 a = (h ? r1 : r0) ? __ldg(src) : z, b = (h ? r1 : r0) ? __ldg(src + 1) : z;
            w[h][0] = a.x; w[h][1] = a.y; w[h][2] = a.z; w[h][3] = a.w;
            w[h][4] = b.x; w[h][5] = b.y; w[h][6] = b.z; w[h][7] = b.w;
        }
        uint4 xv[NTL];
#pragma unroll
        for (int n = 0; n < NTL; ++n) {
            const int t = 8 * n + g;
            xv[n] = t < p.T ? __ldg(reinterpret_cast<const uint4*>(p.x + (size_t)t * p.H + k0 + 8 * t4))
                            : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int pl = 0; pl < 3; ++pl) {
            uint32_t a[2][4];               // [row half][pair]
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const float u = bf16_part(w[h][2 * q]), v = bf16_part(w[h][2 * q + 1]);
                    a[h][q] = pack_bf16x2(u, v);
                    w[h][2 * q] -= u;
                    w[h][2 * q + 1] -= v;
                }
#pragma unroll
            for (int n = 0; n < NTL; ++n) {
                float(&d)[4] = pl == 0 ? hi[n] : lo[n];
                mma_bf16_16816(d[0], d[1], d[2], d[3], a[0][0], a[1][0], a[0][1], a[1][1], xv[n].x, xv[n].y);
                mma_bf16_16816(d[0], d[1], d[2], d[3], a[0][2], a[1][2], a[0][3], a[1][3], xv[n].z, xv[n].w);
            }
        }
    }
    // the decode operands of (token, group) pairs, one per warp
    if (p.ops) {
        const int G8 = 8 * ((p.H / 64 + 7) / 8);
        const OperandArgs o{p.T, p.H, p.x, p.zx, p.iq, p.ctrl};
        for (int pr = blockIdx.x * kSmWarps + warp; pr < p.T * G8; pr += gridDim.x * kSmWarps) {
            compute_z(o, pr / G8, pr % G8, lane);
            if (p.iq) compute_iq(o, pr / G8, pr % G8, lane);
        }
    }
#pragma unroll
    for (int n = 0; n < NTL; ++n)
#pragma unroll
        for (int c = 0; c < 4; ++c) S.part[warp][g + 8 * (c >> 1)][8 * n + 2 * t4 + (c & 1)] = hi[n][c] + lo[n][c];
    __syncthreads();
    for (int i = threadIdx.x; i < kSmExperts * 8 * NTL; i += kSmThreads) {
        const int e = i / (8 * NTL), t = i % (8 * NTL);
        Df v = Df{S.part[0][e][t], 0.f};
#pragma unroll
        for (int u = 1; u < kSmWarps; ++u) v = df_add(v, Df{S.part[u][e][t], 0.f});
        S.sum[e][t] = v;
    }
    __syncthreads();
    cluster_sync();
    for (int i = part * kSmThreads + threadIdx.x; i < kSmExperts * p.T; i += parts * kSmThreads) {
        const int t = i / kSmExperts, e = i % kSmExperts;
        if (e0 + e >= p.E) continue;
        const uint32_t at = smem_u32(&S.sum[e][t]);
        Df v = Df{0.f, 0.f};
        for (int q = 0; q < parts; ++q) {
            Df w;
            asm volatile("ld.shared::cluster.v2.f32 {%0,%1}, [%2];"
                         : "=f"(w.hi), "=f"(w.lo)
                         : "r"(map_peer(at, q))
                         : "memory");
            v = q ? df_add(v, w) : w;
        }
        // the bias and the one final rounding
        p.logits[(size_t)t * p.E + e0 + e] =
            (float)((double)v.hi + (double)v.lo + (p.bias ? (double)p.bias[e0 + e] : 0.0));
    }
    __threadfence();
    __syncthreads();
    cluster_sync();                     // no CTA's sums go away while another reads them
    if (threadIdx.x == 0) S.last = atomicAdd(&p.ctrl->route_ticket, 1u) == gridDim.x - 1;
    __syncthreads();
    if (!S.last) return;
    __threadfence();

    for (int i = threadIdx.x; i < 256; i += kSmThreads) S.cnt[i] = 0;
    for (int t = warp; t < p.T; t += kSmWarps)
        select_scored(r, p.E, p.k, p.logits + (size_t)t * p.E, S.scratch[warp], lane, p.r.topk_ids + (size_t)t * p.k,
                      p.r.topk_w + (size_t)t * p.k, S.ids + t * p.k);
    __syncthreads();
    for (int i = threadIdx.x; i < p.T * p.k; i += kSmThreads) atomicAdd(&S.cnt[S.ids[i]], 1);
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

// ---------------------------------------------------------------- above kSmallT tokens
// One CTA per chunk of tokens, a warp per token; the last CTA scans the chunks' histograms.
__global__ void __launch_bounds__(256) scored_topk_kernel(RouteArgs p, ScoreArgs r) {
    __shared__ double s_scratch[8][256];
    __shared__ int s_cnt[256];
    __shared__ int s_off[257];
    __shared__ int s_last;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int c = blockIdx.x;
    if (c == 0 && threadIdx.x == 0) {                   // no expert pass of this workspace runs now
        p.ctrl->work[0] = 0;
        p.ctrl->work[1] = 0;
    }
    for (int i = threadIdx.x; i < 256; i += blockDim.x) s_cnt[i] = 0;
    __syncthreads();
    const int tend = min(p.T, (c + 1) * kChunk);
    for (int t = c * kChunk + warp; t < tend; t += 8) {
        int32_t* ids = p.r.topk_ids + (size_t)t * p.k;
        select_scored(r, p.E, p.k, p.logits + (size_t)t * p.E, s_scratch[warp], lane, ids, p.r.topk_w + (size_t)t * p.k,
                      nullptr);
        if (lane < p.k) atomicAdd(&s_cnt[ids[lane]], 1);       // the lane's own write
    }
    __syncthreads();
    for (int e = threadIdx.x; e < p.E; e += blockDim.x) p.hist[(size_t)c * p.E + e] = s_cnt[e];
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) s_last = atomicAdd(&p.ctrl->topk_ticket, 1u) == gridDim.x - 1;
    __syncthreads();
    if (!s_last) return;
    __threadfence();
    chunk_scan(p, s_cnt, s_off, gridDim.x);
}

template <int NTL>
cudaError_t launch_small(const RouteArgs& a, const ScoreArgs& r, cudaStream_t s) {
    const size_t smem = sizeof(SmallSmem<NTL>);
    const cudaError_t err = set_smem_limit(scored_small_kernel<NTL>, smem);
    if (err != cudaSuccess) return err;
    // K parts: up to eight CTAs of a cluster, each warp of them with at least one step
    int parts = 8;
    while (parts > 1 && parts * kSmWarps > a.H / kSmStep) parts /= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((a.E + kSmExperts - 1) / kSmExperts * parts);
    cfg.blockDim = dim3(kSmThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = parts;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, scored_small_kernel<NTL>, a, r, parts);
}

}  // namespace

cudaError_t launch_route_scored(const RouteArgs& a, const ScoreArgs& r, cudaStream_t s) {
    if (a.T <= kSmallT) {
        if (a.T <= 8) return launch_small<1>(a, r, s);
        if (a.T <= 16) return launch_small<2>(a, r, s);
        if (a.T <= 32) return launch_small<4>(a, r, s);
        return launch_small<8>(a, r, s);
    }
    const cudaError_t err = launch_route_logits(a, s);
    if (err != cudaSuccess) return err;
    scored_topk_kernel<<<(a.T + kChunk - 1) / kChunk, 256, 0, s>>>(a, r);
    return launch_route_scatter(a, s);
}

}  // namespace moe
