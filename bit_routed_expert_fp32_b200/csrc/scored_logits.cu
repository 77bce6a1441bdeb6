// Router logits of many tokens on tcgen05: L = x Wr^T + b with the fp32 router split exactly
// into three bf16 planes (scored_split_kernel), so that x w1 + x w2 + x w3 has fp32-level
// products: three times the operations of one bf16 product, 180 GFLOP at 16384 tokens of the
// full-size layer (110 us at the measured bf16 rate; the tokens' 235 MB take 36 us of HBM).
//
// A pair of CTAs takes 256 tokens x up to 256 experts (cta_group::2: each CTA 128 tokens and
// half of the experts' rows; the planes are then read once per 256 tokens, which L2 can
// deliver); a stage holds 64 of K: the tokens' box and three plane boxes.  The tensor core's
// running sums are not rounded to nearest, so a chain through all of K would carry a bias
// that grows with it: every second stage (the small planes first) starts a fresh
// accumulator, two of them in turn, and eight warps add each to fp32 sums in registers while
// the next is formed (16384 tokens of the full-size layer, whole call: 193 us with an
// accumulator per stage, which the adding warps then bound, 161 us with one per two, 158 us
// with one per four).  K is also cut over the pairs of a cluster when there are few tokens;
// the parts are added through shared memory in part order, in double-float with the bias, and
// rounded once.
#include "route_common.cuh"
#include "tc5.cuh"

namespace moe {
namespace {

using namespace tc5;

constexpr int kDrain = 2;                  // stages per accumulator
constexpr int kThreads = 384, kTok = 256, kMaxStages = 6, kEpiWarps = 8;

struct LogitArgs {
    int T, H, E;
    int en;               // experts per tile (a multiple of 64, at most 256)
    int etiles;           // expert tiles
    int parts;            // K parts: pairs of a cluster
    int stages;
    uint32_t tmem_cols;   // two accumulators
    const float* bias;
    float* logits;
    Ctrl* ctrl;
};

struct LogitShared {
    uint64_t full[kMaxStages], empty_[kMaxStages], acc_full[2], acc_empty[2], drained, stall_bar;
    uint32_t tmem;
    int abort_flag;
};

__global__ void __launch_bounds__(kThreads, 1)
    scored_logits_kernel(const __grid_constant__ LogitArgs p, const __grid_constant__ CUtensorMap xmap,
                         const __grid_constant__ CUtensorMap wmap) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ LogitShared S;
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int crank = (int)cluster_rank(), rank = crank & 1, part = crank >> 1;
    const uint16_t pair_mask = (uint16_t)(3u << (crank & ~1));
    const int tile = blockIdx.x / (2 * p.parts), tt = tile / p.etiles, e0 = (tile - tt * p.etiles) * p.en;
    const int t0 = tt * kTok + rank * 128;
    const int chunks = p.H / kBK;
    const int kc0 = part * chunks / p.parts, n_stage = (part + 1) * chunks / p.parts - kc0;
    const uint32_t wbytes = (uint32_t)(p.en / 2) * kBK * 2, xbytes = 128 * kBK * 2, stage_bytes = xbytes + 3 * wbytes;

    if (threadIdx.x == 0) {
        prefetch_map(&xmap);
        prefetch_map(&wmap);
        for (int i = 0; i < p.stages; ++i) {
            mbar_init(&S.full[i], 1);
            mbar_init(&S.empty_[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&S.acc_full[i], 1);
            mbar_init(&S.acc_empty[i], 2 * kEpiWarps);
        }
        mbar_init(&S.drained, 1);
        mbar_init(&S.stall_bar, 1);                     // nothing ever arrives on it
        fence_mbar_init();
        S.abort_flag = 0;
    }
    griddep_wait();
    if (warp == 2) tmem_alloc_pair(&S.tmem, p.tmem_cols);
    fence_before();
    __syncthreads();
    cluster_sync();
    fence_after();
    griddep_launch_dependents();
    const uint32_t tmem = S.tmem;
    float acc[128];                                       // epilogue warps: this row's sums

    if (warp == 0) {
        int slot = 0, issued = 0;
        uint32_t par = 1;
        bool stop = false;
        for (int i = 0; i < n_stage; ++i) {
            if (!__all_sync(0xffffffffu, pair_wait(S.abort_flag, &S.empty_[slot], par, p.ctrl, kDetWaitEmpty | 0x70))) {
                stop = true;
                break;
            }
            if (elect_one()) {
                uint8_t* dst = smem + (size_t)slot * stage_bytes;
                const uint32_t bar = map_peer(smem_u32(&S.full[slot]), crank & ~1);
                if (rank == 0) mbar_arrive_expect_tx(&S.full[slot], 2 * stage_bytes);
                tma_load_2d_pair(dst, &xmap, (kc0 + i) * kBK, t0, bar);
#pragma unroll
                for (int pl = 0; pl < 3; ++pl)
                    tma_load_2d_pair(dst + xbytes + pl * wbytes, &wmap, (kc0 + i) * kBK,
                                     pl * p.E + e0 + rank * (p.en / 2), bar);
            }
            __syncwarp();
            ++issued;
            if (++slot == p.stages) {
                slot = 0;
                par ^= 1;
            }
        }
        if (stop && lane == 0) pair_drain(S.full, p.stages, issued, rank == 0, p.ctrl, kDetDrain | 0x70);
        __syncwarp();
    } else if (warp == 1 && rank == 0) {
        const uint32_t idesc = instr_desc(false, 256, p.en);
        const uint64_t ad0 = smem_desc(smem_u32(smem)), bd0 = smem_desc(smem_u32(smem) + xbytes);
        bool ok = true;
        const uint32_t stall = p.ctrl->test_stall;
        if (stall) {
            if (test_stall(&S.stall_bar, stall, lane)) {
                if (lane == 0) {
                    report_error(p.ctrl, MOE_ERR_TIMEOUT, kDetTestStall | 0x70);
                    pair_abort(S.abort_flag);
                }
                ok = false;
            }
            __syncwarp();
        }
        int slot = 0;
        uint32_t par = 0;
        for (int i = 0; i < n_stage && ok; ++i) {
            const int g = i / kDrain, buf = g & 1;
            const bool first = i % kDrain == 0, last = i % kDrain == kDrain - 1 || i == n_stage - 1;
            ok = (!first || pair_wait(S.abort_flag, &S.acc_empty[buf], (uint32_t)((g >> 1) & 1) ^ 1, p.ctrl,
                                      kDetWaitEmpty | 0x71)) &&
                 pair_wait(S.abort_flag, &S.full[slot], par, p.ctrl, kDetWaitFull | 0x70);
            ok = __all_sync(0xffffffffu, ok);
            fence_after();
            if (ok && elect_one()) {
                const uint64_t off = (uint64_t)slot * (stage_bytes >> 4);
#pragma unroll
                for (int pl = 2; pl >= 0; --pl)
#pragma unroll
                    for (int k16 = 0; k16 < kBK / 16; ++k16)
                        umma_ss_pair(tmem + buf * p.en, ad0 + off + 2 * k16, bd0 + off + pl * (wbytes >> 4) + 2 * k16,
                                     idesc, first && pl == 2 && k16 == 0 ? 0u : 1u);
                umma_commit_pair(&S.empty_[slot], pair_mask);
                if (last) umma_commit_pair(&S.acc_full[buf], pair_mask);
            }
            __syncwarp();
            if (++slot == p.stages) {
                slot = 0;
                par ^= 1;
            }
        }
        if (!ok) {                                        // what was issued ends before either CTA leaves
            if (elect_one()) umma_commit_pair(&S.drained, pair_mask);
            __syncwarp();
            if (!mbar_wait_bounded(&S.drained, 0, kWaitLimit)) report_error(p.ctrl, MOE_ERR_TIMEOUT, kDetDrain | 0x71);
        }
    } else if (warp >= 4) {
        // lanes 32 (warp % 4) .. of the pair's 128 rows here; half of the tile's experts
        const int q = warp & 3, half = (warp - 4) >> 2, cols = p.en / 2;
#pragma unroll
        for (int c = 0; c < 128; ++c) acc[c] = 0.f;
        for (int i = 0; i < (n_stage + kDrain - 1) / kDrain; ++i) {
            const int buf = i & 1;
            if (!__all_sync(0xffffffffu, pair_wait(S.abort_flag, &S.acc_full[buf], (uint32_t)(i >> 1) & 1, p.ctrl,
                                                   kDetWaitFull | 0x71)))
                break;
            fence_after();
            const uint32_t tl = tmem + buf * p.en + half * cols + ((uint32_t)(32 * q) << 16);
#pragma unroll
            for (int c = 0; c < 128; c += 16) {
                if (c < cols) {
                    uint32_t v[16];
                    tmem_ld16(tl + c, v);
                    ld_wait(v);
#pragma unroll
                    for (int u = 0; u < 16; ++u) acc[c + u] += __uint_as_float(v[u]);
                }
            }
            fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_peer(map_peer(smem_u32(&S.acc_empty[buf]), crank & ~1));
        }
    }
    __syncwarp();
    // every role of both CTAs is done: the last accumulator was full, so no MMA reads the
    // stages' memory any more (after an abort nothing further is read or written there)
    fence_before();
    __syncthreads();
    cluster_sync();
    fence_after();
    if (warp == 2) tmem_dealloc_pair(tmem, p.tmem_cols);
    const int ld = p.en + 4;                              // floats per row (bank spread)
    float* sums = reinterpret_cast<float*>(smem);
    const bool ok = !ld_volatile(S.abort_flag);
    if (ok && warp >= 4) {
        const int cols = p.en / 2;
        float* dst = sums + (size_t)(32 * (warp & 3) + lane) * ld + ((warp - 4) >> 2) * cols;
#pragma unroll
        for (int c = 0; c < 128; c += 4)
            if (c < cols) *reinterpret_cast<float4*>(dst + c) = make_float4(acc[c], acc[c + 1], acc[c + 2], acc[c + 3]);
    }
    __syncthreads();
    cluster_sync();
    if (ok) {
        const uint32_t sbase = smem_u32(sums);
        const int per = (128 + p.parts - 1) / p.parts, r0 = part * per, r1 = min(128, r0 + per), nq = p.en / 4;
        for (int i = r0 * nq + threadIdx.x; i < r1 * nq; i += kThreads) {
            const int r = i / nq, c = 4 * (i - r * nq), e = e0 + c;
            if (t0 + r >= p.T || e >= p.E) continue;
            const uint32_t at = sbase + (uint32_t)(r * ld + c) * 4;
            Df s[4];
            for (int q = 0; q < p.parts; ++q) {
                const float4 v = ld_peer_v4(map_peer(at, 2 * q + rank));
                const float f[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) s[j] = q ? df_add(s[j], Df{f[j], 0.f}) : Df{f[j], 0.f};
            }
            float* out = p.logits + (size_t)(t0 + r) * p.E + e;
            float o[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (p.bias && e + j < p.E) s[j] = df_add(s[j], Df{__ldg(p.bias + e + j), 0.f});
                o[j] = s[j].hi + s[j].lo;
            }
            if ((p.E & 3) == 0) {
                *reinterpret_cast<float4*>(out) = make_float4(o[0], o[1], o[2], o[3]);
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (e + j < p.E) out[j] = o[j];
            }
        }
    }
    __syncwarp();
    cluster_sync();                     // no CTA's sums go away while another reads them
}

// ---------------------------------------------------------------- few tokens
// With few tokens, or few experts, most of a pair's tile would be empty and its token boxes
// read for few columns, so the weights are the rows instead: the three planes of 40 experts
// stacked, D[3 x 40][tokens] = planes x^T, four MMAs a stage by single CTAs, K over a cluster;
// accumulators, the adding warps and the joining of parts as in the pair kernel, and the
// planes are joined there too.  (130 tokens of the full-size layer, whole call: 30.7 us by
// pairs, 25.2 us so.)
constexpr int kExp = 40, kFewSplit = 8;
constexpr uint32_t kPlanesBytes = 128 * kBK * 2;          // 120 rows, and eight that nothing reads

struct FewArgs {
    int T, H, E;
    int etiles, nt, split, stages;        // nt: tokens per tile (a multiple of 32, at most 256)
    const float* bias;
    float* logits;
    Ctrl* ctrl;
};

struct FewShared {
    uint64_t full[kMaxStages], empty_[kMaxStages], acc_full[2], acc_empty[2], done, stall_bar;
    uint32_t tmem;
    int abort_flag;
};

__global__ void __launch_bounds__(kThreads, 1)
    scored_logits_few_kernel(const __grid_constant__ FewArgs p, const __grid_constant__ CUtensorMap xmap,
                             const __grid_constant__ CUtensorMap wmap) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ FewShared S;
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int part = (int)cluster_rank();
    const int tile = blockIdx.x / p.split, tt = tile / p.etiles, e0 = (tile - tt * p.etiles) * kExp;
    const int t0 = tt * p.nt, ntok = min(p.nt, p.T - t0), chunks = p.H / kBK;
    const int kc0 = part * chunks / p.split, n_stage = (part + 1) * chunks / p.split - kc0;
    const uint32_t stage_bytes = kPlanesBytes + (uint32_t)p.nt * kBK * 2;
    const uint32_t load_bytes = 3 * kExp * kBK * 2 + (uint32_t)p.nt * kBK * 2;
    const int groups = (n_stage + kDrain - 1) / kDrain;

    if (threadIdx.x == 0) {
        prefetch_map(&xmap);
        prefetch_map(&wmap);
        for (int i = 0; i < p.stages; ++i) {
            mbar_init(&S.full[i], 1);
            mbar_init(&S.empty_[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&S.acc_full[i], 1);
            mbar_init(&S.acc_empty[i], kEpiWarps);
        }
        mbar_init(&S.done, 1);
        mbar_init(&S.stall_bar, 1);                     // nothing ever arrives on it
        fence_mbar_init();
        S.abort_flag = 0;
    }
    griddep_wait();
    if (warp == 1) tmem_alloc(&S.tmem, 512);
    fence_before();
    __syncthreads();
    fence_after();
    griddep_launch_dependents();
    const uint32_t tmem = S.tmem;
    const int cols = p.nt / 2;
    float acc[128];                                       // adding warps: this row's sums of half the tokens

    if (warp == 0) {
        int slot = 0, issued = 0;
        uint32_t par = 1;
        for (int i = 0; i < n_stage; ++i) {
            if (!__all_sync(0xffffffffu, wait_or_flag(S.abort_flag, &S.empty_[slot], par, p.ctrl, kDetWaitEmpty | 0x72)))
                break;
            if (elect_one()) {
                uint8_t* dst = smem + (size_t)slot * stage_bytes;
                mbar_arrive_expect_tx(&S.full[slot], load_bytes);
                tma_load_2d(dst + kPlanesBytes, &xmap, (kc0 + i) * kBK, t0, &S.full[slot]);
#pragma unroll
                for (int pl = 0; pl < 3; ++pl)
                    tma_load_2d(dst + pl * kExp * kBK * 2, &wmap, (kc0 + i) * kBK, pl * p.E + e0, &S.full[slot]);
            }
            __syncwarp();
            ++issued;
            if (++slot == p.stages) {
                slot = 0;
                par ^= 1;
            }
        }
        // after an abort no copy may still target shared memory at exit
        if (lane == 0 && ld_volatile(S.abort_flag)) pair_drain(S.full, p.stages, issued, true, p.ctrl, kDetDrain | 0x72);
        __syncwarp();
    } else if (warp == 1) {
        const uint32_t idesc = instr_desc(false, 128, p.nt);
        bool ok = true;
        const uint32_t stall = p.ctrl->test_stall;
        if (stall) {
            if (test_stall(&S.stall_bar, stall, lane)) {
                if (lane == 0) {
                    st_volatile(S.abort_flag, 1);
                    report_error(p.ctrl, MOE_ERR_TIMEOUT, kDetTestStall | 0x72);
                }
                ok = false;
            }
            __syncwarp();
        }
        int slot = 0;
        uint32_t par = 0;
        for (int i = 0; i < n_stage && ok; ++i) {
            const int g = i / kDrain, buf = g & 1;
            const bool first = i % kDrain == 0, last = i % kDrain == kDrain - 1 || i == n_stage - 1;
            ok = (!first || wait_or_flag(S.abort_flag, &S.acc_empty[buf], (uint32_t)((g >> 1) & 1) ^ 1, p.ctrl,
                                         kDetWaitEmpty | 0x73)) &&
                 wait_or_flag(S.abort_flag, &S.full[slot], par, p.ctrl, kDetWaitFull | 0x72);
            ok = __all_sync(0xffffffffu, ok);
            fence_after();
            if (ok && elect_one()) {
                const uint32_t base = smem_u32(smem + (size_t)slot * stage_bytes);
                const uint64_t ad = smem_desc(base), bd = smem_desc(base + kPlanesBytes);
#pragma unroll
                for (int k16 = 0; k16 < kBK / 16; ++k16)
                    umma_ss(tmem + buf * p.nt, ad + 2 * k16, bd + 2 * k16, idesc, first && k16 == 0 ? 0u : 1u);
                umma_commit(&S.empty_[slot]);
                if (last) umma_commit(&S.acc_full[buf]);
            }
            __syncwarp();
            if (++slot == p.stages) {
                slot = 0;
                par ^= 1;
            }
        }
        if (elect_one()) umma_commit(&S.done);          // every MMA issued has completed
        __syncwarp();
    } else if (warp >= 4) {
        // lanes 32 (warp % 4) .. of the tile's plane rows; half of its tokens
        const int q = warp & 3, half = (warp - 4) >> 2;
#pragma unroll
        for (int c = 0; c < 128; ++c) acc[c] = 0.f;
        for (int i = 0; i < groups; ++i) {
            const int buf = i & 1;
            if (!__all_sync(0xffffffffu, wait_or_flag(S.abort_flag, &S.acc_full[buf], (uint32_t)(i >> 1) & 1, p.ctrl,
                                                      kDetWaitFull | 0x73)))
                break;
            fence_after();
            const uint32_t tl = tmem + buf * p.nt + half * cols + ((uint32_t)(32 * q) << 16);
#pragma unroll
            for (int c = 0; c < 128; c += 16) {
                if (c < cols) {
                    uint32_t v[16];
                    tmem_ld16(tl + c, v);
                    ld_wait(v);
#pragma unroll
                    for (int u = 0; u < 16; ++u) acc[c + u] += __uint_as_float(v[u]);
                }
            }
            fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&S.acc_empty[buf]);
        }
    }
    if (!mbar_wait_bounded(&S.done, 0, kWaitLimit)) {
        st_volatile(S.abort_flag, 1);
        report_error(p.ctrl, MOE_ERR_TIMEOUT, kDetDrain | 0x73);
    }
    __syncthreads();                                    // and the producer's copies are in
    fence_after();
    // this CTA's sums, [token][plane row] fp32 over the stages' memory
    float* sums = reinterpret_cast<float*>(smem);
    const bool ok = !ld_volatile(S.abort_flag);
    if (ok && warp >= 4) {
        float* dst = sums + (size_t)((warp - 4) >> 2) * cols * 128 + 32 * (warp & 3) + lane;
#pragma unroll
        for (int c = 0; c < 128; ++c)
            if (c < cols) dst[c * 128] = acc[c];
    }
    fence_before();
    __syncthreads();
    cluster_sync();
    fence_after();
    if (warp == 1) tmem_dealloc(tmem, 512);
    if (ok) {
        const uint32_t sbase = smem_u32(sums);
        for (int i = part * kThreads + threadIdx.x; i < ntok * (kExp / 4); i += p.split * kThreads) {
            const int tok = i / (kExp / 4), c = 4 * (i % (kExp / 4)), e = e0 + c;
            if (e >= p.E) continue;
            const uint32_t at = sbase + (uint32_t)(tok * 128 + c) * 4;
            Df s[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) s[j] = Df{p.bias && e + j < p.E ? __ldg(p.bias + e + j) : 0.f, 0.f};
            for (int q = 0; q < p.split; ++q) {
                const uint32_t peer = map_peer(at, q);
                float4 v[3];
#pragma unroll
                for (int pl = 0; pl < 3; ++pl) v[pl] = ld_peer_v4(peer + pl * kExp * 4);
#pragma unroll
                for (int pl = 0; pl < 3; ++pl) {
                    const float f[4] = {v[pl].x, v[pl].y, v[pl].z, v[pl].w};
#pragma unroll
                    for (int j = 0; j < 4; ++j) s[j] = df_add(s[j], Df{f[j], 0.f});
                }
            }
            float* out = p.logits + (size_t)(t0 + tok) * p.E + e;
            if ((p.E & 3) == 0) {
                *reinterpret_cast<float4*>(out) =
                    make_float4(s[0].hi + s[0].lo, s[1].hi + s[1].lo, s[2].hi + s[2].lo, s[3].hi + s[3].lo);
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (e + j < p.E) out[j] = s[j].hi + s[j].lo;
            }
        }
    }
    __syncwarp();
    cluster_sync();                     // no CTA's sums go away while another reads them
}

cudaError_t launch_few(const FewArgs& p, const CUtensorMap& xm, const CUtensorMap& wm, int ttiles, cudaStream_t s) {
    constexpr size_t smem = 226 * 1024;                   // 512 columns: the whole SM
    const cudaError_t err = set_smem_limit(scored_logits_few_kernel, smem);
    if (err != cudaSuccess) return err;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(p.split * ttiles * p.etiles));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = p.split;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, scored_logits_few_kernel, p, xm, wm);
}

}  // namespace

cudaError_t launch_scored_logits(const RouteArgs& a, int num_ctas, cudaStream_t s) {
    LogitArgs p = {};
    p.T = a.T;
    p.H = a.H;
    p.E = a.E;
    p.bias = a.bias;
    p.logits = a.logits;
    p.ctrl = a.ctrl;
    const int ttiles = (a.T + kTok - 1) / kTok, chunks = a.H / kBK;
    // The kernel and K split with the least estimated time, in clocks: 1536 a stage of a pair
    // or 512 of a single CTA; a wave of clusters some 4000 beside its stages, joining parts
    // 2500, and for the single CTAs 16 a token of the tile.  (1024 tokens of the full-size
    // layer, whole call: 46.6 us by pairs, 44.0 us by single CTAs; 4096 tokens: the same.)
    const int ftt = (a.T + 255) / 256, fnt = ((a.T + ftt - 1) / ftt + 31) / 32 * 32, fet = (a.E + kExp - 1) / kExp;
    double best = 0.0, few_best = 0.0;
    int few_split = 1;
    p.en = (a.E + 63) / 64 * 64;
    for (int parts = 1; parts <= 4 && parts <= chunks; ++parts) {
        const int cap = cluster_capacity(2 * parts, 1, num_ctas);
        const double waves = (ttiles + cap - 1) / cap;
        const double t = waves * ((chunks + parts - 1) / parts * 1536.0 + 4000.0) + (parts > 1 ? 2500.0 : 0.0);
        if (best == 0.0 || t < best) {
            best = t;
            p.parts = parts;
        }
    }
    for (int split = 1; split <= kFewSplit && split <= chunks; ++split) {
        const int cap = cluster_capacity(split, 1, num_ctas);
        const double waves = ((int64_t)ftt * fet + cap - 1) / cap;
        const double t = waves * ((chunks + split - 1) / split * 512.0 + 4000.0 + 16.0 * fnt) + (split > 1 ? 2500.0 : 0.0);
        if (few_best == 0.0 || t < few_best) {
            few_best = t;
            few_split = split;
        }
    }
    CUtensorMap xm, wm;
    if (few_best < best) {
        FewArgs f = {a.T, a.H, a.E, fet, fnt, few_split, 0, a.bias, a.logits, a.ctrl};
        f.stages = (int)((225 * 1024) / (kPlanesBytes + fnt * kBK * 2));
        if (f.stages > kMaxStages) f.stages = kMaxStages;
        if (!make_map(&xm, false, a.x, a.T, a.H, a.H, fnt) ||
            !make_map(&wm, false, a.planes, 3 * (int64_t)a.E, a.H, a.H, kExp))
            return cudaErrorInvalidConfiguration;
        return launch_few(f, xm, wm, ftt, s);
    }
    p.etiles = (a.E + p.en - 1) / p.en;
    p.tmem_cols = 2 * p.en <= 128 ? 128 : 2 * p.en <= 256 ? 256 : 512;
    const size_t stage = 128 * kBK * 2 + (size_t)3 * (p.en / 2) * kBK * 2;
    p.stages = (int)((226 * 1024 - 1024) / stage);
    if (p.stages > kMaxStages) p.stages = kMaxStages;
    size_t smem = p.stages * stage;
    const size_t sums = (size_t)128 * (p.en + 4) * 4;
    if (smem < sums) smem = sums;
    if (smem < tmem_smem(p.tmem_cols)) smem = tmem_smem(p.tmem_cols);
    smem += 1024;
    if (smem > 226 * 1024) smem = 226 * 1024;             // 512 columns: the whole SM
    if (!make_map(&xm, false, a.x, a.T, a.H, a.H, 128) || !make_map(&wm, false, a.planes, 3 * (int64_t)a.E, a.H, a.H, p.en / 2))
        return cudaErrorInvalidConfiguration;
    cudaError_t err = set_smem_limit(scored_logits_kernel, smem);
    if (err != cudaSuccess) return err;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(2 * p.parts * ttiles * p.etiles));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 2 * p.parts;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, scored_logits_kernel, p, xm, wm);
}

}  // namespace moe
