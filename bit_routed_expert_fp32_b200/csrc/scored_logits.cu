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
// With few tokens, or few experts, most of a pair's tile would be empty, so the weights are the
// rows instead: the three planes of 40 experts stacked, D[3 x 40][tokens] = planes x^T, four MMAs
// a stage by single CTAs, K over a cluster; accumulators, the adding warps and the joining of
// parts as in the pair kernel, and the planes are joined there too.  The planes are formed
// here: the stage brings the fp32 rows, and a warp per stage splits them into the operand's
// swizzled layout.  (Full-size layer, whole call: 130 tokens 24.9 us with planes written by a
// kernel before, 21.4 us with them formed here, 34 us by pairs; 512 tokens 33.7, 29.8 and 34 us.
// A stage takes some 960 clocks whatever its tokens, so that the pairs win from 768 tokens:
// 2048 tokens 59 us against 76 us.)
constexpr int kExp = 40, kFewSplit = 8, kFewStages = 5, kFewThreads = 512, kFewTok = 128;
constexpr int kAddWarp0 = 8;                              // warps 2 .. 6 split, 8 .. 15 add
constexpr uint32_t kRowsBytes = kExp * kBK * 4;           // fp32 rows
constexpr uint32_t kPlanesBytes = 128 * kBK * 2;          // 120 rows, and eight that nothing reads

struct FewArgs {
    int T, H, E;
    int etiles, nt, split;       // nt: tokens per tile (a multiple of 32, at most kFewTok)
    const float* bias;
    float* logits;
    int32_t *hist, *sums;        // zeroed for the kernels that follow
    int n_hist, n_sums;
    Ctrl* ctrl;
};

struct FewShared {
    uint64_t full[kFewStages], split[kFewStages], empty_[kFewStages], acc_full[2], acc_empty[2], done, stall_bar;
    uint32_t tmem;
    int abort_flag;
};

__global__ void __launch_bounds__(kFewThreads, 1)
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
    // a stage: planes, tokens, fp32 rows
    const uint32_t xbytes = (uint32_t)p.nt * kBK * 2, stage_bytes = kPlanesBytes + xbytes + kRowsBytes;
    const int groups = (n_stage + kDrain - 1) / kDrain;

    if (threadIdx.x == 0) {
        prefetch_map(&xmap);
        prefetch_map(&wmap);
        for (int i = 0; i < kFewStages; ++i) {
            mbar_init(&S.full[i], 1);
            mbar_init(&S.split[i], 1);
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
    if (warp == 1) tmem_alloc(&S.tmem, 256);
    const int64_t id0 = (int64_t)blockIdx.x * kFewThreads + threadIdx.x, ids = (int64_t)gridDim.x * kFewThreads;
    for (int64_t i = id0; i < p.n_hist; i += ids) p.hist[i] = 0;
    for (int64_t i = id0; i < p.n_sums; i += ids) p.sums[i] = 0;
    fence_before();
    __syncthreads();
    fence_after();
    griddep_launch_dependents();
    const uint32_t tmem = S.tmem;
    const int cols = p.nt / 2;
    float acc[kFewTok / 2];                               // adding warps: this row's sums of half the tokens

    if (warp == 0) {
        int slot = 0, issued = 0;
        uint32_t par = 1;
        for (int i = 0; i < n_stage; ++i) {
            if (!__all_sync(0xffffffffu, mbar_try_wait(&S.empty_[slot], par) ||
                                             wait_or_flag(S.abort_flag, &S.empty_[slot], par, p.ctrl, kDetWaitEmpty | 0x72)))
                break;
            if (elect_one()) {
                uint8_t* dst = smem + (size_t)slot * stage_bytes + kPlanesBytes;
                const int k0 = (kc0 + i) * kBK;
                mbar_arrive_expect_tx(&S.full[slot], xbytes + kRowsBytes);
                tma_load_2d(dst + xbytes, &wmap, k0, e0, &S.full[slot]);
                tma_load_2d(dst, &xmap, k0, t0, &S.full[slot]);
            }
            __syncwarp();
            ++issued;
            if (++slot == kFewStages) {
                slot = 0;
                par ^= 1;
            }
        }
        // after an abort no copy may still target shared memory at exit
        if (lane == 0 && ld_volatile(S.abort_flag)) pair_drain(S.full, kFewStages, issued, true, p.ctrl, kDetDrain | 0x72);
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
        bool ready = false;
        for (int i = 0; i < n_stage && ok; ++i) {
            const int g = i / kDrain, buf = g & 1;
            const bool first = i % kDrain == 0, last = i % kDrain == kDrain - 1 || i == n_stage - 1;
            // a slot that is split has its tokens too: the splitting warp waited for both
            if (!ready)
                ok = (!first || wait_or_flag(S.abort_flag, &S.acc_empty[buf], (uint32_t)((g >> 1) & 1) ^ 1, p.ctrl,
                                             kDetWaitEmpty | 0x73)) &&
                     wait_or_flag(S.abort_flag, &S.split[slot], par, p.ctrl, kDetWaitFull | 0x72);
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
            if (++slot == kFewStages) {
                slot = 0;
                par ^= 1;
            }
            // a wait is some 130 clocks of this warp's time: the next stage's are begun together
            if (i + 1 == n_stage) break;
            ready = mbar_try_wait(&S.split[slot], par);
            if (last) ready &= mbar_try_wait(&S.acc_empty[buf ^ 1], (uint32_t)(((g + 1) >> 1) & 1) ^ 1);
        }
        if (elect_one()) umma_commit(&S.done);          // every MMA issued has completed
        __syncwarp();
    } else if (warp < kAddWarp0) {
        // A warp per slot, so that the slots' waits, reads and writes overlap (and a warp sees every
        // phase of the barrier it waits on); eight weights at a time, one 16-byte piece of each
        // plane's row.
        const int slot = warp - 2;
        for (int i = slot; i < n_stage && slot < kFewStages; i += kFewStages) {
            const uint32_t par = (uint32_t)(i / kFewStages) & 1;
            if (!__all_sync(0xffffffffu, mbar_try_wait(&S.full[slot], par) ||
                                             wait_or_flag(S.abort_flag, &S.full[slot], par, p.ctrl, kDetWaitFull | 0x75)))
                break;
            uint8_t* planes = smem + (size_t)slot * stage_bytes;
            const uint8_t* rows = planes + kPlanesBytes + xbytes;
#pragma unroll 5
            for (int u = 0; u < kExp / 4; ++u) {
                const int row = 4 * u + (lane >> 3), piece = lane & 7;
                const float4* src = reinterpret_cast<const float4*>(rows + row * (kBK * 4) + piece * 32);
                const float4 a = src[0], b = src[1];
                float w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
                for (int pl = 0; pl < 3; ++pl) {
                    uint32_t o[4];
#pragma unroll
                    for (int q = 0; q < 4; ++q) o[q] = next_plane(w[2 * q], w[2 * q + 1]);
                    // the 128-byte swizzle; a plane's 40 rows are five of its 1024-byte blocks
                    *reinterpret_cast<uint4*>(planes + pl * kExp * 128 + row * 128 + ((piece ^ (row & 7)) << 4)) =
                        make_uint4(o[0], o[1], o[2], o[3]);
                }
            }
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&S.split[slot]);
        }
    } else {
        // lanes 32 (warp % 4) .. of the tile's plane rows; half of its tokens
        const int q = warp & 3, half = (warp - kAddWarp0) >> 2;
#pragma unroll
        for (int c = 0; c < kFewTok / 2; ++c) acc[c] = 0.f;
        for (int i = 0; i < groups; ++i) {
            const int buf = i & 1;
            const uint32_t par = (uint32_t)(i >> 1) & 1;
            if (!__all_sync(0xffffffffu, mbar_try_wait(&S.acc_full[buf], par) ||
                                             wait_or_flag(S.abort_flag, &S.acc_full[buf], par, p.ctrl, kDetWaitFull | 0x73)))
                break;
            fence_after();
            const uint32_t tl = tmem + buf * p.nt + half * cols + ((uint32_t)(32 * q) << 16);
#pragma unroll
            for (int c = 0; c < kFewTok / 2; c += 16) {
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
    if (ok && warp >= kAddWarp0) {
        float* dst = sums + (size_t)((warp - kAddWarp0) >> 2) * cols * 128 + 32 * (warp & 3) + lane;
#pragma unroll
        for (int c = 0; c < kFewTok / 2; ++c)
            if (c < cols) dst[c * 128] = acc[c];
    }
    fence_before();
    __syncthreads();
    cluster_sync();
    fence_after();
    if (warp == 1) tmem_dealloc(tmem, 256);
    if (ok) {
        const uint32_t sbase = smem_u32(sums);
        for (int i = part * kFewThreads + threadIdx.x; i < ntok * (kExp / 4); i += p.split * kFewThreads) {
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
    const size_t smem = kFewStages * (kPlanesBytes + (size_t)p.nt * kBK * 2 + kRowsBytes) + 1024;   // > half an SM
    const cudaError_t err = set_smem_limit(scored_logits_few_kernel, kMaxDynSmem);
    if (err != cudaSuccess) return err;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(p.split * ttiles * p.etiles));
    cfg.blockDim = dim3(kFewThreads);
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

LogitPlan plan_scored_logits(const RouteArgs& a, int num_ctas) {
    // The kernel, its tile and K split with the least estimated time, in clocks: a stage of a pair
    // 800 and 3 an expert of the tile, one of a single CTA 960; a wave of clusters some 4000 beside
    // its stages, joining parts 2500, for the single CTAs 16 a token of the tile, and 6000 for the
    // kernel that writes the pairs' planes.  (Full-size layer, whole call, tiles of 64, 128 and 256
    // experts: 1024 tokens 44.8, 40.8 and 48.8 us, 3000 tokens 106, 75.6 and 63.2 us.)
    LogitPlan best = {};
    const int ptt = (a.T + kTok - 1) / kTok, chunks = a.H / kBK;
    double clocks = 0.0;
    for (int cut = 1; cut <= 4; cut *= 2) {
        const int en = ((a.E + cut - 1) / cut + 63) / 64 * 64;
        const int64_t tiles = (int64_t)ptt * ((a.E + en - 1) / en);
        const double stage = 800.0 + 3.0 * en;
        for (int parts = 1; parts <= 4 && parts <= chunks; ++parts) {
            const int cap = cluster_capacity(2 * parts, 1, num_ctas);
            const double waves = (double)((tiles + cap - 1) / cap);
            const double t =
                6000.0 + waves * ((chunks + parts - 1) / parts * stage + 4000.0) + (parts > 1 ? 2500.0 : 0.0);
            if (clocks == 0.0 || t < clocks) {
                clocks = t;
                best = {false, parts, en, ptt};
            }
        }
    }
    const int ttiles = (a.T + kFewTok - 1) / kFewTok, nt = ((a.T + ttiles - 1) / ttiles + 31) / 32 * 32;
    const int64_t tiles = (int64_t)ttiles * ((a.E + kExp - 1) / kExp);
    for (int split = 1; split <= kFewSplit && split <= chunks; ++split) {
        const int cap = cluster_capacity(split, 1, num_ctas);
        const double waves = (tiles + cap - 1) / cap;
        const double t = waves * ((chunks + split - 1) / split * 960.0 + 4000.0 + 16.0 * nt) + (split > 1 ? 2500.0 : 0.0);
        if (t < clocks) {
            clocks = t;
            best = {true, split, nt, ttiles};
        }
    }
    return best;
}

cudaError_t launch_scored_logits(const RouteArgs& a, const LogitPlan& plan, int32_t* sums, int n_sums, cudaStream_t s) {
    CUtensorMap xm, wm;
    if (plan.few) {
        const FewArgs f = {a.T,      a.H,    a.E,  (a.E + kExp - 1) / kExp, plan.nt, plan.parts, a.bias, a.logits,
                           a.hist,   sums,   (a.T + kChunk - 1) / kChunk * a.E, n_sums, a.ctrl};
        if (!make_map(&xm, false, a.x, a.T, a.H, a.H, plan.nt) || !make_map_f32(&wm, a.Wr, a.E, a.H, a.H, kExp))
            return cudaErrorInvalidConfiguration;
        return launch_few(f, xm, wm, plan.ttiles, s);
    }
    LogitArgs p = {};
    p.T = a.T;
    p.H = a.H;
    p.E = a.E;
    p.bias = a.bias;
    p.logits = a.logits;
    p.ctrl = a.ctrl;
    const int ttiles = plan.ttiles;
    p.parts = plan.parts;
    p.en = plan.nt;
    p.etiles = (a.E + p.en - 1) / p.en;
    p.tmem_cols = 2 * p.en <= 128 ? 128 : 2 * p.en <= 256 ? 256 : 512;
    const size_t stage = 128 * kBK * 2 + (size_t)3 * (p.en / 2) * kBK * 2;
    p.stages = (int)((kMaxDynSmem - 1024) / stage);
    if (p.stages > kMaxStages) p.stages = kMaxStages;
    size_t smem = p.stages * stage;
    const size_t joined = (size_t)128 * (p.en + 4) * 4;
    if (smem < joined) smem = joined;
    if (smem < tmem_smem(p.tmem_cols)) smem = tmem_smem(p.tmem_cols);
    smem += 1024;
    if (smem > kMaxDynSmem) smem = kMaxDynSmem;           // 512 columns: the whole SM
    if (!make_map(&xm, false, a.x, a.T, a.H, a.H, 128) || !make_map(&wm, false, a.planes, 3 * (int64_t)a.E, a.H, a.H, p.en / 2))
        return cudaErrorInvalidConfiguration;
    cudaError_t err = set_smem_limit(scored_logits_kernel, kMaxDynSmem);
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
