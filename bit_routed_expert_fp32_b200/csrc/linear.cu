// Dense matrix product with its epilogue: y = act(x W^T + b) + r for 16-bit x and W, the
// products of a layer that are not packed (an expert kept at full precision, the dense FFN
// and the projections around the routed layer).
//
// One tile is 128 output features x NT tokens, D[feature][token] = W_tile x^T on tcgen05
// with the weights as the A operand: a tile has its full M whatever the token count, so one
// token costs the same weight bytes as any other count up to NT.  With SwiGLU the tile has
// two accumulators, the gate rows' and the up rows' of the same features, so that a thread
// holds both values of an output.  K is cut over the CTAs of a cluster when the tiles alone
// do not fill the GPU; each CTA leaves its fp32 sums in its shared memory and every CTA of
// the cluster adds a share of the tile from all of them, in part order (no atomics: the
// result does not depend on timing), and applies the epilogue.
#include "tc5.cuh"

namespace moe {
namespace {

using namespace tc5;

constexpr int kFeat = 128;                 // output features per tile
constexpr int kLinThreads = 128;
constexpr int kTileBytes = kFeat * kBK * 2;
constexpr int kMaxStages = 8;

struct LinKernelArgs {
    int T, N, K;
    int act, res_f32;
    int nt;                  // tokens per tile (a multiple of 16)
    int ftiles;              // feature tiles; CTA ((token tile) ftiles + feature tile) split + part
    int split;               // CTAs of a cluster: K parts
    int stages;
    uint32_t tmem_cols;
    int64_t ldr, ldy;
    const void* bias;
    const void* res;
    void* y;
    int vec;                 // 4 consecutive outputs of a row can be read and written at once
    Ctrl* ctrl;
};

template <bool F16>
__device__ inline float to_f32(uint16_t v) {
    return F16 ? __half2float(__ushort_as_half(v)) : __uint_as_float((uint32_t)v << 16);
}
template <bool F16>
__device__ inline uint16_t from_f32(float v) {
    return F16 ? f32_to_f16_bits(v) : f32_to_bf16_bits(v);
}

// silu with the fast exponential and quotient: relative error about 1e-6, far below the
// 16-bit rounding of the output
__device__ inline float silu_fast(float a) { return __fdividef(a, 1.0f + __expf(-a)); }

__device__ inline float apply_act(int act, float a) {
    switch (act) {
        case MOE_ACT_RELU: return a > 0.f || a != a ? a : 0.f;      // NaN stays NaN
        case MOE_ACT_SILU: return silu_fast(a);
        case MOE_ACT_GELU: return 0.5f * a * (1.f + erff(a * 0.70710678f));
        case MOE_ACT_GELU_TANH: return 0.5f * a * (1.f + tanhf(0.79788456f * (a + 0.044715f * a * a * a)));
    }
    return a;
}

// Shared state of a CTA.
struct LinShared {
    uint64_t full[kMaxStages], empty_[kMaxStages], done, stall_bar;
    uint32_t tmem;
    int abort_flag;
};

__device__ inline int ld_volatile(const int& v) { return *reinterpret_cast<const volatile int*>(&v); }
__device__ inline void st_volatile(int& v, int x) { *reinterpret_cast<volatile int*>(&v) = x; }

__device__ inline bool wait_or_flag(LinShared& S, uint64_t* bar, uint32_t parity, Ctrl* ctrl, uint32_t detail) {
    if (ld_volatile(S.abort_flag)) return false;
    if (mbar_wait_bounded(bar, parity, kWaitLimit)) return true;
    st_volatile(S.abort_flag, 1);
    report_error(ctrl, MOE_ERR_TIMEOUT, detail);
    return false;
}

template <bool F16, bool GLU>
__global__ void __launch_bounds__(kLinThreads) linear_kernel(const __grid_constant__ LinKernelArgs p,
                                                             const __grid_constant__ CUtensorMap wmap,
                                                             const __grid_constant__ CUtensorMap xmap) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ LinShared S;
    constexpr int kPlanes = GLU ? 2 : 1;
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int part = p.split > 1 ? (int)cluster_rank() : 0;
    const int tile = blockIdx.x / p.split, tt = tile / p.ftiles;
    const int f0 = (tile - tt * p.ftiles) * kFeat, t0 = tt * p.nt;
    const int ntok = min(p.nt, p.T - t0);
    const int chunks = (p.K + kBK - 1) / kBK;
    const int kc0 = (int)((int64_t)part * chunks / p.split), kc1 = (int)((int64_t)(part + 1) * chunks / p.split);
    const int n_stage = kc1 - kc0;
    const int stage_bytes = kPlanes * kTileBytes + p.nt * kBK * 2;

    if (threadIdx.x == 0) {
        prefetch_map(&wmap);
        prefetch_map(&xmap);
        for (int i = 0; i < p.stages; ++i) {
            mbar_init(&S.full[i], 1);
            mbar_init(&S.empty_[i], 1);
        }
        mbar_init(&S.done, 1);
        mbar_init(&S.stall_bar, 1);                     // nothing ever arrives on it
        fence_mbar_init();
        S.abort_flag = 0;
    }
    griddep_wait();
    if (warp == 1) tmem_alloc(&S.tmem, p.tmem_cols);
    fence_before();
    __syncthreads();
    fence_after();
    griddep_launch_dependents();
    const uint32_t tmem = S.tmem;

    if (warp == 0) {
        int issued = 0;
        for (int i = 0; i < n_stage; ++i) {
            const int s = i % p.stages;
            const uint32_t par = ((uint32_t)(i / p.stages) & 1) ^ 1;
            if (!mbar_try_wait(&S.empty_[s], par)) wait_or_flag(S, &S.empty_[s], par, p.ctrl, kDetWaitEmpty | 0x60);
            __syncwarp();
            if (ld_volatile(S.abort_flag)) break;
            if (elect_one()) {
                uint8_t* dst = smem + (size_t)s * stage_bytes;
                mbar_arrive_expect_tx(&S.full[s], stage_bytes);
                tma_load_2d(dst, &wmap, (kc0 + i) * kBK, f0, &S.full[s]);
                if (GLU) tma_load_2d(dst + kTileBytes, &wmap, (kc0 + i) * kBK, p.N + f0, &S.full[s]);
                tma_load_2d(dst + kPlanes * kTileBytes, &xmap, (kc0 + i) * kBK, t0, &S.full[s]);
            }
            __syncwarp();
            issued = i + 1;
        }
        // after an abort no copy may still target shared memory: wait (bounded) for the last
        // phase issued on every slot
        if (lane == 0 && ld_volatile(S.abort_flag))
            for (int d = 0; d < p.stages && d < issued; ++d) {
                const int i = issued - 1 - d;
                if (!mbar_wait_bounded(&S.full[i % p.stages], (uint32_t)(i / p.stages) & 1, kWaitLimit)) {
                    report_error(p.ctrl, MOE_ERR_TIMEOUT, kDetDrain | 0x60);
                    break;
                }
            }
    } else if (warp == 1) {
        const uint32_t idesc = instr_desc(F16, kFeat, p.nt);
        bool ok = true;
        const uint32_t stall = p.ctrl->test_stall;
        if (stall) {
            // failure-path tests: a bounded wait on a barrier that nothing completes
            bool got = false;
            if (lane == 0) got = mbar_wait_bounded(&S.stall_bar, 0, stall);
            if (!__shfl_sync(0xffffffffu, got, 0)) {
                if (lane == 0) {
                    st_volatile(S.abort_flag, 1);
                    report_error(p.ctrl, MOE_ERR_TIMEOUT, kDetTestStall | 0x60);
                }
                ok = false;
            }
            __syncwarp();
        }
        for (int i = 0; i < n_stage && ok; ++i) {
            const int s = i % p.stages;
            const uint32_t par = (uint32_t)(i / p.stages) & 1;
            if (!mbar_try_wait(&S.full[s], par)) ok = wait_or_flag(S, &S.full[s], par, p.ctrl, kDetWaitFull | 0x60);
            ok = __all_sync(0xffffffffu, ok);
            fence_after();
            if (ok && elect_one()) {
                const uint32_t base = smem_u32(smem + (size_t)s * stage_bytes);
                const uint64_t ad = smem_desc(base), bd = smem_desc(base + kPlanes * kTileBytes);
#pragma unroll
                for (int k16 = 0; k16 < kBK / 16; ++k16) {
                    const uint32_t acc = (i | k16) != 0 ? 1u : 0u;
                    umma_ss(tmem, ad + 2 * k16, bd + 2 * k16, idesc, acc);
                    if (GLU) umma_ss(tmem + p.nt, ad + (kTileBytes >> 4) + 2 * k16, bd + 2 * k16, idesc, acc);
                }
                umma_commit(&S.empty_[s]);
            }
            __syncwarp();
        }
        if (elect_one()) umma_commit(&S.done);          // every MMA issued has completed
        __syncwarp();
    }
    if (!mbar_wait_bounded(&S.done, 0, kWaitLimit)) {
        st_volatile(S.abort_flag, 1);
        report_error(p.ctrl, MOE_ERR_TIMEOUT, kDetDrain | 0x61);
    }
    __syncthreads();                                    // and the producer's copies are in
    fence_after();
    // this CTA's sums, [plane][token][feature] fp32 over the stages' memory
    float* sums = reinterpret_cast<float*>(smem);
    const bool ok = !ld_volatile(S.abort_flag);
    if (ok) {
        const uint32_t tl = tmem + ((uint32_t)(32 * warp) << 16);
#pragma unroll
        for (int pl = 0; pl < kPlanes; ++pl)
            for (int c = 0; c < ntok; c += 16) {
                uint32_t v[16];
                tmem_ld16(tl + pl * p.nt + c, v);
                ld_wait();
#pragma unroll
                for (int u = 0; u < 16; ++u)
                    sums[(size_t)(pl * p.nt + c + u) * kFeat + threadIdx.x] = __uint_as_float(v[u]);
            }
    }
    fence_before();
    __syncthreads();
    if (p.split > 1) cluster_sync();
    fence_after();
    if (warp == 1) tmem_dealloc(tmem, p.tmem_cols);
    if (ok) {
        const uint32_t sbase = smem_u32(sums);
        for (int i = part * kLinThreads + threadIdx.x; i < ntok * (kFeat / 4); i += p.split * kLinThreads) {
            const int tok = i / (kFeat / 4), f = 4 * (i % (kFeat / 4)), n = f0 + f;
            if (n >= p.N) continue;
            float a[kPlanes][4];
#pragma unroll
            for (int pl = 0; pl < kPlanes; ++pl) {
                const uint32_t at = sbase + (uint32_t)(((pl * p.nt + tok) * kFeat + f) * 4);
                float4 v = *reinterpret_cast<const float4*>(sums + (size_t)(pl * p.nt + tok) * kFeat + f);
                if (p.split > 1) {
                    v = ld_peer_v4(map_peer(at, 0));
                    for (int q = 1; q < p.split; ++q) {
                        const float4 w = ld_peer_v4(map_peer(at, q));
                        v.x += w.x;
                        v.y += w.y;
                        v.z += w.z;
                        v.w += w.w;
                    }
                }
                a[pl][0] = v.x;
                a[pl][1] = v.y;
                a[pl][2] = v.z;
                a[pl][3] = v.w;
            }
            const int64_t t = t0 + tok;
            uint16_t out[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (n + j >= p.N) break;
                float v = a[0][j];
                if (p.bias) v += to_f32<F16>(static_cast<const uint16_t*>(p.bias)[n + j]);
                if (GLU) {
                    float u = a[kPlanes - 1][j];
                    if (p.bias) u += to_f32<F16>(static_cast<const uint16_t*>(p.bias)[p.N + n + j]);
                    v = silu_fast(v) * u;
                } else {
                    v = apply_act(p.act, v);
                }
                if (p.res) {
                    const int64_t ri = t * p.ldr + n + j;
                    v += p.res_f32 ? static_cast<const float*>(p.res)[ri]
                                   : to_f32<F16>(static_cast<const uint16_t*>(p.res)[ri]);
                }
                out[j] = from_f32<F16>(v);
            }
            uint16_t* yp = static_cast<uint16_t*>(p.y) + t * p.ldy + n;
            if (p.vec && n + 3 < p.N) {
                *reinterpret_cast<uint2*>(yp) = make_uint2(out[0] | ((uint32_t)out[1] << 16),
                                                           out[2] | ((uint32_t)out[3] << 16));
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (n + j < p.N) yp[j] = out[j];
            }
        }
    }
    // no CTA's shared memory goes away while another reads it
    __syncwarp();
    if (p.split > 1) cluster_sync();
}

template <bool F16, bool GLU>
cudaError_t launch(const LinearArgs& a, cudaStream_t s) {
    constexpr int planes = GLU ? 2 : 1, max_nt = GLU ? 128 : 256;
    LinKernelArgs p = {};
    p.T = a.T;
    p.N = a.N;
    p.K = a.K;
    p.act = a.act;
    p.res_f32 = a.res_f32;
    p.ldr = a.ldr;
    p.ldy = a.ldy;
    p.bias = a.bias;
    p.res = a.res;
    p.y = a.y;
    p.ctrl = a.ctrl;
    p.vec = a.ldy % 4 == 0 && (reinterpret_cast<uintptr_t>(a.y) & 7) == 0;
    const int ttiles = (a.T + max_nt - 1) / max_nt;
    p.nt = ((a.T + ttiles - 1) / ttiles + 15) & ~15;
    p.tmem_cols = 32;
    while ((int)p.tmem_cols < planes * p.nt) p.tmem_cols *= 2;
    p.ftiles = (a.N + kFeat - 1) / kFeat;
    const int chunks = (a.K + kBK - 1) / kBK;
    const int64_t tiles = (int64_t)p.ftiles * ttiles;
    p.split = 1;
    while (p.split < 8 && tiles * p.split < 148 && p.split * 4 <= chunks) p.split *= 2;
    const int per = (chunks + p.split - 1) / p.split;
    const int stage_bytes = planes * kTileBytes + p.nt * kBK * 2;
    const int sums_bytes = planes * p.nt * kFeat * 4;
    p.stages = (200 * 1024) / stage_bytes;
    if (p.stages > kMaxStages) p.stages = kMaxStages;
    if (p.stages > per) p.stages = per;
    size_t smem = (size_t)p.stages * stage_bytes;
    if (smem < (size_t)sums_bytes) smem = sums_bytes;
    if (smem < tmem_smem(p.tmem_cols)) smem = tmem_smem(p.tmem_cols);
    smem += 1024;
    CUtensorMap wm, xm;
    if (!make_map(&wm, F16, a.w, (int64_t)planes * a.N, a.K, a.ldw, kFeat) ||
        !make_map(&xm, F16, a.x, a.T, a.K, a.ldx, p.nt))
        return cudaErrorInvalidConfiguration;
    if (tiles * p.split > INT32_MAX) return cudaErrorInvalidConfiguration;
    cudaError_t err = set_smem_limit(linear_kernel<F16, GLU>, smem);
    if (err != cudaSuccess) return err;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(tiles * p.split));
    cfg.blockDim = dim3(kLinThreads);
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
    cfg.numAttrs = p.split > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, linear_kernel<F16, GLU>, p, wm, xm);
}

}  // namespace

cudaError_t launch_linear(const LinearArgs& a, cudaStream_t s) {
    if (a.act == MOE_ACT_SWIGLU) return a.f16 ? launch<true, true>(a, s) : launch<false, true>(a, s);
    return a.f16 ? launch<true, false>(a, s) : launch<false, false>(a, s);
}

}  // namespace moe
