// Dense matrix product with its epilogue: y = act(x W^T + b) + r for 16-bit x and W, the
// products of a layer that are not packed (an expert kept at full precision, the dense FFN
// and the projections around the routed layer).
//
// One tile is 128 output features x NT tokens, D[feature][token] = W_tile x^T on tcgen05
// with the weights as the A operand: a tile has its full M whatever the token count, so one
// token costs the same weight bytes as any other count up to NT.  With SwiGLU the tile's 128
// weight rows are the gate and the up rows of 64 features.  K is cut over the CTAs of a
// cluster when the tiles alone do not fill the GPU; each CTA leaves its fp32 sums in its
// shared memory and every CTA of the cluster adds a share of the tile from all of them, in
// part order (no atomics: the result does not depend on timing), and applies the epilogue.
// Sending the sums to the CTA that adds them, instead of its reading them, measured slower
// (one token, 2048 -> 7168: 10.4 against 9.0 us): the barrier then waits for remote stores.
//
// Sums are fp32 throughout.  The tensor core truncates its running sums instead of rounding them:
// through K = 7168 a sum comes out 7e-6 of its size too small on average, 1.5 % of half a step of
// fp16 and 0.2 % of bf16's, as in any 16-bit product on this part (the library's has the same
// share of outputs that are not the nearest value: fp16 2.8 %, with sums that round 0.6 %).  A fresh
// accumulator every so often, as the router's logits have it, would cost the pair kernel the
// epilogue's overlap.
#include "tc5.cuh"

namespace moe {
namespace {

using namespace tc5;

constexpr int kFeat = 128;                 // output features per tile
constexpr int kLinThreads = 256;
constexpr int kTileBytes = kFeat * kBK * 2;
constexpr int kMaxStages = 4;
constexpr int kMaxSplit = 8;               // K parts: the CTAs of a cluster (the portable size)

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
    int vec, vec_res;        // 4 consecutive values of a row of y / the residual can be moved at once
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

template <bool F16>
__device__ inline void unpack8(const uint4& v, float (&f)[8]) {
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if (F16) {
            const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&u[j]));
            f[2 * j] = p.x;
            f[2 * j + 1] = p.y;
        } else {
            f[2 * j] = __uint_as_float(u[j] << 16);
            f[2 * j + 1] = __uint_as_float(u[j] & 0xFFFF0000u);
        }
    }
}
// Two values rounded, the first in the low half.
template <bool F16>
__device__ inline uint32_t pack2(float lo, float hi) {
    uint32_t r;
    if (F16) asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    else asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// a / (1 + e^-z) = a (2^-15 / (2^-15 + 2^(-z log2 e - 15))): so scaled, the divisor leaves the range
// of the approximate reciprocal only below z = -97, where a times it is less than half of bf16's
// smallest value (unscaled from -87 on, where SiLU is still 1e-36).  The relative error, some 2^-22
// and 2^-23 |z|, is far below the output's rounding.
__device__ inline float sigmoid_times(float a, float z) {
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(fmaf(z, -1.44269504f, -15.f)));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(e + 0x1p-15f));
    return a * (r * 0x1p-15f);
}
__device__ inline float silu_fast(float a) { return sigmoid_times(a, a); }

__device__ inline float apply_act(int act, float a) {
    switch (act) {
        case MOE_ACT_RELU: return a > 0.f || a != a ? a : 0.f;      // NaN stays NaN
        case MOE_ACT_SILU: return silu_fast(a);
        case MOE_ACT_GELU: {
            // a Phi(a), Phi(-|a|) = q = erfc(x) / 2 with x = |a| / sqrt 2, and erfc(x) = e^-x^2 t P(t),
            // t = 1 / (1 + 3/8 x): the form of Abramowitz and Stegun's 7.1.26 with seven terms,
            // fitted for the least relative error up to x = 9.6 (6.4e-7; theirs is small beside 1
            // only, 8e-4 of GELU's value at -4).  (GELU prompts take 1 to 5 % longer than with
            // their five terms: 2048 tokens 2048 -> 4096 31.3 against 30.5 us.)
            const float t = __fdividef(1.f, fmaf(0.26516504f, fabsf(a), 1.f));
            float q = fmaf(-0.1350959f, t, 0.38793784f);
            q = fmaf(q, t, -0.12959732f);
            q = fmaf(q, t, 0.28306157f);
            q = fmaf(q, t, 0.16666456f);
            q = fmaf(q, t, 0.21568918f);
            q = fmaf(q, t, 0.21133944f);
            q = 0.5f * t * q * __expf(-0.5f * a * a);
            return a != a ? a : a * (a < 0.f ? q : 1.f - q);
        }
        case MOE_ACT_GELU_TANH: {
            // (1 + tanh z) / 2 = 1 / (1 + e^-2z)
            return sigmoid_times(a, 1.59576912f * (a + 0.044715f * a * a * a));
        }
    }
    return a;
}

// Up to four consecutive residual values (index i on; n valid) into r.
template <bool F16>
__device__ inline void load_res4(const void* res, int f32, bool vec, int64_t i, int n, float (&r)[4]) {
    if (f32) {
        const float* src = static_cast<const float*>(res) + i;
        if (vec) {
            const float4 v = *reinterpret_cast<const float4*>(src);
            r[0] = v.x;
            r[1] = v.y;
            r[2] = v.z;
            r[3] = v.w;
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (j < n) r[j] = src[j];
        }
    } else {
        const uint16_t* src = static_cast<const uint16_t*>(res) + i;
        if (vec) {
            const uint2 v = *reinterpret_cast<const uint2*>(src);
            r[0] = to_f32<F16>(v.x & 0xFFFF);
            r[1] = to_f32<F16>(v.x >> 16);
            r[2] = to_f32<F16>(v.y & 0xFFFF);
            r[3] = to_f32<F16>(v.y >> 16);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (j < n) r[j] = to_f32<F16>(src[j]);
        }
    }
}
// The output's one rounding, and up to four consecutive stores (n valid).
template <bool F16>
__device__ inline void store4(uint16_t* dst, bool vec, int n, const float (&o)[4]) {
    const uint32_t a = from_f32<F16>(o[0]), b = from_f32<F16>(o[1]), c = from_f32<F16>(o[2]), d = from_f32<F16>(o[3]);
    if (vec) {
        *reinterpret_cast<uint2*>(dst) = make_uint2(a | (b << 16), c | (d << 16));
    } else {
        dst[0] = (uint16_t)a;
        if (n > 1) dst[1] = (uint16_t)b;
        if (n > 2) dst[2] = (uint16_t)c;
        if (n > 3) dst[3] = (uint16_t)d;
    }
}
// Whether groups of four values of a row (4-aligned columns) can be moved at once.
inline bool vec4_ok(const void* base, int64_t ld, int size) {
    return ld % 4 == 0 && reinterpret_cast<uintptr_t>(base) % (4 * size) == 0;
}

// The activation of a thread's R x 4 values, the choice outside the loops.
template <int R>
__device__ inline void apply_act_all(int act, float (&o)[R][4]) {
#define MOE_ACT_LOOP(A)                                                                      \
    case A:                                                                                  \
        _Pragma("unroll") for (int i = 0; i < R; ++i) _Pragma("unroll") for (int j = 0; j < 4; ++j) \
            o[i][j] = apply_act(A, o[i][j]);                                                 \
        break;
    switch (act) {
        MOE_ACT_LOOP(MOE_ACT_RELU)
        MOE_ACT_LOOP(MOE_ACT_SILU)
        MOE_ACT_LOOP(MOE_ACT_GELU)
        MOE_ACT_LOOP(MOE_ACT_GELU_TANH)
        default: break;
    }
#undef MOE_ACT_LOOP
}

// Shared state of a CTA.
struct LinShared {
    uint64_t full[kMaxStages], empty_[kMaxStages], done, stall_bar;
    uint32_t tmem;
    int abort_flag;
};

// The outputs of a tile from the parts' sums: a thread forms four columns of every (split *
// kPer)th token.  All that depends on the columns is outside the loop, and up to how many parts
// there are (P) is known to the compiler: with two warps a scheduler the loop takes what its
// instructions and branches take (130 tokens 2048 -> 4096, the kernel without it 5.9 us: with the
// column's work in the loop 9.6 us, so 8.5; 2048 -> 2 x 4096 with P fixed at eight 13.5 us, so 12.7).
template <bool F16, bool GLU, int P>
__device__ inline void linear_outputs(const LinKernelArgs& p, const float* sums, int part, int t0, int ntok, int f0) {
    constexpr int kOut = GLU ? kFeat / 2 : kFeat, kPer = kLinThreads / (kOut / 4);
    const int f = 4 * (threadIdx.x % (kOut / 4)), n = f0 + f;
    if (n >= p.N) return;
    const bool full = n + 3 < p.N, vec_res = p.vec_res && full, vec = p.vec && full;
    uint32_t at[P];
#pragma unroll
    for (int q = 0; q < P; ++q)
        if (q < p.split) at[q] = map_peer(smem_u32(sums) + f * 4, q);
    float bias[4] = {0.f, 0.f, 0.f, 0.f}, bias_up[4] = {0.f, 0.f, 0.f, 0.f};
    if (p.bias) {
        const uint16_t* b = static_cast<const uint16_t*>(p.bias) + n;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (n + j < p.N) {
                bias[j] = to_f32<F16>(b[j]);
                if (GLU) bias_up[j] = to_f32<F16>(b[p.N + j]);
            }
    }
    // four sums from every part, in part order
    auto total = [&](uint32_t off, const float(&b)[4], float(&a)[4]) {
        float4 v[P];
#pragma unroll
        for (int q = 0; q < P; ++q)
            if (q < p.split) v[q] = ld_peer_v4(at[q] + off);
        a[0] = v[0].x;
        a[1] = v[0].y;
        a[2] = v[0].z;
        a[3] = v[0].w;
#pragma unroll
        for (int q = 1; q < P; ++q)
            if (q < p.split) {
                a[0] += v[q].x;
                a[1] += v[q].y;
                a[2] += v[q].z;
                a[3] += v[q].w;
            }
#pragma unroll
        for (int j = 0; j < 4; ++j) a[j] += b[j];
    };
    const int tok0 = part * kPer + threadIdx.x / (kOut / 4), step = p.split * kPer;
    uint16_t* y = static_cast<uint16_t*>(p.y) + (int64_t)(t0 + tok0) * p.ldy + n;
    int64_t ri = (int64_t)(t0 + tok0) * p.ldr + n;
    for (int tok = tok0; tok < ntok; tok += step, y += step * p.ldy, ri += step * p.ldr) {
        float res[4] = {0.f, 0.f, 0.f, 0.f}, o[1][4], u[4];
        if (p.res) load_res4<F16>(p.res, p.res_f32, vec_res, ri, p.N - n, res);
        total(tok * kFeat * 4, bias, o[0]);
        if (GLU) {
            total((tok * kFeat + kOut) * 4, bias_up, u);
#pragma unroll
            for (int j = 0; j < 4; ++j) o[0][j] = silu_fast(o[0][j]) * u[j];
        } else {
            apply_act_all(p.act, o);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) o[0][j] += res[j];
        store4<F16>(y, vec, p.N - n, o[0]);
    }
}

template <bool F16, bool GLU>
__global__ void __launch_bounds__(kLinThreads, 2) linear_kernel(const __grid_constant__ LinKernelArgs p,
                                                             const __grid_constant__ CUtensorMap wmap,
                                                             const __grid_constant__ CUtensorMap xmap) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ LinShared S;
    constexpr int kOut = GLU ? kFeat / 2 : kFeat;       // outputs per tile
    constexpr int kPer = kLinThreads / (kOut / 4);      // tokens a CTA forms at a time, four outputs a thread
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int part = p.split > 1 ? (int)cluster_rank() : 0;
    const int tile = blockIdx.x / p.split, tt = tile / p.ftiles;
    const int f0 = (tile - tt * p.ftiles) * kOut, t0 = tt * p.nt;
    const int ntok = min(p.nt, p.T - t0);
    const int chunks = (p.K + kBK - 1) / kBK;
    const int kc0 = (int)((int64_t)part * chunks / p.split), kc1 = (int)((int64_t)(part + 1) * chunks / p.split);
    const int n_stage = kc1 - kc0;
    const int stage_bytes = kTileBytes + p.nt * kBK * 2;

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
        int issued = 0, s = 0;
        uint32_t par = 1;
        for (int i = 0; i < n_stage; ++i) {
            if (!mbar_try_wait(&S.empty_[s], par)) wait_or_flag(S.abort_flag, &S.empty_[s], par, p.ctrl, kDetWaitEmpty | 0x60);
            __syncwarp();
            if (ld_volatile(S.abort_flag)) break;
            if (elect_one()) {
                uint8_t* dst = smem + (size_t)s * stage_bytes;
                mbar_arrive_expect_tx(&S.full[s], stage_bytes);
                tma_load_2d(dst, &wmap, (kc0 + i) * kBK, f0, &S.full[s]);
                if (GLU) tma_load_2d(dst + kTileBytes / 2, &wmap, (kc0 + i) * kBK, p.N + f0, &S.full[s]);
                tma_load_2d(dst + kTileBytes, &xmap, (kc0 + i) * kBK, t0, &S.full[s]);
            }
            __syncwarp();
            issued = i + 1;
            if (++s == p.stages) {
                s = 0;
                par ^= 1;
            }
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
            if (test_stall(&S.stall_bar, stall, lane)) {
                if (lane == 0) {
                    st_volatile(S.abort_flag, 1);
                    report_error(p.ctrl, MOE_ERR_TIMEOUT, kDetTestStall | 0x60);
                }
                ok = false;
            }
            __syncwarp();
        }
        bool ready = false;
        int s = 0;
        uint32_t par = 0;
        for (int i = 0; i < n_stage && ok; ++i) {
            if (!ready && !mbar_try_wait(&S.full[s], par)) ok = wait_or_flag(S.abort_flag, &S.full[s], par, p.ctrl, kDetWaitFull | 0x60);
            ok = __all_sync(0xffffffffu, ok);
            fence_after();
            if (ok && elect_one()) {
                const uint32_t base = smem_u32(smem + (size_t)s * stage_bytes);
                const uint64_t ad = smem_desc(base), bd = smem_desc(base + kTileBytes);
#pragma unroll
                for (int k16 = 0; k16 < kBK / 16; ++k16)
                    umma_ss(tmem, ad + 2 * k16, bd + 2 * k16, idesc, (i | k16) != 0 ? 1u : 0u);
                umma_commit(&S.empty_[s]);
            }
            __syncwarp();
            if (++s == p.stages) {
                s = 0;
                par ^= 1;
            }
            if (i + 1 < n_stage) ready = mbar_try_wait(&S.full[s], par);
        }
        if (elect_one()) umma_commit(&S.done);          // every MMA issued has completed
        __syncwarp();
    } else {
        // the bias, and the residual rows of this CTA's share of the tile (kPer tokens of every
        // split * kPer, see below), on their way to L2 meanwhile
        const int width = min(kOut, p.N - f0), id = threadIdx.x - 64;
        if (p.bias && id < 2 * kOut / 64) {
            const int j = id % (kOut / 64);
            prefetch_l2(static_cast<const uint16_t*>(p.bias) + (GLU ? id / (kOut / 64) * p.N : 0) + f0 +
                        min(64 * j, width - 1));
        }
        if (p.res) {
            const int rsize = p.res_f32 ? 4 : 2, lines = (width * rsize + 254) / 128;
            for (int i = id;; i += kLinThreads - 64) {
                const int j = i / lines, tok = (part + p.split * (j / kPer)) * kPer + j % kPer;
                if (tok - j % kPer >= ntok) break;
                if (tok < ntok)
                    prefetch_l2(static_cast<const uint8_t*>(p.res) + ((int64_t)(t0 + tok) * p.ldr + f0) * rsize +
                                min((i - j * lines) * 128, width * rsize - 1));
            }
        }
    }
    if (!mbar_wait_bounded(&S.done, 0, kWaitLimit)) {
        st_volatile(S.abort_flag, 1);
        report_error(p.ctrl, MOE_ERR_TIMEOUT, kDetDrain | 0x61);
    }
    __syncthreads();                                    // and the producer's copies are in
    fence_after();
    // this CTA's sums, [token][weight row of the tile] fp32 over the stages' memory
    float* sums = reinterpret_cast<float*>(smem);
    const bool ok = !ld_volatile(S.abort_flag);
    if (ok) {
        // warps w and w + 4 share the lanes 32 (w % 4) .., taking 16 columns in turn
        const uint32_t tl = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
        for (int c = 16 * (warp >> 2); c < ntok; c += 32) {
            uint32_t v[16];
            tmem_ld16(tl + c, v);
            ld_wait(v);
#pragma unroll
            for (int u = 0; u < 16; ++u) sums[(size_t)(c + u) * kFeat + (threadIdx.x & 127)] = __uint_as_float(v[u]);
        }
    }
    fence_before();
    __syncthreads();
    if (p.split > 1) cluster_sync();
    fence_after();
    if (warp == 1) tmem_dealloc(tmem, p.tmem_cols);
    if (ok) {
        if (p.split == 1) linear_outputs<F16, GLU, 1>(p, sums, part, t0, ntok, f0);
        else if (p.split == 2) linear_outputs<F16, GLU, 2>(p, sums, part, t0, ntok, f0);
        else if (p.split <= 4) linear_outputs<F16, GLU, 4>(p, sums, part, t0, ntok, f0);
        else linear_outputs<F16, GLU, kMaxSplit>(p, sums, part, t0, ntok, f0);
    }
    // no CTA's shared memory goes away while another reads it
    __syncwarp();
    if (p.split > 1) cluster_sync();
}

// How the tile kernel runs a product, and the clocks that is estimated to take.
struct TilePlan {
    int nt, ttiles, ftiles, split, stages;
    uint32_t tmem_cols;
    size_t smem;
    double clocks;
};

TilePlan plan_tiles(const LinearArgs& a) {
    const bool glu = a.act == MOE_ACT_SWIGLU;
    const int chunks = (a.K + kBK - 1) / kBK, out = glu ? kFeat / 2 : kFeat;
    TilePlan best = {};
    // Tiles of at most 128 tokens (one of up to 160 where that is all of them): tensor memory
    // and shared memory then let two CTAs share an SM.
    best.ttiles = a.T <= 160 ? 1 : (a.T + 127) / 128;
    best.nt = (int)(((int64_t)a.T + best.ttiles - 1) / best.ttiles + 15) & ~15;
    best.ftiles = (a.N - 1) / out + 1;
    best.tmem_cols = 32;
    while ((int)best.tmem_cols < best.nt) best.tmem_cols *= 2;
    const int64_t tiles = (int64_t)best.ftiles * best.ttiles;
    const int stage_bytes = kTileBytes + best.nt * kBK * 2;
    for (int split = 1; split <= kMaxSplit && (split == 1 || split * 2 <= chunks); ++split) {
        TilePlan p = best;
        // stages: four, or as many as two CTAs on an SM leave room for
        const int fit = p.nt <= 128 ? 112 * 1024 / stage_bytes : 4, per = (chunks + split - 1) / split;
        p.split = split;
        p.stages = fit < 4 ? fit : 4;
        if (p.stages > per) p.stages = per;
        p.smem = (size_t)p.stages * stage_bytes;
        const size_t sums = (size_t)p.nt * kFeat * 4;
        if (p.smem < sums) p.smem = sums;
        if (p.smem < tmem_smem(p.tmem_cols)) p.smem = tmem_smem(p.tmem_cols);
        p.smem += 1024;
        int per_sm = (int)(228 * 1024 / (p.smem + 1024 + sizeof(LinShared)));
        per_sm = per_sm < 1 ? 1 : per_sm > 2 ? 2 : per_sm;
        // The stages' bytes come at the 64 a clock that L2 gives an SM, if there are enough of them
        // in flight for some 2400 clocks; the sums of a token of the tile take some 45 clocks; a
        // wave some 7000 beside that (launch, first load, barriers).  (16 tokens, 2048 -> 7168:
        // 11.4 us with one part, 8.0 with two, 7.7 with three, 7.3 with four, 11.8 with six, in a
        // second wave; 384 tokens, 4096 -> 4096: 20.6 us with two, 28.9 with three, whose 96
        // clusters do not fit at once.)
        const int64_t cap = (int64_t)cluster_capacity(split, per_sm, a.num_ctas);
        const int64_t waves = (tiles + cap - 1) / cap, ctas = tiles * split;
        const int64_t share = ctas <= a.num_ctas ? 1 : per_sm;
        const double flight = (double)share * p.stages * stage_bytes / 2400.0, rate = flight < 64.0 ? flight : 64.0;
        p.clocks = (double)waves * (share * per * (stage_bytes / rate) + 7000.0 + 45.0 * p.nt);
        // more parts where it makes no difference: less is left to each CTA's first load
        if (best.split == 0 || p.clocks <= 1.02 * best.clocks) best = p;
    }
    return best;
}

template <bool F16, bool GLU>
cudaError_t launch(const LinearArgs& a, const TilePlan& pl, cudaStream_t s) {
    constexpr int kOut = GLU ? kFeat / 2 : kFeat;
    LinKernelArgs p = {};
    p.T = a.T;
    p.N = a.N;
    p.K = a.K;
    p.act = a.act;
    p.res_f32 = a.res_f32;
    p.nt = pl.nt;
    p.ftiles = pl.ftiles;
    p.split = pl.split;
    p.stages = pl.stages;
    p.tmem_cols = pl.tmem_cols;
    p.ldr = a.ldr;
    p.ldy = a.ldy;
    p.bias = a.bias;
    p.res = a.res;
    p.y = a.y;
    p.ctrl = a.ctrl;
    p.vec = vec4_ok(a.y, a.ldy, 2);
    p.vec_res = vec4_ok(a.res, a.ldr, a.res_f32 ? 4 : 2);
    const int64_t ctas = (int64_t)pl.ftiles * pl.ttiles * pl.split;
    if (ctas > INT32_MAX) return cudaErrorInvalidConfiguration;
    CUtensorMap wm, xm;
    if (!make_map(&wm, F16, a.w, (int64_t)(GLU ? 2 : 1) * a.N, a.K, a.ldw, kOut) ||
        !make_map(&xm, F16, a.x, a.T, a.K, a.ldx, p.nt))
        return cudaErrorInvalidConfiguration;
    cudaError_t err = set_smem_limit(linear_kernel<F16, GLU>, kMaxDynSmem);
    if (err != cudaSuccess) return err;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(kLinThreads);
    cfg.dynamicSmemBytes = pl.smem;
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

// ---------------------------------------------------------------- many tokens
// Tiles of 256 tokens x 256 weight rows by pairs of CTAs (cta_group::2: D[token][feature],
// each CTA 128 tokens, half of the weight rows from each CTA's shared memory), persistent
// over the tiles, two accumulators in tensor memory, so that the epilogue of a tile overlaps
// the main loop of the next.  With SwiGLU the 256 weight rows are the gate and the up rows
// of 128 features (one CTA brings the former, the other the latter): both values of an
// output lie 128 columns apart in one thread's lane.
// Epilogue (8 warps, two per 32 token rows, each half of the columns): 32 columns at a time
// through a shared-memory square (16-byte pieces swizzled by the row, so that both directions
// are free of bank conflicts), after which loads and stores run along the rows; the residual
// of the next 32 columns is on its way meanwhile.
constexpr int kPairThreads = 384, kPairTok = 256, kPairStages = 6, kPairCols = 512;
constexpr int kPairEpi = 8;                             // epilogue warps (warps 4 .. 11)
constexpr int kPairStageBytes = 2 * 128 * kBK * 2;      // a CTA's share: 128 token rows, 128 weight rows
constexpr size_t kPairSmem = 227 * 1024 - 1024;         // the whole SM (with the static part): 512 columns

struct PairArgs {
    int T, N, K, act, res_f32;
    int ttiles, ftiles;      // tiles along tokens and outputs
    int group;               // token tiles that share a sweep over the outputs (L2 reuse)
    int64_t ldr, ldy;
    const void* bias;
    const void* res;
    void* y;
    int vec, vec8;           // 4 / 8 consecutive values of a row of y can be written at once
    int vec_res;             // 4 consecutive residual values can be read at once
    int vec_bias;            // 8 consecutive bias values can be read at once
    Ctrl* ctrl;
};

struct PairShared {
    uint64_t full[kPairStages], empty_[kPairStages], acc_full[2], acc_empty[2], peer_ready, drained, stall_bar;
    uint32_t tmem;
    int abort_flag;
};

__device__ inline void pair_tile(const PairArgs& p, int tile, int& tt, int& ft) {
    const int per = p.group * p.ftiles, g = tile / per, r = tile - g * per;
    const int rows = min(p.group, p.ttiles - g * p.group);
    ft = r / rows;
    tt = g * p.group + r - ft * rows;
}

template <bool F16, bool GLU>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads, 1)
    linear_pair_kernel(const __grid_constant__ PairArgs p, const __grid_constant__ CUtensorMap wmap,
                       const __grid_constant__ CUtensorMap xmap) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ PairShared S;
    constexpr int kOut = GLU ? 128 : 256;                // outputs per tile
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = (int)cluster_rank();
    const int n_tiles = p.ttiles * p.ftiles, chunks = (p.K + kBK - 1) / kBK;
    const int pair = blockIdx.x >> 1, n_pairs = gridDim.x >> 1;

    if (threadIdx.x == 0) {
        prefetch_map(&wmap);
        prefetch_map(&xmap);
        for (int i = 0; i < kPairStages; ++i) {
            mbar_init(&S.full[i], 1);
            mbar_init(&S.empty_[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&S.acc_full[i], 1);
            mbar_init(&S.acc_empty[i], 2 * kPairEpi);    // the epilogue warps of both CTAs
        }
        mbar_init(&S.peer_ready, 1);
        mbar_init(&S.drained, 1);
        mbar_init(&S.stall_bar, 1);                     // nothing ever arrives on it
        fence_mbar_init();
        S.abort_flag = 0;
    }
    __syncthreads();
    cluster_sync();                                     // both CTAs' barriers exist
    griddep_wait();
    if (warp == 2) {
        tmem_alloc_pair(&S.tmem, kPairCols);
        // the leader's MMAs write both CTAs' columns
        if (rank == 1 && lane == 0) mbar_arrive_peer(map_peer(smem_u32(&S.peer_ready), 0));
        __syncwarp();
    }
    if (warp != 0 && warp != 3) {                       // all but the producer, which needs no columns
        fence_before();
        named_bar_sync(1, kPairThreads - 64);
        fence_after();
        griddep_launch_dependents();
    }

    if (warp == 0) {
        // ---- producer: this CTA's rows, counted on the leader's barrier -----------------
        int slot = 0, issued = 0;
        uint32_t par = 1;
        bool stop = false;
        for (int tile = pair; tile < n_tiles && !stop; tile += n_pairs) {
            int tt, ft;
            pair_tile(p, tile, tt, ft);
            const int trow = tt * kPairTok + rank * 128;
            const int wrow = GLU ? rank * p.N + ft * kOut : ft * kOut + rank * 128;
            for (int kc = 0; kc < chunks; ++kc) {
                if (!__all_sync(0xffffffffu, pair_wait(S.abort_flag, &S.empty_[slot], par, p.ctrl, kDetWaitEmpty | 0x62))) {
                    stop = true;
                    break;
                }
                if (elect_one()) {
                    uint8_t* dst = smem + (size_t)slot * kPairStageBytes;
                    const uint32_t bar = map_peer(smem_u32(&S.full[slot]), 0);
                    if (rank == 0) mbar_arrive_expect_tx(&S.full[slot], 2 * kPairStageBytes);
                    tma_load_2d_pair(dst, &xmap, kc * kBK, trow, bar);
                    tma_load_2d_pair(dst + 128 * kBK * 2, &wmap, kc * kBK, wrow, bar);
                }
                __syncwarp();
                ++issued;
                if (++slot == kPairStages) {
                    slot = 0;
                    par ^= 1;
                }
            }
        }
        if (stop && lane == 0) pair_drain(S.full, kPairStages, issued, rank == 0, p.ctrl, kDetDrain | 0x62);
        __syncwarp();
    } else if (warp == 1 && rank == 0) {
        // ---- MMA issuer (the leader's) ----------------------------------------------------
        const uint32_t tmem = S.tmem;
        constexpr uint32_t idesc = instr_desc(F16, 256, 256);
        const uint64_t ad0 = smem_desc(smem_u32(smem)), bd0 = smem_desc(smem_u32(smem) + 128 * kBK * 2);
        const uint32_t stall = p.ctrl->test_stall;
        bool ok = true;
        if (stall) {
            if (test_stall(&S.stall_bar, stall, lane)) {
                if (lane == 0) {
                    report_error(p.ctrl, MOE_ERR_TIMEOUT, kDetTestStall | 0x62);
                    pair_abort(S.abort_flag);
                }
                ok = false;
            }
            __syncwarp();
        }
        if (ok) ok = __all_sync(0xffffffffu, pair_wait(S.abort_flag, &S.peer_ready, 0, p.ctrl, kDetWaitFull | 0x64));
        int slot = 0, n = 0;
        uint32_t par = 0;
        for (int tile = pair; tile < n_tiles && ok; tile += n_pairs, ++n) {
            const int buf = n & 1;
            ok = pair_wait(S.abort_flag, &S.acc_empty[buf], (uint32_t)((n >> 1) & 1) ^ 1, p.ctrl, kDetWaitEmpty | 0x63);
            ok = __all_sync(0xffffffffu, ok);
            fence_after();
            for (int kc = 0; kc < chunks && ok; ++kc) {
                ok = pair_wait(S.abort_flag, &S.full[slot], par, p.ctrl, kDetWaitFull | 0x62);
                ok = __all_sync(0xffffffffu, ok);
                fence_after();
                if (ok && elect_one()) {
                    const uint64_t off = (uint64_t)slot * (kPairStageBytes >> 4);
#pragma unroll
                    for (int k16 = 0; k16 < kBK / 16; ++k16)
                        umma_ss_pair(tmem + buf * 256, ad0 + off + 2 * k16, bd0 + off + 2 * k16, idesc,
                                     (kc | k16) != 0 ? 1u : 0u);
                    umma_commit_pair(&S.empty_[slot]);
                }
                __syncwarp();
                if (++slot == kPairStages) {
                    slot = 0;
                    par ^= 1;
                }
            }
            if (ok && elect_one()) umma_commit_pair(&S.acc_full[buf]);
            __syncwarp();
        }
        // The last tile's accumulator was full before anyone leaves; after an abort, what was
        // issued must end here.
        if (!ok) {
            if (elect_one()) umma_commit_pair(&S.drained, 1);
            __syncwarp();
            if (!mbar_wait_bounded(&S.drained, 0, kWaitLimit)) report_error(p.ctrl, MOE_ERR_TIMEOUT, kDetDrain | 0x63);
            __syncwarp();
        }
    } else if (warp >= 4) {
        // ---- epilogue -----------------------------------------------------------------
        const int q = warp & 3, half = (warp - 4) >> 2;   // tensor-memory lanes 32q .. 32q+31; columns
        constexpr int kCols = kOut / 2;                   // of this warp
        float4* const sq = reinterpret_cast<float4*>(smem + (size_t)kPairStages * kPairStageBytes) + (warp - 4) * 256;
        const int lr = lane >> 3, c4 = lane & 7;          // row (of 4) and 16-byte piece, along the rows
        const bool res16 = p.res && !p.res_f32;
        int n = 0;
        for (int tile = pair; tile < n_tiles; tile += n_pairs, ++n) {
            int tt, ft;
            pair_tile(p, tile, tt, ft);
            const int buf = n & 1;
            const int t0 = tt * kPairTok + rank * 128 + 32 * q, nb = ft * kOut + half * kCols;
            // whole columns in aligned rows move four values at a time; otherwise a lane keeps to one
            // column, so that the single values of a row still move together.  Rows past the last
            // token (and columns past the last) read its residual and are not written.
            const bool whole = t0 < p.T && nb + kCols <= p.N && p.vec && (!p.res || p.vec_res);
            const int left = p.T - t0;
            // without a residual the values are rounded before they change lanes: half the bytes
            const bool packed = whole && p.vec8 && !p.res && (!p.bias || p.vec_bias);
            uint4 rbuf[8];
            auto load_res = [&](int c0) {
                const int64_t at = (int64_t)t0 * p.ldr + nb + c0 + 4 * c4;
                if (!whole) {                              // row 4 i + j in piece j of rbuf[i], res16 as it is
                    const int64_t col = (int64_t)t0 * p.ldr + min(nb + c0 + lane, p.N - 1);
                    auto rows = [&](auto* src) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            uint32_t f[4];
#pragma unroll
                            for (int j = 0; j < 4; ++j) f[j] = src[min(4 * i + j, left - 1) * p.ldr];
                            rbuf[i] = make_uint4(f[0], f[1], f[2], f[3]);
                        }
                    };
                    if (res16) rows(static_cast<const uint16_t*>(p.res) + col);
                    else rows(static_cast<const uint32_t*>(p.res) + col);
                } else if (res16) {
                    const uint16_t* src = static_cast<const uint16_t*>(p.res) + at;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const uint2 v = *reinterpret_cast<const uint2*>(src + min(4 * i + lr, left - 1) * p.ldr);
                        rbuf[i].x = v.x;
                        rbuf[i].y = v.y;
                    }
                } else {
                    const float* src = static_cast<const float*>(p.res) + at;
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        rbuf[i] = *reinterpret_cast<const uint4*>(src + min(4 * i + lr, left - 1) * p.ldr);
                }
            };
            if (p.res && left > 0) load_res(0);
            if (!__all_sync(0xffffffffu,
                            pair_wait(S.abort_flag, &S.acc_full[buf], (uint32_t)(n >> 1) & 1, p.ctrl, kDetWaitFull | 0x63)))
                break;
            fence_after();
            const uint32_t tl = S.tmem + buf * 256 + half * kCols + ((uint32_t)(32 * q) << 16);
#pragma unroll 1
            for (int c0 = 0; c0 < kCols; c0 += 32) {
                const int n0 = nb + c0, nc = n0 + 4 * c4;
                if (n0 >= p.N) break;
                uint32_t v[32];
                tmem_ld32(tl + c0, v);
                ld_wait(v);
                if (GLU) {
                    // both accumulators' values of an output are in one lane
                    uint32_t u[32];
                    tmem_ld32(tl + 128 + c0, u);
                    ld_wait(u);
                    if (p.bias) {
                        const uint16_t* bp = static_cast<const uint16_t*>(p.bias) + n0;
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if (n0 + j < p.N) {
                                v[j] = __float_as_uint(__uint_as_float(v[j]) + to_f32<F16>(bp[j]));
                                u[j] = __float_as_uint(__uint_as_float(u[j]) + to_f32<F16>(bp[p.N + j]));
                            }
                    }
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        v[j] = __float_as_uint(silu_fast(__uint_as_float(v[j])) * __uint_as_float(u[j]));
                }
                if (packed) {
                    if (!GLU) {
                        if (p.bias) {
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                float b[8];
                                unpack8<F16>(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.bias) + n0)[j], b);
#pragma unroll
                                for (int u = 0; u < 8; ++u)
                                    v[8 * j + u] = __float_as_uint(__uint_as_float(v[8 * j + u]) + b[u]);
                            }
                        }
                        float o[8][4];
#pragma unroll
                        for (int j = 0; j < 32; ++j) o[j >> 2][j & 3] = __uint_as_float(v[j]);
                        apply_act_all(p.act, o);
#pragma unroll
                        for (int j = 0; j < 32; ++j) v[j] = __float_as_uint(o[j >> 2][j & 3]);
                    }
                    uint4* const sp = reinterpret_cast<uint4*>(sq);
                    __syncwarp();
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        uint32_t w[4];
#pragma unroll
                        for (int u = 0; u < 4; ++u)
                            w[u] = pack2<F16>(__uint_as_float(v[8 * j + 2 * u]), __uint_as_float(v[8 * j + 2 * u + 1]));
                        sp[lane * 4 + (j ^ ((lane >> 1) & 3))] = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                    __syncwarp();
                    uint16_t* yp = static_cast<uint16_t*>(p.y) + (int64_t)(t0 + (lane >> 2)) * p.ldy + n0 + 8 * (lane & 3);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int r = 8 * i + (lane >> 2);
                        if (r < left)
                            *reinterpret_cast<uint4*>(yp + 8 * i * p.ldy) = sp[r * 4 + ((lane & 3) ^ ((r >> 1) & 3))];
                    }
                    continue;
                }
                __syncwarp();
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    sq[lane * 8 + (j ^ (lane & 7))] =
                        make_float4(__uint_as_float(v[4 * j]), __uint_as_float(v[4 * j + 1]),
                                    __uint_as_float(v[4 * j + 2]), __uint_as_float(v[4 * j + 3]));
                __syncwarp();
                float o[8][4];
                if (whole) {                               // o[i][j]: row 4 i + lr, column 4 c4 + j
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int r = 4 * i + lr;
                        const float4 f = sq[r * 8 + (c4 ^ (r & 7))];
                        o[i][0] = f.x;
                        o[i][1] = f.y;
                        o[i][2] = f.z;
                        o[i][3] = f.w;
                    }
                } else {                                   // o[i][j]: row 4 i + j, column lane
                    const float* sf = reinterpret_cast<const float*>(sq) + (lane & 3);
#pragma unroll
                    for (int i = 0; i < 8; ++i)
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const int r = 4 * i + j;
                            o[i][j] = sf[4 * (r * 8 + ((lane >> 2) ^ (r & 7)))];
                        }
                }
                if (!GLU) {
                    if (p.bias) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const int col = min(whole ? nc + j : n0 + lane, p.N - 1);
                            const float b = to_f32<F16>(static_cast<const uint16_t*>(p.bias)[col]);
#pragma unroll
                            for (int i = 0; i < 8; ++i) o[i][j] += b;
                        }
                    }
                    apply_act_all(p.act, o);
                }
                uint16_t* yp = static_cast<uint16_t*>(p.y) + (int64_t)(t0 + lr) * p.ldy + nc;
                if (p.res && left > 0) {
                    if (!res16) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            o[i][0] += __uint_as_float(rbuf[i].x);
                            o[i][1] += __uint_as_float(rbuf[i].y);
                            o[i][2] += __uint_as_float(rbuf[i].z);
                            o[i][3] += __uint_as_float(rbuf[i].w);
                        }
                    } else if (whole) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            o[i][0] += to_f32<F16>(rbuf[i].x & 0xFFFF);
                            o[i][1] += to_f32<F16>(rbuf[i].x >> 16);
                            o[i][2] += to_f32<F16>(rbuf[i].y & 0xFFFF);
                            o[i][3] += to_f32<F16>(rbuf[i].y >> 16);
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            o[i][0] += to_f32<F16>(rbuf[i].x);
                            o[i][1] += to_f32<F16>(rbuf[i].y);
                            o[i][2] += to_f32<F16>(rbuf[i].z);
                            o[i][3] += to_f32<F16>(rbuf[i].w);
                        }
                    }
                    if (c0 + 32 < kCols) load_res(c0 + 32);
                }
                if (whole) {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (4 * i + lr < left) store4<F16>(yp + 4 * i * p.ldy, true, 4, o[i]);
                } else if (n0 + lane < p.N) {
                    uint16_t* yc = static_cast<uint16_t*>(p.y) + (int64_t)t0 * p.ldy + n0 + lane;
#pragma unroll
                    for (int i = 0; i < 8; ++i)
#pragma unroll
                        for (int j = 0; j < 4; ++j, yc += p.ldy)
                            if (4 * i + j < left) *yc = (uint16_t)from_f32<F16>(o[i][j]);
                }
            }
            fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_peer(map_peer(smem_u32(&S.acc_empty[buf]), 0));
        }
    }
    __syncwarp();
    fence_before();
    __syncthreads();
    cluster_sync();                     // both CTAs are done with each other's memory
    fence_after();
    if (warp == 2) tmem_dealloc_pair(S.tmem, kPairCols);
}

template <bool F16, bool GLU>
cudaError_t launch_pair(const LinearArgs& a, cudaStream_t s) {
    constexpr int kOut = GLU ? 128 : 256;
    PairArgs p = {};
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
    p.vec = vec4_ok(a.y, a.ldy, 2);
    p.vec8 = a.ldy % 8 == 0 && reinterpret_cast<uintptr_t>(a.y) % 16 == 0;
    p.vec_res = vec4_ok(a.res, a.ldr, a.res_f32 ? 4 : 2);
    p.vec_bias = reinterpret_cast<uintptr_t>(a.bias) % 16 == 0 && (!GLU || a.N % 8 == 0);
    p.ttiles = (a.T + kPairTok - 1) / kPairTok;
    p.ftiles = (a.N + kOut - 1) / kOut;
    p.group = 8;
    if ((int64_t)p.ttiles * p.ftiles > INT32_MAX / 2) return cudaErrorInvalidConfiguration;
    CUtensorMap wm, xm;
    if (!make_map(&wm, F16, a.w, (int64_t)(GLU ? 2 : 1) * a.N, a.K, a.ldw, 128) ||
        !make_map(&xm, F16, a.x, a.T, a.K, a.ldx, 128))
        return cudaErrorInvalidConfiguration;
    cudaError_t err = set_smem_limit(linear_pair_kernel<F16, GLU>, kPairSmem);
    if (err != cudaSuccess) return err;
    const int pairs = p.ttiles * p.ftiles < a.num_ctas / 2 ? p.ttiles * p.ftiles : a.num_ctas / 2;
    return launch_pdl(linear_pair_kernel<F16, GLU>, dim3(2 * pairs), dim3(kPairThreads), kPairSmem, s, p, wm, xm);
}

// ---------------------------------------------------------------- a few tokens
// One to kVecTok tokens: the weights' bytes are all that counts, and the tile kernel's fixed
// steps (tensor memory, two cluster barriers) cost as much as reading them.  Here a warp takes
// four weight rows (two outputs' gate and up rows with SwiGLU) and a part of K, 16 bytes a
// lane and row at a time, in fp32 FMAs; K is cut over the warps of a CTA, whose sums meet in
// shared memory in part order.
constexpr int kVecWarps = 8, kVecRows = 4, kVecTok = 4;

struct VecArgs {
    int T, N, K, act, res_f32;
    int parts;               // K parts: 1, 2, 4 or 8 warps of a CTA share their rows
    int64_t ldx, ldw, ldr, ldy;
    const uint16_t *x, *w, *bias;
    const void* res;
    uint16_t* y;
};

// 16 bytes that are read once (they stay out of L1).  Not through the non-coherent path, which is
// for what nothing writes while the kernel runs: this one may start while an input is written.
__device__ inline uint4 ld_stream(const void* p) {
    uint4 r;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
                 : "l"(p));
    return r;
}
// Eight elements at k of a row of K, zero past its end.
__device__ inline uint4 load8(const uint16_t* row, int k, int K) {
    if (k + 8 <= K) return *reinterpret_cast<const uint4*>(row + k);
    uint32_t u[4] = {0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (k + j < K) u[j >> 1] |= (uint32_t)row[k + j] << (16 * (j & 1));
    return make_uint4(u[0], u[1], u[2], u[3]);
}

template <bool F16, bool GLU, int NT>
__global__ void __launch_bounds__(32 * kVecWarps) linear_vec_kernel(const __grid_constant__ VecArgs p) {
    constexpr int kOut = GLU ? kVecRows / 2 : kVecRows;  // outputs of a warp
    constexpr int U = NT == 1 ? 4 : NT == 2 ? 2 : 1;     // steps whose loads are issued together
    __shared__ float s_sum[kVecWarps][kVecRows][NT];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int groups = kVecWarps / p.parts, grp = warp / p.parts, part = warp - grp * p.parts;
    const int n0 = (blockIdx.x * groups + grp) * kOut;
    const int steps = (p.K + 255) / 256, s0 = part * steps / p.parts, s1 = (part + 1) * steps / p.parts;
    const uint16_t* rows[kVecRows];
#pragma unroll
    for (int r = 0; r < kVecRows; ++r) {
        const int n = n0 + r % kOut;
        rows[r] = p.w + (n < p.N ? n + (int64_t)(r / kOut) * p.N : 0) * p.ldw;
    }
    float acc[kVecRows][NT];
#pragma unroll
    for (int r = 0; r < kVecRows; ++r)
#pragma unroll
        for (int t = 0; t < NT; ++t) acc[r][t] = 0.f;
    griddep_wait();
    griddep_launch_dependents();
    auto add = [&](const uint4(&wv)[kVecRows], const uint4(&xv)[NT]) {
        float xf[NT][8];
#pragma unroll
        for (int t = 0; t < NT; ++t) unpack8<F16>(xv[t], xf[t]);
#pragma unroll
        for (int r = 0; r < kVecRows; ++r) {
            float wf[8];
            unpack8<F16>(wv[r], wf);
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int j = 0; j < 8; ++j) acc[r][t] = fmaf(wf[j], xf[t][j], acc[r][t]);
        }
    };
    // whole blocks of U steps without a condition (rows past the last output read row 0, tokens
    // past the last the first token), so that their loads go out together; then the rest
    const uint16_t* xr[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) xr[t] = p.x + (t < p.T ? t : 0) * p.ldx;
    int s = s0;
    for (; s + U <= s1 && (s + U) * 256 <= p.K; s += U) {
        uint4 wv[U][kVecRows], xv[U][NT];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int k = (s + u) * 256 + lane * 8;
#pragma unroll
            for (int r = 0; r < kVecRows; ++r) wv[u][r] = ld_stream(rows[r] + k);
#pragma unroll
            for (int t = 0; t < NT; ++t) xv[u][t] = *reinterpret_cast<const uint4*>(xr[t] + k);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) add(wv[u], xv[u]);
    }
    for (; s < s1; ++s) {
        const int k = s * 256 + lane * 8;
        uint4 wv[kVecRows], xv[NT];
#pragma unroll
        for (int r = 0; r < kVecRows; ++r) wv[r] = k < p.K ? load8(rows[r], k, p.K) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int t = 0; t < NT; ++t) xv[t] = k < p.K ? load8(xr[t], k, p.K) : make_uint4(0, 0, 0, 0);
        add(wv, xv);
    }
#pragma unroll
    for (int r = 0; r < kVecRows; ++r)
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            float v = acc[r][t];
#pragma unroll
            for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
            if (lane == 0) s_sum[warp][r][t] = v;
        }
    __syncthreads();
    // one output a thread
    const int i = threadIdx.x;
    if (i >= groups * kOut * p.T) return;
    const int t = i / (groups * kOut), o = i - t * groups * kOut, g = o / kOut, r = o - g * kOut;
    const int n = (blockIdx.x * groups + g) * kOut + r;
    if (n >= p.N) return;
    float a = 0.f, b = 0.f;
    for (int q = 0; q < p.parts; ++q) {
        a += s_sum[g * p.parts + q][r][t];
        if (GLU) b += s_sum[g * p.parts + q][kOut + r][t];
    }
    if (p.bias) {
        a += to_f32<F16>(p.bias[n]);
        if (GLU) b += to_f32<F16>(p.bias[p.N + n]);
    }
    float v = GLU ? silu_fast(a) * b : apply_act(p.act, a);
    if (p.res) {
        const int64_t ri = t * p.ldr + n;
        v += p.res_f32 ? static_cast<const float*>(p.res)[ri] : to_f32<F16>(static_cast<const uint16_t*>(p.res)[ri]);
    }
    p.y[t * p.ldy + n] = from_f32<F16>(v);
}

template <bool F16, bool GLU, int NT>
cudaError_t launch_vec(const LinearArgs& a, cudaStream_t s) {
    constexpr int kOut = GLU ? kVecRows / 2 : kVecRows;
    VecArgs p = {a.T, a.N, a.K, a.act, a.res_f32, 1, a.ldx, a.ldw, a.ldr, a.ldy, static_cast<const uint16_t*>(a.x),
                 static_cast<const uint16_t*>(a.w), static_cast<const uint16_t*>(a.bias), a.res,
                 static_cast<uint16_t*>(a.y)};
    // K parts: 16 to 32 warps an SM, each with two steps or more (one token, 2048 -> 7168: 11.0
    // us with 12, 7.9 us with 24, 8.7 us with 48, in a second wave)
    const int64_t warps = (a.N + kOut - 1) / kOut;
    const int steps = (a.K + 255) / 256;
    while (p.parts < kVecWarps && warps * p.parts < (int64_t)16 * a.num_ctas && p.parts * 2 <= steps) p.parts *= 2;
    const int per = kVecWarps / p.parts * kOut;
    return launch_pdl(linear_vec_kernel<F16, GLU, NT>, dim3((unsigned)((a.N + per - 1) / per)), dim3(32 * kVecWarps), 0,
                      s, p);
}
template <bool F16, bool GLU>
cudaError_t launch_vec_n(const LinearArgs& a, cudaStream_t s) {
    return a.T == 1 ? launch_vec<F16, GLU, 1>(a, s) : a.T == 2 ? launch_vec<F16, GLU, 2>(a, s) : launch_vec<F16, GLU, 4>(a, s);
}

}  // namespace

cudaError_t launch_linear(const LinearArgs& a, cudaStream_t s) {
    const bool glu = a.act == MOE_ACT_SWIGLU;
    // The vector kernel saves the tile kernel's fixed steps; its loads come nearer to HBM's rate
    // the fewer tokens share the registers.  Measured (vector against tile kernel, us, weights from
    // HBM): one token 29 MB 7.9 / 8.8, 34 MB 8.3 / 9.2, 59 MB as 7168 -> 4096 12.2 / 12.9, 73 MB
    // 18.1 / 15.1, 88 MB 18.9 / 17.5; four tokens 17 MB 7.7 / 6.9 to 7.5, 34 MB 12.1 / 9.4 (from L2,
    // 2 MB 3.2 / 4.2, 8 MB 4.6 / 5.5).  The limits by bytes are coarse: what costs the vector kernel
    // is CTAs that do not spread evenly over the SMs (59 MB as 5760 -> 5120, whose 320 CTAs leave
    // some SMs three and others two: 16.2 / 12.6; as 4608 -> 6400 13.5 / 12.6).
    const int64_t bytes = (int64_t)2 * a.K * a.N * (glu ? 2 : 1);
    if (bytes <= (a.T == 1 ? (int64_t)64 << 20 : a.T <= kVecTok ? (int64_t)20 << 20 : 0)) {
        if (glu) return a.f16 ? launch_vec_n<true, true>(a, s) : launch_vec_n<false, true>(a, s);
        return a.f16 ? launch_vec_n<true, false>(a, s) : launch_vec_n<false, false>(a, s);
    }
    // A pair's stage takes its MMAs (512 clocks, 545 measured), a wave of pairs some 13000 beside
    // its tiles, the last wave's activation 4000 that the tile kernel's smaller tiles do not see.
    // (2048 -> 4096, tile against pair kernel, us: 130 tokens 8.5 / 14.9, 512 14.2 / 15.5, 768
    // 20.3 / 16.6; 512 -> 4096: 512 tokens 9.3 / 8.3, with silu 9.8 / 10.5.)
    const TilePlan pl = plan_tiles(a);
    const int64_t ptiles = (int64_t)((a.T - 1) / kPairTok + 1) * ((a.N - 1) / (glu ? 128 : 256) + 1);
    const int64_t waves = (ptiles + a.num_ctas / 2 - 1) / (a.num_ctas / 2);
    const double base = a.act == MOE_ACT_NONE ? 13000.0 : 17000.0;
    if (base + (double)waves * ((a.K + kBK - 1) / kBK) * 545.0 < pl.clocks) {
        if (glu) return a.f16 ? launch_pair<true, true>(a, s) : launch_pair<false, true>(a, s);
        return a.f16 ? launch_pair<true, false>(a, s) : launch_pair<false, false>(a, s);
    }
    if (glu) return a.f16 ? launch<true, true>(a, pl, s) : launch<false, true>(a, pl, s);
    return a.f16 ? launch<true, false>(a, pl, s) : launch<false, false>(a, pl, s);
}

}  // namespace moe
