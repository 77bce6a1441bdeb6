// tcgen05, tensor-map and cluster wrappers of the kernels whose operands are plain 16-bit
// matrices (linear.cu, scored_logits.cu): both operands from shared memory, K-major rows of
// 64 elements in the 128-byte swizzle.
#pragma once
#include <cuda.h>
#include <cudaTypedefs.h>

#include "kernels.h"

namespace moe {
namespace tc5 {

constexpr int kBK = 64;                          // K elements per stage: one 128-byte swizzled row
constexpr long long kWaitLimit = 4000000000LL;   // clock cycles (about 2 s) of any one wait

// One CTA allocates `ncols` (a power of two from 32) tensor-memory columns.  The kernels here
// allocate only after griddep_wait(), so that a kernel launched early never holds columns
// that one still running before it needs.
__device__ inline void tmem_alloc(uint32_t* dst_smem, uint32_t ncols) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst_smem)),
                 "r"(ncols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ inline void tmem_dealloc(uint32_t taddr, uint32_t ncols) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
__device__ inline void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ inline void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// Shared-memory matrix descriptor of a K-major tile in the 128-byte swizzle (8-row groups
// 1024 bytes apart); 16 K elements further on is + 2.
__device__ inline uint64_t smem_desc(uint32_t saddr) {
    return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)1 << 16) | ((uint64_t)(1024 >> 4) << 32) |
           ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

// kind::f16 instruction descriptor: A and B both bf16 or both fp16 (K-major), fp32 D, M x N.
__host__ __device__ constexpr uint32_t instr_desc(bool f16, int m, int n) {
    return (1u << 4) | (f16 ? 0u : (1u << 7) | (1u << 10)) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

// D[M][N] (+)= A[M][16] B[N][16]^T
__device__ inline void umma_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(acc)
        : "memory");
}

// Arrives on `bar` when every MMA issued so far by this thread has completed.
__device__ inline void umma_commit(uint64_t* bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
                 : "memory");
}

// 16 consecutive 32-bit columns of each thread's own lane; not there before ld_wait(r).
__device__ inline void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}
// Waits for all of the thread's tensor-memory loads; the values pass through it, so that no
// use of them can be moved ahead of the wait.
__device__ inline void ld_wait(uint32_t (&r)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
                 :
                 : "memory");
}
__device__ inline void ld_wait(uint32_t (&r)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                   "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]),
                   "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
                   "+r"(r[30]), "+r"(r[31])
                 :
                 : "memory");
}

// One box of a 2-D tensor map into shared memory; x in elements (a multiple of 64 here, so
// every copy starts on 128 bytes), y in rows; rows and columns past the matrix read as zero.
__device__ inline void tma_load_2d(void* dst, const CUtensorMap* map, int x, int y, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], "
        "[%4];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(smem_u32(bar))
        : "memory");
}
__device__ inline void prefetch_map(const CUtensorMap* map) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}

// ---- CTA pairs (cta_group::2): one MMA over two SMs, D of 256 rows, 128 in each CTA; each
// CTA holds its 128 rows of A and half of B's rows; the leader (rank 0) issues -------------
__device__ inline void tmem_alloc_pair(uint32_t* dst_smem, uint32_t ncols) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst_smem)),
                 "r"(ncols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ inline void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols) {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
__device__ inline void umma_ss_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(acc)
        : "memory");
}
// Arrives on the barrier at this shared-memory offset in both CTAs of the pair (ctas: their
// bits among the cluster's ranks).
__device__ inline void umma_commit_pair(uint64_t* bar, uint16_t ctas = 3) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_u32(bar)),
        "h"(ctas)
        : "memory");
}
// A box into this CTA's shared memory whose bytes count on a barrier of either CTA of the
// pair (a shared::cluster address).
__device__ inline void tma_load_2d_pair(void* dst, const CUtensorMap* map, int x, int y, uint32_t bar_cluster) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], "
        "[%1, {%2, %3}], [%4];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar_cluster)
        : "memory");
}

// 32 consecutive columns of each thread's own lane; not there before ld_wait(r).
__device__ inline void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
        "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
}

// Generic writes to shared memory become visible to the MMAs that follow a barrier.
__device__ inline void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// ---- clusters (the CTAs that share one tile's K axis) ---------------------------------
__device__ inline uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ inline void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ inline void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ inline void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ inline uint32_t map_peer(uint32_t saddr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(saddr), "r"(rank));
    return r;
}
// Arrives on a barrier of any CTA of the cluster (its shared::cluster address).
__device__ inline void mbar_arrive_peer(uint32_t bar_cluster) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar_cluster) : "memory");
}
__device__ inline void st_peer_u32(uint32_t addr, uint32_t v) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ inline float4 ld_peer_v4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

// The line of p into L2.
__device__ inline void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// ---- waits ---------------------------------------------------------------------------------
__device__ inline int ld_volatile(const int& v) { return *reinterpret_cast<const volatile int*>(&v); }
__device__ inline void st_volatile(int& v, int x) { *reinterpret_cast<volatile int*>(&v) = x; }

// Bounded wait of one CTA's thread: when it runs out, or another thread's has, the flag is up
// and false is returned.
__device__ inline bool wait_or_flag(int& abort_flag, uint64_t* bar, uint32_t parity, Ctrl* ctrl, uint32_t detail) {
    if (ld_volatile(abort_flag)) return false;
    if (mbar_wait_bounded(bar, parity, kWaitLimit)) return true;
    st_volatile(abort_flag, 1);
    report_error(ctrl, MOE_ERR_TIMEOUT, detail);
    return false;
}
// The same for a thread of a CTA pair, which gives up at once when either CTA has.
__device__ inline void pair_abort(int& abort_flag) {
    st_volatile(abort_flag, 1);
    st_peer_u32(map_peer(smem_u32(&abort_flag), cluster_rank() ^ 1), 1);
}
__device__ inline bool pair_wait(int& abort_flag, uint64_t* bar, uint32_t parity, Ctrl* ctrl, uint32_t detail) {
    if (mbar_try_wait(bar, parity)) return true;
    const long long t0 = clock64();
    while (!ld_volatile(abort_flag)) {
#pragma unroll 1
        for (int i = 0; i < 64; ++i)
            if (mbar_try_wait(bar, parity)) return true;
        if (clock64() - t0 > kWaitLimit) {
            pair_abort(abort_flag);
            report_error(ctrl, MOE_ERR_TIMEOUT, detail);
        }
    }
    return false;
}
// Before a pair's producer leaves after an abort (one thread of each CTA): no copy may still
// target shared memory.  The leader, on whose barriers the bytes of both CTAs count, waits
// (bounded) for the last phase issued on every slot; the other CTA, which may have issued past
// the leader, gives its last copies (microseconds) some half a millisecond.
__device__ inline void pair_drain(uint64_t* full, int stages, int issued, bool leader, Ctrl* ctrl, uint32_t detail) {
    if (leader) {
        for (int d = 0; d < stages && d < issued; ++d) {
            const int i = issued - 1 - d;
            if (!mbar_wait_bounded(&full[i % stages], (uint32_t)(i / stages) & 1, kWaitLimit)) {
                report_error(ctrl, MOE_ERR_TIMEOUT, detail);
                return;
            }
        }
    } else {
        const long long c0 = clock64();
        while (clock64() - c0 < 1000000) __nanosleep(1000);
    }
}
// Failure-path tests (moe_workspace_set_test_stall): a warp's bounded wait on a barrier that
// nothing completes; true when it ran out.
__device__ inline bool test_stall(uint64_t* bar, uint32_t cycles, int lane) {
    bool got = true;
    if (lane == 0) got = mbar_wait_bounded(bar, 0, cycles);
    got = __shfl_sync(0xffffffffu, got, 0);
    __syncwarp();
    return !got;
}

// Shared memory a CTA with `cols` tensor-memory columns must take at least: its share of the
// SM's 228 KB is then no smaller than its share of the 512 columns, so whichever CTAs of
// these kernels share an SM, their allocations fit.  An allocation that had to wait could
// wait for good: CTAs of two clusters could each hold the columns that a partner of the
// other needs.
__host__ inline size_t tmem_smem(uint32_t cols) { return (size_t)cols * (228 * 1024 / 512); }

// ---- host ------------------------------------------------------------------------------
inline PFN_cuTensorMapEncodeTiled_v12000 encoder() {
    static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        cudaDriverEntryPointQueryResult q;
        void* f = nullptr;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            f = nullptr;
        return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
    }();
    return fn;
}

// rows x cols of 16-bit elements, row stride ld elements (a multiple of 8), boxes of
// box_rows x 64 elements.
inline bool make_map(CUtensorMap* m, bool f16, const void* base, int64_t rows, int64_t cols, int64_t ld,
                     int box_rows) {
    const auto enc = encoder();
    if (!enc) return false;
    cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)ld * 2};
    cuuint32_t box[2] = {(cuuint32_t)kBK, (cuuint32_t)box_rows};
    cuuint32_t es[2] = {1, 1};
    return enc(m, f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
               const_cast<void*>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The same for fp32, boxes of box_rows x 64 elements, rows one after the other.
inline bool make_map_f32(CUtensorMap* m, const void* base, int64_t rows, int64_t cols, int64_t ld, int box_rows) {
    const auto enc = encoder();
    if (!enc) return false;
    cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)ld * 4};
    cuuint32_t box[2] = {64, (cuuint32_t)box_rows};
    cuuint32_t es[2] = {1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, const_cast<void*>(base), dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace tc5
}  // namespace moe
