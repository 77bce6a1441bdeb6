// How many clusters the current device holds at once (its GPCs differ in their SMs, so this is
// less than SMs / cluster size): asked of the runtime once per device, cluster size and CTAs
// per SM, then remembered.
#include <atomic>

#include "kernels.h"

namespace moe {
namespace {

__global__ void capacity_kernel() {}

}  // namespace

int cluster_capacity(int size, int per_sm, int num_ctas) {
    constexpr int kMaxSize = 8, kMaxPerSm = 3;
    static std::atomic<int> cached[64][kMaxSize + 1][kMaxPerSm + 1];
    const int guess = num_ctas * per_sm * 7 / 8 / size;   // where the runtime cannot be asked
    int dev = 0;
    if (size < 1 || size > kMaxSize || per_sm < 1 || per_sm > kMaxPerSm || cudaGetDevice(&dev) != cudaSuccess ||
        dev < 0 || dev >= 64)
        return guess > 0 ? guess : 1;
    int n = cached[dev][size][per_sm].load(std::memory_order_relaxed);
    if (n > 0) return n;
    const int smem = (per_sm == 1 ? 200 : per_sm == 2 ? 100 : 72) * 1024;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(size * num_ctas);
    cfg.blockDim = dim3(256);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = size;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (set_smem_limit(capacity_kernel, kMaxDynSmem) != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&n, capacity_kernel, &cfg) != cudaSuccess || n < 1) {
        cudaGetLastError();
        n = guess > 0 ? guess : 1;
    }
    cached[dev][size][per_sm].store(n, std::memory_order_relaxed);
    return n;
}

}  // namespace moe
