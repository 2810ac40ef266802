// moe_clusters.cuh -- how many clusters of a kernel the current device runs at
// once (host code only).
#pragma once

#include <map>
#include <mutex>
#include <tuple>
#include <cuda_runtime_api.h>

namespace moe {

// Clusters of `ctas` CTAs of `kernel`, at this block size and dynamic shared
// memory, that the current device runs at once (a cluster's CTAs share a
// processing cluster of the GPU: GB300 holds 76, 36 and 15 of 2, 4 and 8 CTAs
// that fill an SM each, not 76, 38 and 19).  Kept per device, kernel and launch
// shape.  0 where it cannot be asked: then nothing is kept, and no error is left
// behind for the caller's next call.
inline int active_clusters(const void* kernel, int threads, int smem, int ctas) {
    static std::mutex mu;
    static std::map<std::tuple<int, const void*, int, int, int>, int> known;
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) {
        cudaGetLastError();
        return 0;
    }
    std::lock_guard<std::mutex> lock(mu);
    const auto key = std::make_tuple(dev, kernel, threads, smem, ctas);
    const auto it = known.find(key);
    if (it != known.end()) return it->second;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = ctas;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) {
        cudaGetLastError();
        return 0;
    }
    return known[key] = n;
}

}  // namespace moe
