// The tiled packed-weight products for bf16 rows (one translation unit a type, so that they
// compile side by side).
#include "matmul_tc.cuh"

namespace gptq {
gptq_status matmul_tc_bf16(const CUtensorMap &map, const CUtensorMap &wmap, const MmTcArg &p, int dir, int bits, bool pair, int blocks,
                         size_t smem, cudaStream_t st) {
    return dir == 0 ? launch_tc_bits<__nv_bfloat16, 0>(map, wmap, p, bits, pair, blocks, smem, st)
                    : launch_tc_bits<__nv_bfloat16, 1>(map, wmap, p, bits, pair, blocks, smem, st);
}

// Clusters of `cluster` blocks that fit the current device at once (0: the question failed).
int matmul_tc_occupancy(int cluster) {
    constexpr int smem = 200 * 1024;
    auto kernel = k_matmul_tc<__nv_bfloat16, 4, 0, false, false>;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(cluster);
    cfg.blockDim = dim3(MM_THREADS);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = cluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaFuncSetAttribute(reinterpret_cast<const void *>(kernel), cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)SMEM_MOST) != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) {
        cudaGetLastError();
        return 0;
    }
    return n;
}
}  // namespace gptq
