// swa_q8_decode_128.cu - the kernels of swa_q8_decode.cuh for d = 128 (a file to a head
// dimension, so that they compile side by side).
#include "swa_q8_decode.cuh"

#include <atomic>

namespace swa {
cudaError_t launch_q8_decode_128(const Q8DecodeParams& p, const Q8DecodeMaps& maps, cudaStream_t stream) {
  return launch_d<128>(p, maps, stream);
}

int q8_clusters_at_once(int size) {
  static std::atomic<int> known[kMaxDevices][kQ8MaxCluster + 1];   // one more than the number
  int dev = 0;
  if (size < 1 || size > kQ8MaxCluster || cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return 0;
  int n = known[dev][size].load(std::memory_order_relaxed);
  if (n == 0) {
    // of the kernel that has an SM to itself by its shared memory; those of smaller heads, of which an SM holds two,
    // are counted by the same number
    constexpr Q8Variant v = kQ8Variants[0];
    constexpr int smem = q8_smem_bytes<128, 1, v.warps, v.tiles>(true);
    auto kern = swa_q8_decode_kernel<128, 1, v.warps, v.tiles, v.per_sm, SWA_Q8_E4M3, false>;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)size;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)size);
    cfg.blockDim = dim3(v.warps * 32);
    cfg.dynamicSmemBytes = smem;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int found = 0;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&found, kern, &cfg) != cudaSuccess) {
      (void)cudaGetLastError();
      found = 0;
    }
    known[dev][size].store(n = found + 1, std::memory_order_relaxed);
  }
  return n - 1;
}
}  // namespace swa
