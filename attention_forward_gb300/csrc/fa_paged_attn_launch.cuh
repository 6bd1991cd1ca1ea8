// fa_paged_attn_launch.cuh -- launch of the attention over 16-bit paged caches,
// shared by its translation units (one per kind of cache and type).
#pragma once
#include <algorithm>
#include <mutex>
#include <type_traits>

#include "fa_paged_attn.cuh"

namespace fa {

template <class S, bool BF16, bool kMod>
cudaError_t paged_launch_one(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                             const PagedAttnParams& p, int grid, cudaStream_t stream) {
  static_assert(paged_smem_bytes<S>() <= 232448 && S::kStages <= PagedMiscBars::kMaxStages,
                "shared memory budget");
  static_assert(S::kCtas * (paged_smem_bytes<S>() + 1024) <= 233472, "CTAs an SM");
  // launched to overlap the end of the kernel before, which it waits for, as the
  // merge overlaps this one's (programmatic dependent launch)
  cudaLaunchConfig_t cfg{};
  cfg.blockDim = dim3(S::kThreads, 1, 1);
  cfg.dynamicSmemBytes = paged_smem_bytes<S>();
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = S::kCluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  {  // once per device: the shared-memory opt-in, and the clusters that it holds
    static std::mutex mu;
    static int clusters[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    std::lock_guard<std::mutex> lock(mu);
    if (clusters[dev] == 0) {
      e = cudaFuncSetAttribute(fa_paged_attn_kernel<S, BF16, kMod>,
                               cudaFuncAttributeMaxDynamicSharedMemorySize, paged_smem_bytes<S>());
      if (e != cudaSuccess) return e;
      int n = 1 << 30;
      if constexpr (S::kCluster > 1) {
        cfg.gridDim = dim3(S::kCluster, 1, 1);
        cfg.attrs = attr + 1;
        cfg.numAttrs = 1;
        e = cudaOccupancyMaxActiveClusters(&n, fa_paged_attn_kernel<S, BF16, kMod>, &cfg);
        if (e != cudaSuccess) return e;
        if (n < 1) return cudaErrorInvalidConfiguration;
        cfg.attrs = attr;
      }
      clusters[dev] = n;
    }
    grid = std::min(grid / S::kCluster, clusters[dev]);  // now the deal's
  }
  cfg.gridDim = dim3(static_cast<unsigned>(grid * S::kCluster), 1, 1);
  cfg.numAttrs = S::kCluster > 1 ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, fa_paged_attn_kernel<S, BF16, kMod>, q, k, v, p);
  if (e != cudaSuccess || p.whole) return e;
  const long long units = static_cast<long long>(p.B) * p.Hkv * p.n_row_blocks;
  const long long blocks = units * S::kCluster;
  cfg.blockDim = dim3(kPagedMergeThreads, 1, 1);
  cfg.dynamicSmemBytes = 0;
  cfg.numAttrs = 1;
  auto with = [&](auto channels) {
    constexpr int kCh = decltype(channels)::value;
    cfg.gridDim = dim3(static_cast<unsigned>(units), S::kDv / kCh, S::kCluster);
    return cudaLaunchKernelEx(&cfg, fa_paged_merge_kernel<S, BF16, kCh>, p, grid);
  };
  // (64 channels of 64 rows are four float4 a thread and part, and 168 registers: 128
  // heads, 32 sequences of 8192 keys 108 us, 32 channels 101 us)
  if constexpr (S::kN < 64)
    if (blocks * (S::kDv / 64) >= p.sms) return with(std::integral_constant<int, 64>{});
  if (blocks * (S::kDv / 32) >= p.sms) return with(std::integral_constant<int, 32>{});
  return with(std::integral_constant<int, 8>{});
}

}  // namespace fa
