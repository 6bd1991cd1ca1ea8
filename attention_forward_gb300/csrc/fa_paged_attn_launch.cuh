// fa_paged_attn_launch.cuh -- launch of the attention over 16-bit paged caches,
// shared by its translation units (one per kind of cache and type).
#pragma once
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
  {  // the shared-memory opt-in, once per device
    static std::mutex mu;
    static bool done[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    std::lock_guard<std::mutex> lock(mu);
    if (!done[dev]) {
      e = cudaFuncSetAttribute(fa_paged_attn_kernel<S, BF16, kMod>,
                               cudaFuncAttributeMaxDynamicSharedMemorySize, paged_smem_bytes<S>());
      if (e != cudaSuccess) return e;
      done[dev] = true;
    }
  }
  // launched to overlap the end of the kernel before, which it waits for, as the
  // merge overlaps this one's (programmatic dependent launch)
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
  cfg.blockDim = dim3(S::kThreads, 1, 1);
  cfg.dynamicSmemBytes = paged_smem_bytes<S>();
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, fa_paged_attn_kernel<S, BF16, kMod>, q, k, v, p);
  if (e != cudaSuccess || p.whole) return e;
  const long long units = static_cast<long long>(p.B) * p.Hkv * p.n_row_blocks;
  const long long blocks = units * S::kPeers;
  cfg.blockDim = dim3(kPagedMergeThreads, 1, 1);
  cfg.dynamicSmemBytes = 0;
  auto with = [&](auto channels) {
    constexpr int kCh = decltype(channels)::value;
    cfg.gridDim = dim3(static_cast<unsigned>(units), S::kDv / kCh, S::kPeers);
    return cudaLaunchKernelEx(&cfg, fa_paged_merge_kernel<S, BF16, kCh>, p, grid / S::kPeers);
  };
  // (64 channels of 64 rows are four float4 a thread and part, and 168 registers: 128
  // heads, 32 sequences of 8192 keys 108 us, 32 channels 101 us)
  if constexpr (S::kN < 64)
    if (blocks * (S::kDv / 64) >= p.sms) return with(std::integral_constant<int, 64>{});
  if (blocks * (S::kDv / 32) >= p.sms) return with(std::integral_constant<int, 32>{});
  return with(std::integral_constant<int, 8>{});
}

}  // namespace fa
