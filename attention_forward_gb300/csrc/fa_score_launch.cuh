// fa_score_launch.cuh -- launch of fa_score_kernel, shared by its translation
// units (one per head dimension).
#pragma once
#include <mutex>

#include "fa_score.cuh"

namespace fa {

template <int D, bool BF16>
cudaError_t score_launch(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                         const CUtensorMap& o, const ScoreParams& p, int grid,
                         cudaStream_t stream) {
  {  // the shared-memory opt-in, once per device
    static std::mutex mu;
    static bool done[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    std::lock_guard<std::mutex> lock(mu);
    if (!done[dev]) {
      e = cudaFuncSetAttribute(fa_score_kernel<D, BF16>,
                               cudaFuncAttributeMaxDynamicSharedMemorySize,
                               PrefillLayout<D>::kSmemBytes);
      if (e != cudaSuccess) return e;
      done[dev] = true;
    }
  }
  fa_score_kernel<D, BF16><<<grid, kThreads, PrefillLayout<D>::kSmemBytes, stream>>>(q, k, v, o, p);
  return cudaGetLastError();
}

template <int D, bool BF16>
cudaError_t score_regs(int* regs) {
  cudaFuncAttributes a{};
  const cudaError_t e = cudaFuncGetAttributes(&a, fa_score_kernel<D, BF16>);
  if (e == cudaSuccess) *regs = a.numRegs;
  return e;
}

}  // namespace fa
