// fa_score_launch.cuh -- launch of fa_score_kernel, shared by its translation
// units (one per head dimension and type).
#pragma once
#include <mutex>
#include <type_traits>

#include "fa_score.cuh"

namespace fa {

template <int D, bool BF16, int kCap, bool kBias, bool kDocs, bool kHalves>
cudaError_t score_launch_one(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
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
      e = cudaFuncSetAttribute(fa_score_kernel<D, BF16, kCap, kBias, kDocs, kHalves>,
                               cudaFuncAttributeMaxDynamicSharedMemorySize,
                               ScoreLayout<D>::kSmemBytes);
      if (e != cudaSuccess) return e;
      done[dev] = true;
    }
  }
  // its setup overlaps the end of the kernel before, which it waits for
  // (programmatic dependent launch)
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = ScoreLayout<D>::kSmemBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fa_score_kernel<D, BF16, kCap, kBias, kDocs, kHalves>, q, k, v, o,
                            p);
}

template <int D, bool BF16, int kCap, bool kBias>
cudaError_t score_launch_docs(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                              const CUtensorMap& o, const ScoreParams& p, int grid,
                              cudaStream_t stream) {
  auto with = [&](auto docs) {
    constexpr bool kDocs = decltype(docs)::value;
    return p.halves ? score_launch_one<D, BF16, kCap, kBias, kDocs, true>(q, k, v, o, p, grid, stream)
                    : score_launch_one<D, BF16, kCap, kBias, kDocs, false>(q, k, v, o, p, grid, stream);
  };
  return p.doc_k ? with(std::true_type{}) : with(std::false_type{});
}

template <int D, bool BF16>
cudaError_t score_launch(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                         const CUtensorMap& o, const ScoreParams& p, int grid,
                         cudaStream_t stream) {
  if constexpr (BF16)
    if (p.cap_fixed) return score_launch_docs<D, BF16, kCapFixed, false>(q, k, v, o, p, grid, stream);
  if (p.capped)
    return p.slopes ? score_launch_docs<D, BF16, kCapRunning, true>(q, k, v, o, p, grid, stream)
                    : score_launch_docs<D, BF16, kCapRunning, false>(q, k, v, o, p, grid, stream);
  return p.slopes ? score_launch_docs<D, BF16, kCapNone, true>(q, k, v, o, p, grid, stream)
                  : score_launch_docs<D, BF16, kCapNone, false>(q, k, v, o, p, grid, stream);
}

template <int D, bool BF16, int kCap, bool kBias, bool kDocs, bool kHalves = false>
cudaError_t score_regs_one(int* regs) {
  cudaFuncAttributes a{};
  const cudaError_t e =
      cudaFuncGetAttributes(&a, fa_score_kernel<D, BF16, kCap, kBias, kDocs, kHalves>);
  if (e == cudaSuccess && a.numRegs != 128) *regs = a.numRegs;
  if constexpr (!kHalves)
    return e != cudaSuccess ? e : score_regs_one<D, BF16, kCap, kBias, kDocs, true>(regs);
  return e;
}

// Registers per thread of every form: 128, or one that differs.
template <int D, bool BF16>
cudaError_t score_regs(int* regs) {
  *regs = 128;
  cudaError_t e = cudaSuccess;
  auto look = [&](cudaError_t r) { e = e == cudaSuccess ? r : e; };
  look(score_regs_one<D, BF16, kCapNone, false, false>(regs));
  look(score_regs_one<D, BF16, kCapNone, false, true>(regs));
  look(score_regs_one<D, BF16, kCapNone, true, false>(regs));
  look(score_regs_one<D, BF16, kCapNone, true, true>(regs));
  look(score_regs_one<D, BF16, kCapRunning, false, false>(regs));
  look(score_regs_one<D, BF16, kCapRunning, false, true>(regs));
  look(score_regs_one<D, BF16, kCapRunning, true, false>(regs));
  look(score_regs_one<D, BF16, kCapRunning, true, true>(regs));
  if constexpr (BF16) {
    look(score_regs_one<D, BF16, kCapFixed, false, false>(regs));
    look(score_regs_one<D, BF16, kCapFixed, false, true>(regs));
  }
  return e;
}

}  // namespace fa
