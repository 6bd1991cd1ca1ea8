// fa_cache.cu -- launchers of the 4-bit cache's write and read kernels.
#include "fa_cache.cuh"

namespace fa {
namespace {

// A grid of (token blocks, B * Hkv): fa_cache_* checks that both fit.
dim3 grid_of(const CacheCopyParams& p, int tokens) {
  return dim3(static_cast<unsigned>((p.S + tokens - 1) / tokens),
              static_cast<unsigned>(p.B) * static_cast<unsigned>(p.Hkv));
}

// Launched to overlap the end of the kernel before, which the kernels wait for
// (programmatic dependent launch).
template <class Kernel>
cudaError_t launch(Kernel kernel, const CacheCopyParams& p, int tokens, cudaStream_t stream) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid_of(p, tokens);
  cfg.blockDim = dim3(kCacheCopyThreads, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <int D, bool BF16>
cudaError_t write(const CacheCopyParams& p, cudaStream_t stream) {
  return launch(fa_cache_write_kernel<D, BF16>, p, kCacheWriteRows<D> * kCacheWriteTurns, stream);
}

template <int D, bool BF16>
cudaError_t read(const CacheCopyParams& p, cudaStream_t stream) {
  return launch(fa_cache_read_kernel<D, BF16>, p, kCacheReadRows<D> * kCacheReadTurns, stream);
}

}  // namespace

cudaError_t launch_cache_write(int D, bool bf16, const CacheCopyParams& p, cudaStream_t stream) {
  if (D == 128) return bf16 ? write<128, true>(p, stream) : write<128, false>(p, stream);
  return bf16 ? write<64, true>(p, stream) : write<64, false>(p, stream);
}

cudaError_t launch_cache_read(int D, bool bf16, const CacheCopyParams& p, cudaStream_t stream) {
  if (D == 128) return bf16 ? read<128, true>(p, stream) : read<128, false>(p, stream);
  return bf16 ? read<64, true>(p, stream) : read<64, false>(p, stream);
}

}  // namespace fa
