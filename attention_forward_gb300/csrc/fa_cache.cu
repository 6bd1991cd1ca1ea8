// fa_cache.cu -- launchers of the 4-bit cache's write and read kernels.
#include "fa_cache.cuh"

namespace fa {
namespace {

// A grid of (token blocks, B * Hkv): fa_cache_* checks that both fit.
template <int D>
dim3 grid_of(const CacheCopyParams& p) {
  constexpr int kTokens = kCacheCopyRows<D> * kCacheCopyTurns;
  return dim3(static_cast<unsigned>((p.S + kTokens - 1) / kTokens),
              static_cast<unsigned>(p.B) * static_cast<unsigned>(p.Hkv));
}

template <int D, bool BF16>
cudaError_t write(const CacheCopyParams& p, cudaStream_t stream) {
  fa_cache_write_kernel<D, BF16><<<grid_of<D>(p), kCacheCopyThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

template <int D, bool BF16>
cudaError_t read(const CacheCopyParams& p, cudaStream_t stream) {
  fa_cache_read_kernel<D, BF16><<<grid_of<D>(p), kCacheCopyThreads, 0, stream>>>(p);
  return cudaGetLastError();
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
