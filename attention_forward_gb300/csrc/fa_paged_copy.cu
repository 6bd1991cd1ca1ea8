// fa_paged_copy.cu -- launchers of the 16-bit paged caches' write and read.
#include "fa_paged_copy.cuh"

namespace fa {
namespace {

// Launched to overlap the end of the kernel before, which the kernels wait for
// (programmatic dependent launch).
template <class Kernel, class P>
cudaError_t launch(Kernel kernel, const P& p, dim3 grid, cudaStream_t stream) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kPagedCopyThreads, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace

cudaError_t launch_paged_write(bool latent, bool bf16, bool pairs, const PagedWriteParams& p,
                               int slices, cudaStream_t stream) {
  const dim3 grid(static_cast<unsigned>((p.S + (1 << p.token_shift) - 1) >> p.token_shift),
                  static_cast<unsigned>(p.B), static_cast<unsigned>(slices));
  auto with = [&](auto kernel) { return launch(kernel, p, grid, stream); };
  if (latent)
    return bf16 ? (pairs ? with(fa_paged_write_kernel<true, true, true>)
                         : with(fa_paged_write_kernel<true, true, false>))
                : (pairs ? with(fa_paged_write_kernel<true, false, true>)
                         : with(fa_paged_write_kernel<true, false, false>));
  return bf16 ? (pairs ? with(fa_paged_write_kernel<false, true, true>)
                       : with(fa_paged_write_kernel<false, true, false>))
              : (pairs ? with(fa_paged_write_kernel<false, false, true>)
                       : with(fa_paged_write_kernel<false, false, false>));
}

cudaError_t launch_paged_read(bool latent, const PagedReadParams& p, cudaStream_t stream) {
  const int words = latent ? kLatentRow / 8 : p.D / 8;
  const int rows = kPagedCopyThreads / words * kPagedAtOnce;
  const dim3 grid(static_cast<unsigned>((p.S + rows - 1) / rows),
                  static_cast<unsigned>(p.B) * static_cast<unsigned>(p.Hkv), latent ? 1u : 2u);
  return latent ? launch(fa_paged_read_kernel<true>, p, grid, stream)
                : launch(fa_paged_read_kernel<false>, p, grid, stream);
}

}  // namespace fa
