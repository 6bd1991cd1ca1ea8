// fa_merge.cu -- the merge of equal key ranges of all rows, one block a row.  It
// starts while the kernel before it still runs (programmatic dependent
// launch).
#include "fa_merge.cuh"
#include "fa_merge.h"

namespace fa {
namespace {

template <int D, bool BF16>
__global__ void __launch_bounds__(kMergeWarps * 32) fa_merge_kernel(const MergeParams p) {
  __shared__ MergeSmem<D> sm;
  const long long row = blockIdx.x;
  grid_dependency_wait();
  merge_row<D, BF16>(p.part_o, p.part_lse, p.n_splits,
                     [&](int s) -> long long { return s * p.rows + row; }, p.o, p.lse, row, sm);
}

template <int D, bool BF16>
cudaError_t launch(const MergeParams& p, cudaStream_t stream) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(p.rows), 1, 1);
  cfg.blockDim = dim3(kMergeWarps * 32, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fa_merge_kernel<D, BF16>, p);
}

}  // namespace

cudaError_t launch_merge(int D, bool bf16, const MergeParams& p, cudaStream_t stream) {
  if (D == 128) return bf16 ? launch<128, true>(p, stream) : launch<128, false>(p, stream);
  return bf16 ? launch<64, true>(p, stream) : launch<64, false>(p, stream);
}

}  // namespace fa
