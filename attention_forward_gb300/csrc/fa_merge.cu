// fa_merge.cu -- the merge of equal key ranges of all rows.  It starts while the
// kernel before it still runs (programmatic dependent launch).
#include "fa_merge.cuh"
#include "fa_merge.h"

namespace fa {
namespace {

// Parts up to which a row is one warp's: their loads go out at once.
constexpr int kWarpParts = 8;

template <int D, bool BF16, bool kByWarp>
__global__ void __launch_bounds__(kMergeWarps * 32) fa_merge_kernel(const MergeParams p) {
  grid_dependency_wait();
  if constexpr (kByWarp) {
    const long long row = static_cast<long long>(blockIdx.x) * kMergeWarps + (threadIdx.x >> 5);
    if (row >= p.rows) return;
    merge_row_warp<D, BF16>(p.part_o, p.part_lse, p.n_splits,
                            [&](int s) -> long long { return s * p.rows + row; }, p.o, p.lse, row);
  } else {
    __shared__ MergeSmem<D> sm;
    const long long row = blockIdx.x;
    merge_row<D, BF16>(p.part_o, p.part_lse, p.n_splits,
                       [&](int s) -> long long { return s * p.rows + row; }, p.o, p.lse, row, sm);
  }
}

template <int D, bool BF16>
cudaError_t launch(const MergeParams& p, cudaStream_t stream) {
  const bool by_warp = p.n_splits <= kWarpParts;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(by_warp ? (p.rows + kMergeWarps - 1) / kMergeWarps : p.rows),
                     1, 1);
  cfg.blockDim = dim3(kMergeWarps * 32, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return by_warp ? cudaLaunchKernelEx(&cfg, fa_merge_kernel<D, BF16, true>, p)
                 : cudaLaunchKernelEx(&cfg, fa_merge_kernel<D, BF16, false>, p);
}

}  // namespace

cudaError_t launch_merge(int D, bool bf16, const MergeParams& p, cudaStream_t stream) {
  if (D == 128) return bf16 ? launch<128, true>(p, stream) : launch<128, false>(p, stream);
  return bf16 ? launch<64, true>(p, stream) : launch<64, false>(p, stream);
}

}  // namespace fa
