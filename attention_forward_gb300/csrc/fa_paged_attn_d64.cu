// fa_paged_attn_d64.cu -- the attention over 16-bit paged caches: heads of 64 channels.
#include "fa_paged_attn_launch.cuh"

namespace fa {

cudaError_t launch_paged_attn_d64(bool bf16, const CUtensorMap& q, const CUtensorMap& k,
                                  const CUtensorMap& v, const PagedAttnParams& p, int grid,
                                  cudaStream_t stream) {
  auto with = [&](auto shape) {
    using S = decltype(shape);
    if (p.cap > 0.f || p.slopes)
      return bf16 ? paged_launch_one<S, true, true>(q, k, v, p, grid, stream)
                  : paged_launch_one<S, false, true>(q, k, v, p, grid, stream);
    return bf16 ? paged_launch_one<S, true, false>(q, k, v, p, grid, stream)
                : paged_launch_one<S, false, false>(q, k, v, p, grid, stream);
  };
  if (paged_attn_row_block(64, p.rows) == 16) return with(PagedShape<1, 1, false, 16, 6, 2>{});
  return with(PagedShape<1, 1, false, 64, 8, 1>{});
}

}  // namespace fa
