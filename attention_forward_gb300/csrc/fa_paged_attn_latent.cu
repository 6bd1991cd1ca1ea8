// fa_paged_attn_latent.cu -- the attention over 16-bit paged caches: latent rows.
#include "fa_paged_attn_launch.cuh"

namespace fa {

cudaError_t launch_paged_attn_latent(bool bf16, const CUtensorMap& q, const CUtensorMap& k,
                                     const PagedAttnParams& p, int grid, cudaStream_t stream) {
  auto with = [&](auto shape) {
    using S = decltype(shape);
    return bf16 ? paged_launch_one<S, true, false>(q, k, k, p, grid, stream)
                : paged_launch_one<S, false, false>(q, k, k, p, grid, stream);
  };
  switch (paged_attn_row_block(kLatent, p.rows)) {
    case 16: return with(PagedShape<9, 8, true, 16, 2, 1>{});
    case 32: return with(PagedShape<9, 8, true, 32, 2, 1>{});
    default:
      return paged_attn_peers(kLatent, p.rows) == 2 ? with(PagedShape<9, 8, true, 64, 2, 1, 1, 2>{})
                                                      : with(PagedShape<9, 8, true, 64, 2, 1, 1>{});
  }
}

}  // namespace fa
