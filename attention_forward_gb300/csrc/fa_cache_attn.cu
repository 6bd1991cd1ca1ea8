// fa_cache_attn.cu -- launcher of the attention over the 4-bit cache.
#include "fa_cache_attn.cuh"
#include "fa_merge.h"

namespace fa {
namespace {

template <int D, bool BF16, int NT>
cudaError_t launch(const CacheAttnParams& p, cudaStream_t stream) {
  static_assert(sizeof(CacheAttnSmem<D, NT>) <= 48 * 1024, "no opt-in shared memory");
  const unsigned grid = static_cast<unsigned>(p.n_splits) * static_cast<unsigned>(p.n_row_blocks) *
                        static_cast<unsigned>(p.B * p.Hkv);
  fa_cache_attn_kernel<D, BF16, NT><<<grid, kCacheAttnWarps * 32, sizeof(CacheAttnSmem<D, NT>),
                                      stream>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || p.n_splits == 1) return e;
  const MergeParams m{p.part_o, p.part_lse, p.o, p.lse,
                      static_cast<long long>(p.B) * p.H * p.Sq, p.n_splits};
  return launch_merge(D, BF16, m, stream);
}

template <int D, bool BF16>
cudaError_t by_rows(const CacheAttnParams& p, cudaStream_t stream) {
  return cache_attn_row_block(p.rows) == 8 ? launch<D, BF16, 1>(p, stream)
                                           : launch<D, BF16, 2>(p, stream);
}

}  // namespace

int cache_attn_row_block(int rows) { return rows <= 8 ? 8 : 16; }

cudaError_t launch_cache_attn(int D, bool bf16, const CacheAttnParams& p, cudaStream_t stream) {
  if (D == 128) return bf16 ? by_rows<128, true>(p, stream) : by_rows<128, false>(p, stream);
  return bf16 ? by_rows<64, true>(p, stream) : by_rows<64, false>(p, stream);
}

}  // namespace fa
