// fa_cache_attn.cu -- launcher of the attention over the 4-bit cache.
#include "fa_cache_attn.cuh"

namespace fa {
namespace {

template <int D, bool BF16, int NT, bool kMod>
cudaError_t launch(const CacheAttnParams& p, int grid, cudaStream_t stream) {
  static_assert(sizeof(CacheAttnSmem<D, NT>) <= 48 * 1024, "no opt-in shared memory");
  // launched to overlap the end of the kernel before, which it waits for, as
  // the merge overlaps this one's (programmatic dependent launch)
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
  cfg.blockDim = dim3(kCacheAttnThreads, 1, 1);
  cfg.dynamicSmemBytes = sizeof(CacheAttnSmem<D, NT>);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, fa_cache_attn_kernel<D, BF16, NT, kMod>, p);
  if (e != cudaSuccess || p.whole) return e;
  const long long units = static_cast<long long>(p.B) * p.Hkv * p.n_row_blocks;
  const bool by_unit = units >= p.sms;
  cfg.gridDim = dim3(static_cast<unsigned>(by_unit ? units : static_cast<long long>(p.B) * p.Hkv * p.rows),
                     1, 1);
  cfg.dynamicSmemBytes = 0;
  return by_unit ? cudaLaunchKernelEx(&cfg, fa_cache_merge_kernel<D, BF16, NT, true>, p, grid)
                 : cudaLaunchKernelEx(&cfg, fa_cache_merge_kernel<D, BF16, NT, false>, p, grid);
}

template <int D, bool BF16>
cudaError_t by_rows(const CacheAttnParams& p, int grid, cudaStream_t stream) {
  const bool mod = p.cap > 0.f || p.slopes;
  if (cache_attn_row_block(p.rows) == 8)
    return mod ? launch<D, BF16, 1, true>(p, grid, stream) : launch<D, BF16, 1, false>(p, grid, stream);
  return mod ? launch<D, BF16, 2, true>(p, grid, stream) : launch<D, BF16, 2, false>(p, grid, stream);
}

}  // namespace

int cache_attn_row_block(int rows) { return rows <= 8 ? 8 : 16; }

int cache_attn_grid(int rows, long long units, int room, int sm_count) {
  const long long chunks = units * ((room + kCacheAttnKeys - 1) / kCacheAttnKeys);
  const long long most = room <= kCacheWholeKeys ? units
                                                 : (chunks + kCacheMinChunks - 1) / kCacheMinChunks;
  const long long slots = static_cast<long long>(sm_count > 0 ? sm_count : 152) *
                          cache_attn_occupancy(cache_attn_row_block(rows));
  return static_cast<int>(most < slots ? most : slots);
}

cudaError_t launch_cache_attn(int D, bool bf16, const CacheAttnParams& p, int grid,
                              cudaStream_t stream) {
  if (D == 128) return bf16 ? by_rows<128, true>(p, grid, stream) : by_rows<128, false>(p, grid, stream);
  return bf16 ? by_rows<64, true>(p, grid, stream) : by_rows<64, false>(p, grid, stream);
}

}  // namespace fa
