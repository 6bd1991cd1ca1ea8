// fa_cache_api.cu -- the 4-bit cache's entry points: argument checks, the
// attention's grid and workspace, and the launches.
#include <algorithm>
#include <cmath>
#include <cstdint>

#include "fa_cache.h"
#include "fa_host.h"

namespace {

bool aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

size_t up256(size_t n) { return (n + 255) / 256 * 256; }

struct PageShape {
  int num_pages, page_size, max_pages;
};

bool pages_ok(const PageShape& s) {
  return s.num_pages >= 1 && s.max_pages >= 1 && s.page_size >= 16 && s.page_size <= 1024 &&
         (s.page_size & (s.page_size - 1)) == 0 &&
         static_cast<long long>(s.max_pages) * s.page_size <= (1 << 24);
}

int shift_of(int n) {
  int k = 0;
  while ((1 << k) < n) ++k;
  return k;
}

// The checks common to the three calls: sizes, pointers, then what is not
// supported, as fa_fwd orders them.
fa_status_t check_cache(const void* const (&pool)[4], const int* page_table, int B, int heads,
                        int Hkv, int S, int D, const PageShape& s, int dtype) {
  for (const void* p : pool)
    if (!p || !aligned(p, 16)) return FA_ERR_INVALID_ARG;
  if (!page_table || !aligned(page_table, 4)) return FA_ERR_INVALID_ARG;
  if (B < 1 || Hkv < 1 || heads < 1 || S < 1 || S > (1 << 24) || heads % Hkv != 0)
    return FA_ERR_INVALID_ARG;
  if (static_cast<long long>(B) * heads >= 65536) return FA_ERR_INVALID_ARG;
  if (!pages_ok(s)) return FA_ERR_INVALID_ARG;
  if (D != 64 && D != 128) return FA_ERR_UNSUPPORTED;
  if (dtype != FA_F16 && dtype != FA_BF16) return FA_ERR_UNSUPPORTED;
  return FA_OK;
}

fa::CachePool make_pool(const void* const (&pool)[4]) {
  fa::CachePool c;
  for (int n = 0; n < 2; ++n) {
    c.codes[n] = static_cast<uint8_t*>(const_cast<void*>(pool[2 * n]));
    c.params[n] = static_cast<uint32_t*>(const_cast<void*>(pool[2 * n + 1]));
  }
  return c;
}

fa_status_t copy(bool write, const void* const (&pool)[4], const void* k, const void* v,
                 const int* page_table, const int* start, const int* count, int B, int Hkv, int S,
                 int D, const PageShape& s, int dtype, cudaStream_t stream) {
  fa_status_t st = check_cache(pool, page_table, B, Hkv, Hkv, S, D, s, dtype);
  if (st != FA_OK) return st;
  if (!k || !v || !aligned(k, 16) || !aligned(v, 16) || !aligned(start, 4) || !aligned(count, 4))
    return FA_ERR_INVALID_ARG;
  fa::LaunchEnv env{};
  if ((st = fa::launch_env(stream, &env)) != FA_OK) return st;
  fa::CacheCopyParams p{};
  p.pool = make_pool(pool);
  p.rows[0] = const_cast<void*>(k);
  p.rows[1] = const_cast<void*>(v);
  p.page_table = page_table;
  p.start = start;
  p.count = count;
  p.status = env.status;
  p.B = B;
  p.Hkv = Hkv;
  p.S = S;
  p.num_pages = s.num_pages;
  p.page_shift = shift_of(s.page_size);
  p.max_pages = s.max_pages;
  const cudaError_t e = write ? fa::launch_cache_write(D, dtype == FA_BF16, p, stream)
                              : fa::launch_cache_read(D, dtype == FA_BF16, p, stream);
  return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

// The attention counts chunks of keys in an int, by the table's room: the lengths
// are the device's to read.
bool chunks_ok(int B, int H, int Hkv, int Sq, const PageShape& s) {
  const long long rows = static_cast<long long>(H / Hkv) * Sq;
  const int block = fa::cache_attn_row_block(static_cast<int>(rows));
  const long long chunks = (static_cast<long long>(s.max_pages) * s.page_size +
                            fa::kCacheAttnKeys - 1) / fa::kCacheAttnKeys;
  return static_cast<long long>(B) * Hkv * ((rows + block - 1) / block) * chunks <= fa::kCacheMaxChunks;
}

// The attention's persistent CTAs and the memory for their parts.
struct AttnPlan {
  int row_blocks, grid, whole;
  size_t o_bytes, bytes;
};

AttnPlan plan_attn(int B, int H, int Hkv, int Sq, int D, const PageShape& s, int sm_count) {
  AttnPlan a{};
  const int rows = (H / Hkv) * Sq, block = fa::cache_attn_row_block(rows);
  a.row_blocks = (rows + block - 1) / block;
  a.grid = fa::cache_attn_grid(rows, static_cast<long long>(B) * Hkv * a.row_blocks,
                               s.max_pages * s.page_size, sm_count);
  a.whole = s.max_pages * s.page_size <= fa::kCacheWholeKeys ? 1 : 0;
  if (!a.whole) {
    const size_t n = 2u * static_cast<size_t>(a.grid) * block;
    a.o_bytes = up256(n * D * sizeof(float));
    a.bytes = a.o_bytes + up256(n * sizeof(float));
  }
  return a;
}

}  // namespace

extern "C" {

fa_status_t fa_cache_write(const void* k, const void* v, void* k_codes, void* k_params,
                           void* v_codes, void* v_params, const int* page_table, const int* start,
                           const int* count, int B, int Hkv, int S, int D, int num_pages,
                           int page_size, int max_pages, int dtype, fa_stream_t stream) {
  return copy(true, {k_codes, k_params, v_codes, v_params}, k, v, page_table, start, count, B, Hkv,
              S, D, {num_pages, page_size, max_pages}, dtype, reinterpret_cast<cudaStream_t>(stream));
}

fa_status_t fa_cache_read(const void* k_codes, const void* k_params, const void* v_codes,
                          const void* v_params, const int* page_table, const int* start,
                          const int* count, void* k, void* v, int B, int Hkv, int S, int D,
                          int num_pages, int page_size, int max_pages, int dtype,
                          fa_stream_t stream) {
  return copy(false, {k_codes, k_params, v_codes, v_params}, k, v, page_table, start, count, B,
              Hkv, S, D, {num_pages, page_size, max_pages}, dtype,
              reinterpret_cast<cudaStream_t>(stream));
}

size_t fa_cache_workspace_bytes(int B, int H, int Hkv, int Sq, int D, int page_size,
                                int max_pages) {
  const PageShape s{1, page_size, max_pages};
  if (B < 1 || H < 1 || Hkv < 1 || Sq < 1 || Sq > 256 || H % Hkv != 0 || (D != 64 && D != 128) ||
      static_cast<long long>(B) * H >= 65536 || !pages_ok(s) || !chunks_ok(B, H, Hkv, Sq, s))
    return 0;
  return plan_attn(B, H, Hkv, Sq, D, s, fa::device_sms()).bytes;
}

fa_status_t fa_fwd_cache(const void* q, const void* k_codes, const void* k_params,
                         const void* v_codes, const void* v_params, const int* page_table,
                         const int* length, void* o, float* lse, int B, int H, int Hkv, int Sq,
                         int D, int num_pages, int page_size, int max_pages, float scale,
                         int dtype, float softcap, const float* slopes,
                         void* workspace, size_t workspace_bytes, fa_stream_t stream) {
  const PageShape s{num_pages, page_size, max_pages};
  fa_status_t st = check_cache({k_codes, k_params, v_codes, v_params}, page_table, B, H, Hkv, Sq,
                               D, s, dtype);
  if (st != FA_OK) return st;
  if (!q || !o || !lse || !length || !aligned(q, 16) || !aligned(o, 16) || !aligned(lse, 16) ||
      !aligned(length, 4) || !aligned(slopes, 4))
    return FA_ERR_INVALID_ARG;
  if (Sq > 256 || !chunks_ok(B, H, Hkv, Sq, s)) return FA_ERR_INVALID_ARG;
  if (!(scale > 0.f) || !std::isfinite(scale)) return FA_ERR_INVALID_ARG;
  if (!fa::softcap_ok(softcap)) return FA_ERR_INVALID_ARG;
  cudaStream_t strm = reinterpret_cast<cudaStream_t>(stream);
  fa::LaunchEnv env{};
  if ((st = fa::launch_env(strm, &env)) != FA_OK) return st;
  const AttnPlan plan = plan_attn(B, H, Hkv, Sq, D, s, env.sm_count);
  std::unique_lock<std::mutex> hold;
  if (plan.bytes > 0 && !workspace && !env.captured) {
    if ((st = fa::library_workspace(strm, plan.bytes, &workspace, &hold)) != FA_OK) return st;
    workspace_bytes = plan.bytes;
  }
  if (plan.bytes > 0 && (!workspace || workspace_bytes < plan.bytes || !aligned(workspace, 256)))
    return FA_ERR_WORKSPACE;

  fa::CacheAttnParams p{};
  p.pool = make_pool({k_codes, k_params, v_codes, v_params});
  p.q = q;
  p.o = o;
  p.lse = lse;
  if (plan.bytes > 0) {
    p.part_o = static_cast<float*>(workspace);
    p.part_lse = reinterpret_cast<float*>(static_cast<char*>(workspace) + plan.o_bytes);
  }
  p.page_table = page_table;
  p.length = length;
  p.slopes = slopes;
  p.status = env.status;
  p.B = B;
  p.H = H;
  p.Hkv = Hkv;
  p.Sq = Sq;
  p.rows = (H / Hkv) * Sq;
  p.n_row_blocks = plan.row_blocks;
  p.whole = plan.whole;
  p.sms = env.sm_count;
  p.num_pages = num_pages;
  p.page_shift = shift_of(page_size);
  p.max_pages = max_pages;
  p.scale = scale;
  p.cap = softcap;
  if (softcap > 0.f) {
    p.inv_cap = static_cast<float>(1.0 / softcap);
    p.cap_arg = static_cast<float>(2.8853900817779268 / softcap);
  }
  return fa::launch_cache_attn(D, dtype == FA_BF16, p, plan.grid, strm) == cudaSuccess ? FA_OK
                                                                                       : FA_ERR_CUDA;
}

}  // extern "C"
