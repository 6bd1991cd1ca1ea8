// fa_paged_api.cu -- entry points of the 16-bit paged caches: argument checks, the
// attention's grid and workspace, and the launches.
#include <algorithm>
#include <cmath>
#include <cstdint>

#include "fa_host.h"
#include "fa_paged.h"

namespace fa {

cudaError_t launch_paged_attn_d64(bool, const CUtensorMap&, const CUtensorMap&, const CUtensorMap&,
                                  const PagedAttnParams&, int, cudaStream_t);
cudaError_t launch_paged_attn_d128(bool, const CUtensorMap&, const CUtensorMap&, const CUtensorMap&,
                                   const PagedAttnParams&, int, cudaStream_t);
cudaError_t launch_paged_attn_latent(bool, const CUtensorMap&, const CUtensorMap&,
                                     const PagedAttnParams&, int, cudaStream_t);

cudaError_t launch_paged_attn(int kind, bool bf16, const CUtensorMap& q, const CUtensorMap& k,
                              const CUtensorMap& v, const PagedAttnParams& p, int grid,
                              cudaStream_t stream) {
  if (kind == kLatent) return launch_paged_attn_latent(bf16, q, k, p, grid, stream);
  return kind == 128 ? launch_paged_attn_d128(bf16, q, k, v, p, grid, stream)
                     : launch_paged_attn_d64(bf16, q, k, v, p, grid, stream);
}

int paged_attn_row_block(int kind, int rows) {
  if (rows <= 16) return 16;
  return kind == kLatent && rows <= 32 ? 32 : 64;
}

int paged_attn_peers(int kind, int rows) { return kind == kLatent && rows > 64 ? 2 : 1; }

// CTAs an SM holds (PagedShape's kCtas).
static int paged_attn_ctas(int kind, int block) {
  if (kind == kLatent) return 1;
  return block == 16 ? 2 : 1;
}

bool paged_attn_whole(int kind, long long units, int room, int sm_count) {
  const int sms = sm_count > 0 ? sm_count : 152;
  int most = kind == kLatent ? 256 : 512;
  if (units >= sms)
    most = 1024;
  else if (5 * units >= 2 * sms)
    most *= 2;
  return room <= most;
}

int paged_attn_grid(int kind, int rows, long long units, int room, int sm_count) {
  const int peers = paged_attn_peers(kind, rows);
  const long long chunks =
      units * ((room + kCacheAttnKeys - 1) / kCacheAttnKeys + paged_segment(peers));
  const long long most = paged_attn_whole(kind, units, room, sm_count)
                             ? units : (chunks + kPagedMinChunks - 1) / kPagedMinChunks;
  const long long slots = static_cast<long long>(sm_count > 0 ? sm_count : 152) *
                          paged_attn_ctas(kind, paged_attn_row_block(kind, rows)) / peers;
  return static_cast<int>(most < slots ? most : slots) * peers;
}

}  // namespace fa

namespace {

bool aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
size_t up256(size_t n) { return (n + 255) / 256 * 256; }

struct PageShape {
  int num_pages, page_size, max_pages;
};

int shift_of(int n) {
  int k = 0;
  while ((1 << k) < n) ++k;
  return k;
}

bool pages_ok(const PageShape& s) {
  return s.num_pages >= 1 && s.max_pages >= 1 && s.page_size >= 16 && s.page_size <= 1024 &&
         (s.page_size & (s.page_size - 1)) == 0 &&
         static_cast<long long>(s.max_pages) * s.page_size <= (1 << 24);
}

// The pool's rows are counted in 31 bits (TMA coordinates).
bool pool_ok(const PageShape& s, int Hkv) {
  return static_cast<long long>(s.num_pages) * Hkv * s.page_size <= 0x7fffffffLL;
}

// The checks common to the calls, as the 4-bit cache's: sizes, pointers, then what
// is not supported.
fa_status_t check(const void* pool0, const void* pool1, const int* page_table, int B, int heads,
                  int Hkv, int S, int D, const PageShape& s, int dtype) {
  if (!pool0 || !pool1 || !page_table) return FA_ERR_INVALID_ARG;
  if (!aligned(pool0, 16) || !aligned(pool1, 16) || !aligned(page_table, 4)) return FA_ERR_INVALID_ARG;
  if (B < 1 || Hkv < 1 || heads < 1 || S < 1 || S > (1 << 24) || heads % Hkv != 0)
    return FA_ERR_INVALID_ARG;
  if (static_cast<long long>(B) * heads >= 65536) return FA_ERR_INVALID_ARG;
  if (!pages_ok(s) || !pool_ok(s, Hkv)) return FA_ERR_INVALID_ARG;
  if (D != 64 && D != 128) return FA_ERR_UNSUPPORTED;
  if (dtype != FA_F16 && dtype != FA_BF16) return FA_ERR_UNSUPPORTED;
  return FA_OK;
}

// Tokens of a block and slices of its heads: 8 tokens (16 latent ones) with all heads
// where they make blocks enough for the GPU, else a head a thread.
fa_status_t write(bool latent, fa::PagedWriteParams& p, int pairs, const PageShape& s, int dtype,
                  cudaStream_t stream) {
  if (!aligned(p.q, 16) || !aligned(p.q_out, 16) || !aligned(p.k, 16) || !aligned(p.v, 16) ||
      !p.k || !p.v || !aligned(p.freqs, 4) || !aligned(p.start, 4) || !aligned(p.count, 4))
    return FA_ERR_INVALID_ARG;
  if ((p.q == nullptr) != (p.q_out == nullptr) || (pairs != 0 && pairs != 1)) return FA_ERR_INVALID_ARG;
  fa::LaunchEnv env{};
  const fa_status_t st = fa::launch_env(stream, &env);
  if (st != FA_OK) return st;
  if (!p.q) p.H = 0;
  p.status = env.status;
  p.num_pages = s.num_pages;
  p.page_shift = shift_of(s.page_size);
  p.max_pages = s.max_pages;
  // (4 x 4096 tokens, us by 4, 8, 16 tokens: 32 + 16 heads of 128 channels 46.2, 38.4,
  // 39.2; latent rows and 16 heads 23.8, 19.3, 15.7, by 32 35.5)
  p.token_shift = std::min(latent ? 4 : 3, shift_of(p.S));
  const long long blocks = ((static_cast<long long>(p.S) + (1 << p.token_shift) - 1) >> p.token_shift) * p.B;
  int slices = 1;
  if (blocks < 4LL * env.sm_count) {
    const int heads = p.H + p.Hkv + (latent ? fa::kLatent / fa::kLatentRope : p.Hkv);
    const int at_once = 256 / ((latent ? 4 : p.D / 16) << p.token_shift);
    slices = (heads + at_once - 1) / at_once;
  }
  const cudaError_t e = fa::launch_paged_write(latent, dtype == FA_BF16, pairs != 0, p, slices, stream);
  return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

fa_status_t read(bool latent, fa::PagedReadParams& p, const PageShape& s, cudaStream_t stream) {
  if (!p.out[0] || !p.out[1] || !aligned(p.out[0], 16) || !aligned(p.out[1], 16) ||
      !aligned(p.start, 4) || !aligned(p.count, 4))
    return FA_ERR_INVALID_ARG;
  fa::LaunchEnv env{};
  const fa_status_t st = fa::launch_env(stream, &env);
  if (st != FA_OK) return st;
  p.status = env.status;
  p.num_pages = s.num_pages;
  p.page_shift = shift_of(s.page_size);
  p.max_pages = s.max_pages;
  return fa::launch_paged_read(latent, p, stream) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

// The attention counts chunks of keys in an int, by the table's room: the lengths
// are the device's to read.
bool chunks_ok(int kind, int B, int H, int Hkv, int Sq, const PageShape& s) {
  const long long rows = static_cast<long long>(H / Hkv) * Sq;
  const int block = fa::paged_attn_row_block(kind, static_cast<int>(rows));
  const long long chunks = (static_cast<long long>(s.max_pages) * s.page_size +
                            fa::kCacheAttnKeys - 1) / fa::kCacheAttnKeys +
                           fa::paged_segment(fa::paged_attn_peers(kind, static_cast<int>(rows)));
  return static_cast<long long>(B) * Hkv * ((rows + block - 1) / block) * chunks <= fa::kCacheMaxChunks;
}

// The attention's persistent CTAs and the memory for their parts.
struct AttnPlan {
  int row_blocks, part_rows, grid, whole;
  size_t o_bytes, bytes;
};

AttnPlan plan_attn(int kind, int B, int H, int Hkv, int Sq, const PageShape& s, int sm_count) {
  AttnPlan a{};
  const int rows = (H / Hkv) * Sq, block = fa::paged_attn_row_block(kind, rows);
  const int room = s.max_pages * s.page_size;
  const int unit_rows = block * fa::paged_attn_peers(kind, rows);
  a.row_blocks = (rows + unit_rows - 1) / unit_rows;
  a.part_rows = std::min(rows, block);
  a.part_rows = a.part_rows > 16   ? (a.part_rows + 31) & ~31
                : a.part_rows > 8 ? 16
                                  : (a.part_rows + 3) & ~3;  // as paged_part_row has them
  const long long units = static_cast<long long>(B) * Hkv * a.row_blocks;
  a.grid = fa::paged_attn_grid(kind, rows, units, room, sm_count);
  a.whole = fa::paged_attn_whole(kind, units, room, sm_count) ? 1 : 0;
  if (!a.whole) {
    const size_t parts = 2u * static_cast<size_t>(a.grid);
    a.o_bytes = up256(parts * a.part_rows * kind * sizeof(float));
    a.bytes = a.o_bytes + up256(parts * block * sizeof(float));
  }
  return a;
}

bool attn_sizes_ok(int B, int H, int Hkv, int Sq) {
  return B >= 1 && H >= 1 && Hkv >= 1 && Sq >= 1 && Sq <= 256 && H % Hkv == 0 &&
         static_cast<long long>(B) * H < 65536;
}

// kind: a head's channels, or kLatent.
fa_status_t attend(int kind, const void* q, const void* k, const void* v, const int* page_table,
                   const int* length, void* o, float* lse, int B, int H, int Hkv, int Sq,
                   const PageShape& s, float scale, int dtype, float softcap, const float* slopes,
                   void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  if (!q || !o || !lse || !length || !aligned(q, 16) || !aligned(o, 16) || !aligned(lse, 16) ||
      !aligned(length, 4) || !aligned(slopes, 4))
    return FA_ERR_INVALID_ARG;
  if (Sq > 256 || !chunks_ok(kind, B, H, Hkv, Sq, s)) return FA_ERR_INVALID_ARG;
  if (!(scale > 0.f) || !std::isfinite(scale)) return FA_ERR_INVALID_ARG;
  if (!fa::softcap_ok(softcap)) return FA_ERR_INVALID_ARG;
  fa::LaunchEnv env{};
  fa_status_t st = fa::launch_env(stream, &env);
  if (st != FA_OK) return st;
  const AttnPlan plan = plan_attn(kind, B, H, Hkv, Sq, s, env.sm_count);
  std::unique_lock<std::mutex> hold;
  if (plan.bytes > 0 && !workspace && !env.captured) {
    if ((st = fa::library_workspace(stream, plan.bytes, &workspace, &hold)) != FA_OK) return st;
    workspace_bytes = plan.bytes;
  }
  if (plan.bytes > 0 && (!workspace || workspace_bytes < plan.bytes || !aligned(workspace, 256)))
    return FA_ERR_WORKSPACE;

  fa::PagedAttnParams p{};
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
  p.timeout_ns = env.timeout_ns;
  p.B = B;
  p.H = H;
  p.Hkv = Hkv;
  p.Sq = Sq;
  p.rows = (H / Hkv) * Sq;
  p.part_rows = plan.part_rows;
  p.n_row_blocks = plan.row_blocks;
  p.sms = env.sm_count;
  p.whole = plan.whole;
  p.num_pages = s.num_pages;
  p.page_shift = shift_of(s.page_size);
  p.max_pages = s.max_pages;
  p.pool_rows = s.num_pages * Hkv * s.page_size;
  p.scale = scale;
  p.cap = softcap;
  if (softcap > 0.f) {
    p.inv_cap = static_cast<float>(1.0 / softcap);
    p.cap_arg = static_cast<float>(2.8853900817779268 / softcap);
  }
  const bool bf16 = dtype == FA_BF16;
  const int k_chunks = kind == fa::kLatent ? fa::kLatentRow / 64 : kind / 64;
  CUtensorMap tq, tk, tv;
  st = fa::encode_rows_of_chunks(&tq, q, static_cast<long long>(B) * H * Sq, k_chunks,
                                 fa::paged_attn_row_block(kind, p.rows), bf16);
  if (st != FA_OK) return st;
  // one descriptor for both pools, two where they lie too far apart
  const bool one = kind == fa::kLatent || k == v;
  const char *kb = static_cast<const char*>(k), *vb = static_cast<const char*>(v);
  st = fa::encode_pools(&tk, std::min(kb, vb), one ? nullptr : std::max(kb, vb), p.pool_rows, k_chunks,
                        bf16);
  tv = tk;
  if (st == FA_OK && !one) {
    p.k_at = kb > vb ? 1 : 0;
    p.v_at = 1 - p.k_at;
  } else if (st == FA_ERR_UNSUPPORTED) {
    if ((st = fa::encode_pools(&tk, k, nullptr, p.pool_rows, k_chunks, bf16)) == FA_OK)
      st = fa::encode_pools(&tv, v, nullptr, p.pool_rows, k_chunks, bf16);
  }
  if (st != FA_OK) return st;
  return fa::launch_paged_attn(kind, bf16, tq, tk, tv, p, plan.grid, stream) == cudaSuccess ? FA_OK
                                                                                            : FA_ERR_CUDA;
}

}  // namespace

extern "C" {

fa_status_t fa_paged_write(const void* q, const void* k, const void* v, void* q_out, void* k_pages,
                           void* v_pages, const int* page_table, const int* start, const int* count,
                           const float* freqs, int rotary, int interleaved, int B, int H, int Hkv,
                           int S, int D, int num_pages, int page_size, int max_pages, int dtype,
                           fa_stream_t stream) {
  const PageShape s{num_pages, page_size, max_pages};
  const fa_status_t st = check(k_pages, v_pages, page_table, B, q ? H : Hkv, Hkv, S, D, s, dtype);
  if (st != FA_OK) return st;
  if (freqs ? (rotary < 16 || rotary > D || rotary % 16 != 0) : rotary != 0) return FA_ERR_INVALID_ARG;
  fa::PagedWriteParams p{};
  p.q = q;
  p.k = k;
  p.v = v;
  p.q_out = q_out;
  p.pool[0] = k_pages;
  p.pool[1] = v_pages;
  p.freqs = freqs;
  p.page_table = page_table;
  p.start = start;
  p.count = count;
  p.B = B;
  p.H = H;
  p.Hkv = Hkv;
  p.S = S;
  p.D = D;
  p.rot = rotary;
  p.q_width = D;
  return write(false, p, interleaved, s, dtype, reinterpret_cast<cudaStream_t>(stream));
}

fa_status_t fa_paged_read(const void* k_pages, const void* v_pages, const int* page_table,
                          const int* start, const int* count, void* k, void* v, int B, int Hkv,
                          int S, int D, int num_pages, int page_size, int max_pages, int dtype,
                          fa_stream_t stream) {
  const PageShape s{num_pages, page_size, max_pages};
  const fa_status_t st = check(k_pages, v_pages, page_table, B, Hkv, Hkv, S, D, s, dtype);
  if (st != FA_OK) return st;
  fa::PagedReadParams p{};
  p.pool[0] = k_pages;
  p.pool[1] = v_pages;
  p.out[0] = k;
  p.out[1] = v;
  p.page_table = page_table;
  p.start = start;
  p.count = count;
  p.B = B;
  p.Hkv = Hkv;
  p.S = S;
  p.D = D;
  return read(false, p, s, reinterpret_cast<cudaStream_t>(stream));
}

size_t fa_paged_workspace_bytes(int B, int H, int Hkv, int Sq, int D, int page_size, int max_pages) {
  const PageShape s{1, page_size, max_pages};
  if (!attn_sizes_ok(B, H, Hkv, Sq) || (D != 64 && D != 128) || !pages_ok(s) ||
      !chunks_ok(D, B, H, Hkv, Sq, s))
    return 0;
  return plan_attn(D, B, H, Hkv, Sq, s, fa::device_sms()).bytes;
}

fa_status_t fa_fwd_paged(const void* q, const void* k_pages, const void* v_pages,
                         const int* page_table, const int* length, void* o, float* lse, int B, int H,
                         int Hkv, int Sq, int D, int num_pages, int page_size, int max_pages,
                         float scale, int dtype, float softcap, const float* slopes, void* workspace,
                         size_t workspace_bytes, fa_stream_t stream) {
  const PageShape s{num_pages, page_size, max_pages};
  const fa_status_t st = check(k_pages, v_pages, page_table, B, H, Hkv, Sq, D, s, dtype);
  if (st != FA_OK) return st;
  return attend(D, q, k_pages, v_pages, page_table, length, o, lse, B, H, Hkv, Sq, s, scale, dtype,
                softcap, slopes, workspace, workspace_bytes, reinterpret_cast<cudaStream_t>(stream));
}

fa_status_t fa_latent_write(const void* c, const void* k_rope, void* pages, const void* q_rope,
                            void* q, const int* page_table, const int* start, const int* count,
                            const float* freqs, int interleaved, int B, int H, int S, int q_width,
                            int num_pages, int page_size, int max_pages, int dtype,
                            fa_stream_t stream) {
  const PageShape s{num_pages, page_size, max_pages};
  const fa_status_t st = check(pages, pages, page_table, B, q_rope ? H : 1, 1, S, 64, s, dtype);
  if (st != FA_OK) return st;
  if (q_rope && (q_width < fa::kLatentRope || q_width % 8 != 0 || q_width > 65536))
    return FA_ERR_INVALID_ARG;
  fa::PagedWriteParams p{};
  p.q = q_rope;
  p.k = k_rope;
  p.v = c;
  p.q_out = q;
  p.pool[0] = pages;
  p.freqs = freqs;
  p.page_table = page_table;
  p.start = start;
  p.count = count;
  p.B = B;
  p.H = H;
  p.Hkv = 1;
  p.S = S;
  p.D = fa::kLatentRope;
  p.rot = freqs ? fa::kLatentRope : 0;
  p.q_width = q_width;
  return write(true, p, interleaved, s, dtype, reinterpret_cast<cudaStream_t>(stream));
}

fa_status_t fa_latent_read(const void* pages, const int* page_table, const int* start,
                           const int* count, void* c, void* k_rope, int B, int S, int num_pages,
                           int page_size, int max_pages, int dtype, fa_stream_t stream) {
  const PageShape s{num_pages, page_size, max_pages};
  const fa_status_t st = check(pages, pages, page_table, B, 1, 1, S, 64, s, dtype);
  if (st != FA_OK) return st;
  fa::PagedReadParams p{};
  p.pool[0] = pages;
  p.out[0] = c;
  p.out[1] = k_rope;
  p.page_table = page_table;
  p.start = start;
  p.count = count;
  p.B = B;
  p.Hkv = 1;
  p.S = S;
  return read(true, p, s, reinterpret_cast<cudaStream_t>(stream));
}

size_t fa_latent_workspace_bytes(int B, int H, int Sq, int page_size, int max_pages) {
  const PageShape s{1, page_size, max_pages};
  if (!attn_sizes_ok(B, H, 1, Sq) || !pages_ok(s) || !chunks_ok(fa::kLatent, B, H, 1, Sq, s)) return 0;
  return plan_attn(fa::kLatent, B, H, 1, Sq, s, fa::device_sms()).bytes;
}

fa_status_t fa_fwd_latent(const void* q, const void* pages, const int* page_table, const int* length,
                          void* o, float* lse, int B, int H, int Sq, int num_pages, int page_size,
                          int max_pages, float scale, int dtype, void* workspace,
                          size_t workspace_bytes, fa_stream_t stream) {
  const PageShape s{num_pages, page_size, max_pages};
  const fa_status_t st = check(pages, pages, page_table, B, H, 1, Sq, 64, s, dtype);
  if (st != FA_OK) return st;
  return attend(fa::kLatent, q, pages, pages, page_table, length, o, lse, B, H, 1, Sq, s, scale,
                dtype, 0.f, nullptr, workspace, workspace_bytes, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
