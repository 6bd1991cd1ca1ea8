// fa_cache.h -- parameter blocks, limits and launch entry points of the 4-bit
// key/value cache (internal).
#pragma once
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

namespace fa {

// Channels that share one scale and minimum.
constexpr int kCacheGroup = 32;
// Values beyond this magnitude are held as it: 15 scales above the smallest
// minimum stay within fp16.
constexpr float kCacheLimit = 61440.f;
// FA_ERR_INVALID_ARG, from a kernel.  Recorded by a maximum: a timeout (5) that
// another kernel left in the status word is the worse news and stays.
constexpr unsigned kStatusBadIndex = 1;

// The four arrays of a cache: rows of (page, kv head, slot).
struct CachePool {
  uint8_t* codes[2];    // K, V: [num_pages, Hkv, page_size, D / 2]
  uint32_t* params[2];  // K, V: [num_pages, Hkv, page_size, D / 32] (scale, minimum) fp16 pairs
};

struct CacheCopyParams {
  CachePool pool;
  void* rows[2];          // K, V: [B, Hkv, S, D] 16-bit
  const int* page_table;  // [B, max_pages]
  const int* start;       // [B] or null (0)
  const int* count;       // [B] or null (S)
  unsigned* status;
  int B, Hkv, S, num_pages, page_shift, max_pages;
};

struct CacheAttnParams {
  CachePool pool;
  const void* q;          // [B, H, Sq, D]
  void* o;
  float* lse;             // [B, H, Sq]
  float* part_o;          // [2 * grid, row block, D] fp32, O / l of a segment
  float* part_lse;        // [2 * grid, row block]
  const int* page_table;
  const int* length;      // [B]
  const float* slopes;    // [H] or null
  unsigned* status;
  int B, H, Hkv, Sq;
  int rows;               // (H / Hkv) * Sq query rows per kv head
  int n_row_blocks;
  int sms;                // multiprocessors
  int whole;              // CTAs take whole units: no parts, no merge
  int num_pages, page_shift, max_pages;
  float scale;
  float cap;              // cap > 0: score = cap * tanh(score / cap)
  float inv_cap, cap_arg; // 1 / cap, 2 log2(e) / cap
};

cudaError_t launch_cache_write(int D, bool bf16, const CacheCopyParams& p, cudaStream_t stream);
cudaError_t launch_cache_read(int D, bool bf16, const CacheCopyParams& p, cudaStream_t stream);

// Query rows that one pass of the cache attention over the keys takes: 8, or 16
// where a kv head has more than 8.
int cache_attn_row_block(int rows);
constexpr int kCacheAttnWarps = 4;
constexpr int kCacheAttnKeys = 16 * kCacheAttnWarps;  // a chunk of the work: a tile for each warp
constexpr int kCacheAttnStages = 3;                   // tiles of a warp's ring
constexpr long long kCacheMaxChunks = 0x7fffff00;     // of a call: an int's, and room to round up
constexpr int kCachePiece = 4096;  // keys whose tiles' places are in shared memory at once
// CTAs an SM holds: the registers of 16 accumulated rows are more.
constexpr int cache_attn_occupancy(int row_block) { return row_block == 8 ? 4 : 3; }
// A CTA's least share: more parts take longer to merge than they save (one
// sequence of 2048 keys, 8 kv heads: 7.4 us by 4 chunks, 9.0 by 8, 12.8 by 12; of
// 32768: 18.6, 17.3, 18.7).
constexpr int kCacheMinChunks = 4;
// Page tables of at most this many keys are not split, which saves the merge's
// launch.  On the GPU, units of 4 rows, us, whole and split: 512 keys 7.0 and 7.1
// (1 unit), 7.2 and 8.1 (64), 8.9 and 11.7 (256); 1000 keys 10.6 and 7.0 (1), 10.3
// and 7.5 (8), 10.7 and 9.2 (64), 10.9 and 12.0 (128), 13.6 and 17.3 (256); 4 x 16
// heads of 701 keys 10.0 and 10.3; 2048 keys, 8 units, 17.2 and 7.4.  So few units of
// more than 512 keys lose up to 3.5 us in a graph; called from the host, one launch
// less pays for it (8 units of 1000 keys: 17.3 us a call whole, 19.7 split).
constexpr int kCacheWholeKeys = 1024;
// CTAs for `units` row blocks of up to `room` keys.
int cache_attn_grid(int rows, long long units, int room, int sm_count);
cudaError_t launch_cache_attn(int D, bool bf16, const CacheAttnParams& p, int grid,
                              cudaStream_t stream);

}  // namespace fa
