// fa_paged.h -- parameter blocks and launch entry points of the 16-bit paged
// caches: keys and values, and latent rows (internal).
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstddef>

#include "fa_cache.h"

namespace fa {

// A latent row: the latent vector, which is the value too, then the rotated part
// of the key.
constexpr int kLatent = 512, kLatentRope = 64, kLatentRow = kLatent + kLatentRope;
// Latent attention's heads where they are expanded: keys of kNope channels of
// their own and the shared rotated ones, values of kNope.
constexpr int kNope = 128;

// A write: new rows into the pages, rotated to their positions.  Keys and values:
// k and v [B, Hkv, S, D] go to the two pools, q [B, H, S, D] to q_out.  Latent: v
// [B, S, 512] and k [B, S, 64] go to one pool, q [B, H, S, 64] to the last channels
// of q_out's rows.
struct PagedWriteParams {
  const void *q, *k, *v;  // q: null for none
  void* q_out;
  void* pool[2];
  const float* freqs;     // [rot / 2] radians a position, or null
  const int* page_table;
  const int* start;       // [B] or null (0)
  const int* count;       // [B] or null (S)
  unsigned* status;
  int B, H, Hkv, S, D;    // H: 0 without q
  int rot;                // channels that are rotated, 0 for none
  int q_width;            // channels of a row of q_out
  int num_pages, page_shift, max_pages;
  int token_shift;        // tokens of a block: 1 << token_shift
};

// A read: positions start ... into rows of out[0], out[1] (keys and values, or the
// latent and the rotated part).
struct PagedReadParams {
  const void* pool[2];
  void* out[2];
  const int *page_table, *start, *count;
  unsigned* status;
  int B, Hkv, S, D;
  int num_pages, page_shift, max_pages;
};

struct PagedAttnParams {
  void* o;            // [B, H, Sq, values' width]
  float* lse;         // [B, H, Sq]
  float* part_o;      // [2 * grid, values' width, part_rows] fp32, O / l of a segment
  float* part_lse;    // [2 * grid, rows of a CTA]
  const int* page_table;
  const int* length;  // [B]
  const float* slopes;
  unsigned* status;
  unsigned long long timeout_ns;
  int B, H, Hkv, Sq;
  int rows;           // (H / Hkv) * Sq query rows per kv head
  int part_rows;      // rows that a part holds: a CTA's, up to 4, 8, 16 or a multiple of 32
  int n_row_blocks;   // of a CTA's rows, or a pair's
  int sms;
  int whole;          // CTAs take whole units: no parts, no merge
  int num_pages, page_shift, max_pages;
  int pool_rows;      // rows of the pool: the coordinate of what does not exist
  int k_at, v_at;     // the arrays' places in their descriptors
  float scale, cap, inv_cap, cap_arg;
};

cudaError_t launch_paged_write(bool latent, bool bf16, bool pairs, const PagedWriteParams& p,
                               int slices, cudaStream_t stream);
cudaError_t launch_paged_read(bool latent, const PagedReadParams& p, cudaStream_t stream);

// Query rows that one pass of the attention over the keys takes, and the CTAs that
// an SM holds.  kind: 64 or 128, a head's channels; kLatent, latent rows.
int paged_attn_row_block(int kind, int rows);
// CTAs that take the same keys side by side: 2 for latent rows where there are more query
// rows than a CTA takes (128 heads, 32 sequences of up to 8192 rows: 96.2 us; each block of
// rows as a unit of its own, whose keys are read at another time, 107.9).
int paged_attn_peers(int kind, int rows);
// A CTA's least share of the keys, in chunks: the whole pipeline starts in one chunk's
// time, and the merge's is the same for any number of parts.  By 1, 2 and 4 chunks, us:
// 3 sequences of 704 latent keys 10.3, 12.5, 14.9; 8 units of 704 keys (128 channels)
// 8.6, 10.7, 11.4, of 2048 9.2, 10.1, 10.1, of 4096 11.1, 10.6, 10.2.
constexpr int kPagedMinChunks = 1;
// The end of a segment (a range of one unit's keys) takes as long as so many chunks: a unit
// is dealt as so many more, behind its own, so that a CTA with two segments has fewer
// chunks (pairs, by 1 and 3: 32 sequences of 8192 rows 112 and 111 us, 4 of 2048 and
// 4 tokens 27.9 and 27.0; by 0 and 1, 8 units of 16384 keys: 20.0 and 19.5 us).
constexpr int paged_segment(int peers) { return peers == 2 ? 3 : 1; }
// Whether page tables with room for that many keys are dealt in whole units, without a
// merge.  Whole and split, us: 8 units of 128 channels 8.5 and 8.4 at 512 keys, 10.2 and
// 8.6 at 704; 64 units 10.3 and 12.3 at 704, 13.3 and 12.6 at 1024; latent rows, 1 unit
// 6.9 and 9.4 at 128 keys, 9.6 and 9.4 at 256, 64 units 14.7 and 15.3 at 512, 18.9 and
// 17.9 at 704, 152 units 26.6 and 31.1 at 704.  17 to 64 rows of 128 channels: 8 units 10.2 and
// 10.6 at 512 keys, 64 units 16.7 and 22.5 at 1024, 160 units 24.4 and 26.0 at 704, 31.2 and
// 30.1 at 1024.
bool paged_attn_whole(int kind, long long units, int room, int sm_count);
// CTAs for `units` (of a CTA's rows, or a pair's).
int paged_attn_grid(int kind, int rows, long long units, int room, int sm_count);
cudaError_t launch_paged_attn(int kind, bool bf16, const CUtensorMap& q, const CUtensorMap& k,
                              const CUtensorMap& v, const PagedAttnParams& p, int grid,
                              cudaStream_t stream);

}  // namespace fa
