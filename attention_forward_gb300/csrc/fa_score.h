// fa_score.h -- parameter block and launch entry points of the attention with
// modified scores (internal).
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include "fa_internal.h"

namespace fa {

// Terms of the tanh polynomial (odd).
constexpr int kCapTerms = 4;
// |score / cap| up to which it is used.
constexpr float kCapPolyMax = 0.5f;

struct ScoreParams {
  float* lse;                 // [B*H, Sq]
  unsigned long long* sched;  // this launch's scheduler slot
  unsigned* status;
  unsigned long long timeout_ns;
  int H, Hkv, group, Sq, Skv;  // group = H / Hkv
  // Rows are taken per row head: a query head's Sq rows, or, packed, the
  // group * Sq rows of the query heads that share a kv head.
  int packed;
  int row_heads;              // B * H, or packed B * Hkv
  int rows;                   // rows of a row head
  int halves;                 // items of 128 rows, whose key tiles the stages share
  int n_qtiles;               // ceil(rows / rows of an item)
  int n_items;                // n_qtiles * row_heads * n_splits
  int causal;
  float scale_log2;           // scale * log2(e)
  int capped;                 // scores have a tanh cap
  int cap_fixed;              // and the cap bounds them: no reference maximum
  float cap_mul;              // t = s * cap_mul: 1, or the scale (plan_cap)
  float cap_poly[kCapTerms];  // log2-scaled score = t * (c0 + c1 t^2 + ...)
  float cap_t_max, cap_u_max; // |t| and t^2 up to which the polynomial holds
  float cap_u_fast;           // the latter where t is s itself, else -1
  float cap_arg;              // t * cap_arg = 2 log2(e) s scale / cap
  float cap_log2;             // cap * log2(e)
  const float* slopes;        // [H] or null
  const int* prefix;          // [B] or null
  const int* doc_q;           // [B, Sq] or null
  const int* doc_k;           // [B, Skv]
  // per batch row: the id that all keys of a tile have (kDocMixed: none), and
  // the key tiles [x, y) of each 128-row stage that hold documents of its rows
  const int* tile_doc;        // [B, n_key_tiles]
  const int2* stage_tiles;    // [B, n_stages]
  int n_key_tiles, n_stages;
  int n_splits, tiles_per_split;
  float* part_o;              // n_splits > 1: [n_splits, B*H*Sq, D] fp32, O / l
  float* part_lse;
};

constexpr int kDocMixed = -2147483647 - 1;

struct DocParams {
  const int* doc_q;   // [B, Sq]
  const int* doc_k;   // [B, Skv]
  int* tile_doc;      // [B, n_key_tiles]
  int2* tile_range;   // [B, n_key_tiles]: smallest and largest id >= 0
  int2* stage_tiles;  // [B, n_stages]
  int B, Sq, Skv, rows, n_key_tiles, n_stages;
};

cudaError_t launch_doc_tiles(const DocParams& p, cudaStream_t stream);
cudaError_t score_num_regs(int D, bool bf16, int* regs);
cudaError_t launch_score(int D, bool bf16, const CUtensorMap& q, const CUtensorMap& k,
                         const CUtensorMap& v, const CUtensorMap& o, const ScoreParams& p,
                         int grid, cudaStream_t stream);

}  // namespace fa
