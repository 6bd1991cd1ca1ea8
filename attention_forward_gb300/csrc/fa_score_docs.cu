// fa_score_docs.cu -- what the documents of a call leave to compute: per key
// tile the id all of its keys share, per 128-row stage the tiles that hold
// documents of its rows.
//
// One block per batch row, two passes over its ids (4 bytes a token against
// the attention's 4 D per key and head): the id range of every key tile, then
// for every stage the first and last tile whose range meets the range of the
// stage's rows.  Ranges cover any order of ids; documents that lie together
// make them exact.
#include <climits>

#include "fa_score.h"

namespace fa {
namespace {

constexpr int kDocThreads = 1024;

__global__ void __launch_bounds__(kDocThreads) fa_doc_tiles_kernel(const DocParams p) {
  const int b = static_cast<int>(blockIdx.x);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int kWarps = kDocThreads / 32;
  const int* dk = p.doc_k + static_cast<size_t>(b) * p.Skv;
  const int* dq = p.doc_q + static_cast<size_t>(b) * p.Sq;
  int* tile_doc = p.tile_doc + static_cast<size_t>(b) * p.n_key_tiles;
  int2* range = p.tile_range + static_cast<size_t>(b) * p.n_key_tiles;
  int2* stage = p.stage_tiles + static_cast<size_t>(b) * p.n_stages;

  for (int t = warp; t < p.n_key_tiles; t += kWarps) {
    int lo = INT_MAX, hi = -1, least = INT_MAX;
#pragma unroll
    for (int k = 0; k < kBN / 32; ++k) {
      const int key = t * kBN + 32 * k + lane;
      if (key < p.Skv) {
        const int d = dk[key];
        least = min(least, d);
        if (d >= 0) {
          lo = min(lo, d);
          hi = max(hi, d);
        }
      }
    }
    lo = __reduce_min_sync(0xffffffffu, lo);
    hi = __reduce_max_sync(0xffffffffu, hi);
    least = __reduce_min_sync(0xffffffffu, least);
    if (lane == 0) {
      range[t] = make_int2(lo, hi);
      tile_doc[t] = lo == hi && least >= 0 ? lo : kDocMixed;
    }
  }
  __syncthreads();

  for (int s = warp; s < p.n_stages; s += kWarps) {
    const int first = s * kBM, last = min(first + kBM, p.rows) - 1;
    // the query tokens among the stage's rows (packed rows run through the
    // group's heads: a stage across two of them has every token)
    int i0 = first % p.Sq, i1 = last % p.Sq;
    if (first / p.Sq != last / p.Sq) {
      i0 = 0;
      i1 = p.Sq - 1;
    }
    int lo = INT_MAX, hi = -1;
    for (int i = i0 + lane; i <= i1; i += 32) {
      const int d = dq[i];
      if (d >= 0) {
        lo = min(lo, d);
        hi = max(hi, d);
      }
    }
    lo = __reduce_min_sync(0xffffffffu, lo);
    hi = __reduce_max_sync(0xffffffffu, hi);
    int t0 = INT_MAX, t1 = -1;
    for (int t = lane; t < p.n_key_tiles; t += 32) {
      const int2 r = range[t];
      if (r.x <= hi && r.y >= lo && r.x <= r.y && lo <= hi) {
        t0 = min(t0, t);
        t1 = max(t1, t);
      }
    }
    t0 = __reduce_min_sync(0xffffffffu, t0);
    t1 = __reduce_max_sync(0xffffffffu, t1);
    if (lane == 0) stage[s] = t1 < 0 ? make_int2(0, 0) : make_int2(t0, t1 + 1);
  }
}

}  // namespace

cudaError_t launch_doc_tiles(const DocParams& p, cudaStream_t stream) {
  fa_doc_tiles_kernel<<<p.B, kDocThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace fa
