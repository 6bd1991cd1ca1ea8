// fa_score_docs.cu -- what the documents of a call leave to compute: per key
// tile the id all of its keys share, per 128-row stage the tiles that hold
// documents of its rows.
//
// One warp a task, two kernels or one (below), each a few dependent loads long (4
// bytes a token are read): the id ranges of every key tile and every stage's rows, then
// for every stage the first and last tile whose range meets its own.  Ranges
// cover any order of ids; documents that lie together make them exact.  As one
// block per batch row they took 15 us for 16384 tokens.
#include <climits>

#include "fa_score.h"
#include "sm103_ptx.cuh"

namespace fa {
namespace {

constexpr int kDocWarps = 8;
// Up to 64 tasks one kernel does both, a launch less on the host: whole calls of
// 100, 2000, 4000, 8000 tokens (2, 32, 63, 126 tasks) took 8.2, 14.0, 22.7, 28.1 us
// with it, 8.9, 14.4, 22.4, 26.3 with two.
constexpr int kDocOneWarps = 32, kDocOneTasks = 64;

__device__ __forceinline__ int2 warp_range(int lo, int hi) {
  return make_int2(__reduce_min_sync(0xffffffffu, lo), __reduce_max_sync(0xffffffffu, hi));
}

// Tasks 0 ... n_key_tiles - 1: the smallest and largest id >= 0 of a tile's
// keys, and the id they all have; the others: those of a stage's rows.
__device__ __forceinline__ void doc_range(const DocParams& p, int b, int task, int lane) {
  int lo = INT_MAX, hi = -1, least = INT_MAX;
  if (task < p.n_key_tiles) {
    const int* dk = p.doc_k + static_cast<size_t>(b) * p.Skv;
#pragma unroll
    for (int k = 0; k < kBN / 32; ++k) {
      const int key = task * kBN + 32 * k + lane;
      if (key < p.Skv) {
        const int d = dk[key];
        least = min(least, d);
        if (d >= 0) {
          lo = min(lo, d);
          hi = max(hi, d);
        }
      }
    }
    const int2 r = warp_range(lo, hi);
    least = __reduce_min_sync(0xffffffffu, least);
    if (lane == 0) {
      p.tile_range[static_cast<size_t>(b) * p.n_key_tiles + task] = r;
      p.tile_doc[static_cast<size_t>(b) * p.n_key_tiles + task] =
          r.x == r.y && least >= 0 ? r.x : kDocMixed;
    }
    return;
  }
  const int* dq = p.doc_q + static_cast<size_t>(b) * p.Sq;
  const int s = task - p.n_key_tiles, first = s * kBM, last = min(first + kBM, p.rows) - 1;
  // the query tokens among the stage's rows (packed rows run through the
  // group's heads: a stage across two of them has every token)
  int i0 = first % p.Sq, i1 = last % p.Sq;
  if (first / p.Sq != last / p.Sq) {
    i0 = 0;
    i1 = p.Sq - 1;
  }
  // at most 128 tokens: a stage has 128 rows, packed rows at most 128 tokens
#pragma unroll
  for (int k = 0; k < kBM / 32; ++k) {
    const int i = i0 + 32 * k + lane;
    if (i <= i1) {
      const int d = dq[i];
      if (d >= 0) {
        lo = min(lo, d);
        hi = max(hi, d);
      }
    }
  }
  const int2 r = warp_range(lo, hi);
  if (lane == 0) p.stage_tiles[static_cast<size_t>(b) * p.n_stages + s] = r;
}

// A stage's range of ids, as its task left it, to its range of tiles.
__device__ __forceinline__ void doc_tiles(const DocParams& p, int b, int s, int lane) {
  int2* stage = p.stage_tiles + static_cast<size_t>(b) * p.n_stages + s;
  const int2* range = p.tile_range + static_cast<size_t>(b) * p.n_key_tiles;
  const int2 mine = *stage;
  int t0 = INT_MAX, t1 = -1;
#pragma unroll 4
  for (int t = lane; t < p.n_key_tiles; t += 32) {
    const int2 r = range[t];
    if (r.x <= mine.y && r.y >= mine.x && r.x <= r.y && mine.x <= mine.y) {
      t0 = min(t0, t);
      t1 = max(t1, t);
    }
  }
  const int2 r = warp_range(t0, t1);
  if (lane == 0) *stage = r.y < 0 ? make_int2(0, 0) : make_int2(r.x, r.y + 1);
}

__global__ void __launch_bounds__(kDocWarps * 32) fa_doc_ranges_kernel(const DocParams p) {
  const int task = static_cast<int>(blockIdx.x) * kDocWarps + (threadIdx.x >> 5);
  grid_dependency_wait();
  grid_launch_dependents();
  if (task < p.n_key_tiles + p.n_stages)
    doc_range(p, static_cast<int>(blockIdx.y), task, threadIdx.x & 31);
}

__global__ void __launch_bounds__(kDocWarps * 32) fa_doc_tiles_kernel(const DocParams p) {
  const int s = static_cast<int>(blockIdx.x) * kDocWarps + (threadIdx.x >> 5);
  grid_dependency_wait();
  grid_launch_dependents();
  if (s < p.n_stages) doc_tiles(p, static_cast<int>(blockIdx.y), s, threadIdx.x & 31);
}

// Both, a block to a batch row.
__global__ void __launch_bounds__(kDocOneWarps * 32) fa_doc_one_kernel(const DocParams p) {
  const int b = static_cast<int>(blockIdx.y), warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  grid_dependency_wait();
  grid_launch_dependents();
  for (int task = warp; task < p.n_key_tiles + p.n_stages; task += kDocOneWarps)
    doc_range(p, b, task, lane);
  __syncthreads();
  for (int s = warp; s < p.n_stages; s += kDocOneWarps) doc_tiles(p, b, s, lane);
}

cudaError_t launch(void (*kernel)(DocParams), int blocks, int warps, const DocParams& p,
                   cudaStream_t stream) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks), static_cast<unsigned>(p.B), 1);
  cfg.blockDim = dim3(static_cast<unsigned>(warps) * 32, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace

cudaError_t launch_doc_tiles(const DocParams& p, cudaStream_t stream) {
  const int tasks = p.n_key_tiles + p.n_stages;
  if (tasks <= kDocOneTasks) return launch(fa_doc_one_kernel, 1, kDocOneWarps, p, stream);
  auto blocks = [](int n) { return (n + kDocWarps - 1) / kDocWarps; };
  const cudaError_t e = launch(fa_doc_ranges_kernel, blocks(tasks), kDocWarps, p, stream);
  return e != cudaSuccess ? e : launch(fa_doc_tiles_kernel, blocks(p.n_stages), kDocWarps, p, stream);
}

}  // namespace fa
