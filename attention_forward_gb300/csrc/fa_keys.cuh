// fa_keys.cuh -- what the attentions over paged caches share: the deal of the
// keys to persistent CTAs by the lengths that the device finds, and the tanh cap.
// P: a parameter block with B, Hkv, n_row_blocks, max_pages, page_shift, length,
// status, cap, inv_cap and cap_arg.
#pragma once
#include "fa_cache.h"
#include "sm103_ptx.cuh"

namespace fa {

// cap tanh(x / cap): for |y| = |x / cap| < 1/4 the odd series through y^7 (its
// next term is 3e-7 of the value), else 1 - 2 / (1 + e^(2 y)), which is off by
// a few 2^-24 of the cap and saturates to +-cap as the exponential reaches
// infinity or 0.
template <class P>
__device__ __forceinline__ float cap_score(float x, const P& p) {
  const float y = x * p.inv_cap, u = y * y;
  const float small = fmaf(u, fmaf(u, fmaf(u, -17.f / 315.f, 2.f / 15.f), -1.f / 3.f), 1.f) * x;
  const float e = ex2_approx(x * p.cap_arg);
  const float large = fmaf(-2.f * p.cap, __fdividef(1.f, 1.f + e), p.cap);
  return u < 0.0625f ? small : large;
}

// ---- how the work is dealt to the CTAs (the merge kernels use it too) ----
// A sequence's length, limited to what its page table can hold.
template <class P>
__device__ __forceinline__ int cache_length(const P& p, int b) {
  return max(0, min(p.length[b], p.max_pages << p.page_shift));
}

// Chunks of a unit of that length; one without keys is a chunk all the same.
__device__ __forceinline__ int cache_chunks(int len) {
  return max(1, (len + kCacheAttnKeys - 1) / kCacheAttnKeys);
}

// All C chunks dealt to n CTAs: C / n each, the first C % n one more.  C < 2^31
// (fa_fwd_cache checks it).
struct CacheDeal {
  int n, per, more;
  __device__ __forceinline__ int begin(int x) const { return x * per + min(x, more); }
  __device__ __forceinline__ int cta_of(int c) const {
    const int big = more * (per + 1);  // chunks of the CTAs that have one more
    return c < big ? c / (per + 1) : more + (c - big) / per;
  }
};

// At least `least` chunks to a CTA.
__device__ __forceinline__ CacheDeal cache_deal(int all, int grid, int least = kCacheMinChunks) {
  CacheDeal d;
  d.n = min((all + least - 1) / least, grid);
  d.per = all / d.n;
  d.more = all - d.per * d.n;
  return d;
}

// Of a block of kWarps warps.
template <int kWarps>
struct KeyScan {
  int warp_sum[kWarps];
  int before, b, len;
};

// The block's threads take the sequences in runs of equal length and add up
// their chunks.  Returns the chunks of all units, and a unit's of the sequences
// before the thread's run (`upto`); `report` records lengths that had to be
// limited.  `extra`: chunks more that every unit is dealt as, behind its own.
template <class P, int kWarps>
__device__ __forceinline__ int cache_scan(const P& p, KeyScan<kWarps>& s, bool report, int& upto,
                                          int extra = 0) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int run = (p.B + 32 * kWarps - 1) / (32 * kWarps);
  const int b0 = min(p.B, static_cast<int>(threadIdx.x) * run), b1 = min(p.B, b0 + run);
  int sum = 0;
  for (int b = b0; b < b1; ++b) {
    const int len = cache_length(p, b);
    if (report && len != p.length[b]) atomicMax(p.status, kStatusBadIndex);
    sum += cache_chunks(len) + extra;
  }
  int inc = sum;
#pragma unroll
  for (int k = 1; k < 32; k <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, inc, k);
    if (lane >= k) inc += o;
  }
  if (lane == 31) s.warp_sum[warp] = inc;
  __syncthreads();
  int base = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) base += s.warp_sum[w];
    all += s.warp_sum[w];
  }
  upto = base + inc - sum;
  return all * (p.Hkv * p.n_row_blocks);
}

// The sequence of chunk c, its length, and the chunks before it (all units').
template <class P, int kWarps>
__device__ __forceinline__ void cache_find(const P& p, KeyScan<kWarps>& s, int upto, int c, int& b,
                                           int& len, int& before, int extra = 0) {
  const int run = (p.B + 32 * kWarps - 1) / (32 * kWarps);
  const int b0 = min(p.B, static_cast<int>(threadIdx.x) * run), b1 = min(p.B, b0 + run);
  const int units = p.Hkv * p.n_row_blocks;
  int at = upto * units;
  for (int k = b0; k < b1 && at <= c; ++k) {
    const int l = cache_length(p, k);
    const int n = (cache_chunks(l) + extra) * units;
    if (c < at + n) {
      s.before = at;
      s.b = k;
      s.len = l;
    }
    at += n;
  }
  __syncthreads();
  b = s.b;
  len = s.len;
  before = s.before;
}

}  // namespace fa
