// fa_merge.cuh -- merge of one query row's partials over ranges of the keys:
// O = sum_s w_s O_s / sum_s w_s with w_s = exp(LSE_s - max LSE), LSE = max LSE +
// ln sum_s w_s.
//
// One warp takes a row of few parts, the four warps of a block a row of many,
// dealt between them; eight loads of a lane are in flight at once.  With few
// rows the work is a chain of a few memory latencies, with many it is the
// bytes, 4 (D + 1) a part.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "sm103_ptx.cuh"

namespace fa {

constexpr int kMergeWarps = 4;

template <int D>
struct MergeSmem {
  float part[kMergeWarps][D];
  float sums[kMergeWarps], tops[kMergeWarps];
};

// A warp's share of a row: parts first, first + step, ... of n_parts.  Returns
// their largest LSE, against which o and sum are weighted (-inf: none has a
// key).  part_row(s): the row of part s in part_o [., D] (fp32, O / l) and
// part_lse [.]; LSE = -inf with O = 0 where a part has no visible key.
template <int D, class PartRow>
__device__ __forceinline__ float merge_parts(const float* part_o, const float* part_lse,
                                             int n_parts, int first, int step, PartRow part_row,
                                             float (&o)[D / 32], float& sum) {
  constexpr int kDims = D / 32, kAtOnce = 8;
  constexpr float kLog2e = 1.4426950408889634f;
  const int lane = threadIdx.x & 31;
  float top = -INFINITY;
  sum = 0.f;
#pragma unroll
  for (int d = 0; d < kDims; ++d) o[d] = 0.f;
  for (int s0 = first; s0 < n_parts; s0 += step * kAtOnce) {
    float lse[kAtOnce], x[kAtOnce][kDims];
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      const int s = s0 + k * step;
      lse[k] = -INFINITY;
#pragma unroll
      for (int d = 0; d < kDims; ++d) x[k][d] = 0.f;
      if (s < n_parts) {
        const long long at = part_row(s);
        lse[k] = part_lse[at];
        const float* po = part_o + at * D + lane * kDims;
        if constexpr (kDims == 4) {
          const float4 v = *reinterpret_cast<const float4*>(po);
          x[k][0] = v.x; x[k][1] = v.y; x[k][2] = v.z; x[k][3] = v.w;
        } else {
          const float2 v = *reinterpret_cast<const float2*>(po);
          x[k][0] = v.x; x[k][1] = v.y;
        }
      }
    }
    float now = top;
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) now = fmaxf(now, lse[k]);
    const float base = now == -INFINITY ? 0.f : now;
    const float old = ex2_approx((top - base) * kLog2e);
    top = now;
    sum *= old;
#pragma unroll
    for (int d = 0; d < kDims; ++d) o[d] *= old;
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      const float w = ex2_approx((lse[k] - base) * kLog2e);
      sum += w;
#pragma unroll
      for (int d = 0; d < kDims; ++d) o[d] = fmaf(w, x[k][d], o[d]);
    }
  }
  return top;
}

template <bool BF16>
__device__ __forceinline__ uint32_t merge_pack(float a, float b) {
  if constexpr (BF16) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
  } else {
    const __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
}

// The row by the whole block.
template <int D, bool BF16, class PartRow>
__device__ __forceinline__ void merge_row(const float* part_o, const float* part_lse, int n_parts,
                                          PartRow part_row, void* o_out, float* lse_out,
                                          long long row, MergeSmem<D>& sm) {
  constexpr int kDims = D / 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float o[kDims], sum;
  float top = merge_parts<D>(part_o, part_lse, n_parts, warp, kMergeWarps, part_row, o, sum);
#pragma unroll
  for (int d = 0; d < kDims; ++d) sm.part[warp][lane * kDims + d] = o[d];
  if (lane == 0) {
    sm.sums[warp] = sum;
    sm.tops[warp] = top;
  }
  __syncthreads();
  const int ch = 2 * static_cast<int>(threadIdx.x);
  if (ch >= D) return;
  float a = 0.f, b = 0.f;
  sum = 0.f;
  top = sm.tops[0];
#pragma unroll
  for (int w = 1; w < kMergeWarps; ++w) top = fmaxf(top, sm.tops[w]);
  const float base = top == -INFINITY ? 0.f : top;
#pragma unroll
  for (int w = 0; w < kMergeWarps; ++w) {
    const float f = ex2_approx((sm.tops[w] - base) * 1.4426950408889634f);
    a = fmaf(sm.part[w][ch], f, a);
    b = fmaf(sm.part[w][ch + 1], f, b);
    sum = fmaf(sm.sums[w], f, sum);
  }
  // no part has a key: 0; a NaN stays one
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  reinterpret_cast<uint32_t*>(o_out)[(row * D + ch) / 2] = merge_pack<BF16>(a * inv, b * inv);
  if (ch == 0) lse_out[row] = sum == 0.f ? -INFINITY : top + logf(sum);
}

// The row by one warp.
template <int D, bool BF16, class PartRow>
__device__ __forceinline__ void merge_row_warp(const float* part_o, const float* part_lse,
                                               int n_parts, PartRow part_row, void* o_out,
                                               float* lse_out, long long row) {
  constexpr int kDims = D / 32;
  const int lane = threadIdx.x & 31;
  float o[kDims], sum;
  const float top = merge_parts<D>(part_o, part_lse, n_parts, 0, 1, part_row, o, sum);
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  uint32_t* out = reinterpret_cast<uint32_t*>(o_out) + (row * D + lane * kDims) / 2;
  if constexpr (kDims == 4) {
    *reinterpret_cast<uint2*>(out) = make_uint2(merge_pack<BF16>(o[0] * inv, o[1] * inv),
                                                merge_pack<BF16>(o[2] * inv, o[3] * inv));
  } else {
    *out = merge_pack<BF16>(o[0] * inv, o[1] * inv);
  }
  if (lane == 0) lse_out[row] = sum == 0.f ? -INFINITY : top + logf(sum);
}

}  // namespace fa
