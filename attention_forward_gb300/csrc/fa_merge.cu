// fa_merge.cu -- merge of split-key partials: O = sum_s w_s O_s / sum_s w_s with
// w_s = exp(LSE_s - max LSE), LSE = max LSE + ln sum_s w_s.
//
// One block of four warps per row.  The ranges are dealt to the warps, eight
// loads of a lane in flight at once: the kernel is a chain of a few dependent
// memory latencies, not of bytes (4 (D + 1) per row and range).  Each block
// reads all ranges' LSE again, a lane each.  It starts while the kernel before
// it still runs (programmatic dependent launch).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fa_merge.h"
#include "sm103_ptx.cuh"

namespace fa {
namespace {

constexpr int kMergeWarps = 4;

template <int D, bool BF16>
__global__ void __launch_bounds__(kMergeWarps * 32) fa_merge_kernel(const MergeParams p) {
  constexpr int kDims = D / 32, kAtOnce = 8;
  constexpr float kLog2e = 1.4426950408889634f;
  __shared__ float part[kMergeWarps][D];
  __shared__ float sums[kMergeWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long row = blockIdx.x;
  grid_dependency_wait();
  float top = -INFINITY;
  for (int s = lane; s < p.n_splits; s += 32) top = fmaxf(top, p.part_lse[s * p.rows + row]);
#pragma unroll
  for (int k = 16; k >= 1; k >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, k));
  const float base = top == -INFINITY ? 0.f : top;
  float sum = 0.f, o[kDims] = {};
  for (int s0 = warp; s0 < p.n_splits; s0 += kMergeWarps * kAtOnce) {
    float lse[kAtOnce], x[kAtOnce][kDims];
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      const int s = s0 + k * kMergeWarps;
      lse[k] = -INFINITY;
#pragma unroll
      for (int d = 0; d < kDims; ++d) x[k][d] = 0.f;
      if (s < p.n_splits) {
        const long long at = s * p.rows + row;
        lse[k] = p.part_lse[at];
        const float* po = p.part_o + at * D + lane * kDims;
        if constexpr (kDims == 4) {
          const float4 v = *reinterpret_cast<const float4*>(po);
          x[k][0] = v.x; x[k][1] = v.y; x[k][2] = v.z; x[k][3] = v.w;
        } else {
          const float2 v = *reinterpret_cast<const float2*>(po);
          x[k][0] = v.x; x[k][1] = v.y;
        }
      }
    }
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      const float w = ex2_approx((lse[k] - base) * kLog2e);
      sum += w;
#pragma unroll
      for (int d = 0; d < kDims; ++d) o[d] = fmaf(w, x[k][d], o[d]);
    }
  }
#pragma unroll
  for (int d = 0; d < kDims; ++d) part[warp][lane * kDims + d] = o[d];
  if (lane == 0) sums[warp] = sum;
  __syncthreads();
  const int ch = 2 * static_cast<int>(threadIdx.x);
  if (ch >= D) return;
  float a = 0.f, b = 0.f;
  sum = 0.f;
#pragma unroll
  for (int w = 0; w < kMergeWarps; ++w) {
    a += part[w][ch];
    b += part[w][ch + 1];
    sum += sums[w];
  }
  // no range has a key: 0; a NaN stays one
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  uint32_t out;
  if constexpr (BF16) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a * inv, b * inv);
    out = *reinterpret_cast<const uint32_t*>(&v);
  } else {
    const __half2 v = __floats2half2_rn(a * inv, b * inv);
    out = *reinterpret_cast<const uint32_t*>(&v);
  }
  reinterpret_cast<uint32_t*>(p.o)[(row * D + ch) / 2] = out;
  if (ch == 0) p.lse[row] = sum == 0.f ? -INFINITY : top + logf(sum);
}

template <int D, bool BF16>
cudaError_t launch(const MergeParams& p, cudaStream_t stream) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(p.rows), 1, 1);
  cfg.blockDim = dim3(kMergeWarps * 32, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fa_merge_kernel<D, BF16>, p);
}

}  // namespace

cudaError_t launch_merge(int D, bool bf16, const MergeParams& p, cudaStream_t stream) {
  if (D == 128) return bf16 ? launch<128, true>(p, stream) : launch<128, false>(p, stream);
  return bf16 ? launch<64, true>(p, stream) : launch<64, false>(p, stream);
}

}  // namespace fa
