// fa_expanded.cu -- latent attention with its heads expanded: launcher and entry
// point.
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <mutex>

#include "fa_expanded.cuh"
#include "fa_host.h"
#include "fa_merge.h"

namespace fa {
namespace {

template <bool BF16, bool kSplit>
cudaError_t launch(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                   const CUtensorMap& r, const ExpandedParams& p, int grid, cudaStream_t stream) {
  {  // the shared-memory opt-in, and the registers that the kernel's split is made
     // for, once per device
    static std::mutex mu;
    static bool done[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    std::lock_guard<std::mutex> lock(mu);
    if (!done[dev]) {
      cudaFuncAttributes a{};
      if ((e = cudaFuncGetAttributes(&a, fa_expanded_kernel<BF16, kSplit>)) != cudaSuccess) return e;
      if (a.numRegs != 128) return cudaErrorInvalidKernelImage;
      e = cudaFuncSetAttribute(fa_expanded_kernel<BF16, kSplit>,
                               cudaFuncAttributeMaxDynamicSharedMemorySize, ExpandedLayout::kSmemBytes);
      if (e != cudaSuccess) return e;
      done[dev] = true;
    }
  }
  // its setup overlaps the end of the kernel before, which it waits for
  // (programmatic dependent launch)
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = ExpandedLayout::kSmemBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fa_expanded_kernel<BF16, kSplit>, q, k, v, r, p);
}

}  // namespace
}  // namespace fa

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
size_t up256(size_t n) { return (n + 255) / 256 * 256; }

bool sizes_ok(int B, int H, int Sq, int Skv) {
  return B >= 1 && H >= 1 && Sq >= 1 && Skv >= 1 && static_cast<long long>(B) * H < 65536 &&
         Sq <= (1 << 24) && Skv <= (1 << 24);
}

// Keys split where the items are fewer than the SMs, by the smallest estimate of the
// time in ns: rounds of items, each its start and end and its key tiles, and the merge's
// start and its parts through L2.  (16 heads, 509 rows, in a graph, us by ranges: 1500 keys
// 32.3 whole, 29.6 by 2, 25.8 by 3, 24.1 by 4, 28.7 by 6; 4096 keys 76.1 whole, 36.7 by 4, 49.6
// by 6, 91.9 by 32.  The plan takes 4 in both.)
struct Plan {
  int n_qtiles, n_splits, tiles_per_split;
  size_t o_bytes, bytes;
};

Plan make_plan(int B, int H, int Sq, int Skv, int sm_count) {
  Plan p{};
  const long long sms = sm_count > 0 ? sm_count : 152;
  p.n_qtiles = (Sq + fa::kRowsPerCta - 1) / fa::kRowsPerCta;
  const long long items = static_cast<long long>(p.n_qtiles) * B * H;
  const int n_tiles = (Skv + fa::kBN - 1) / fa::kBN;
  p.n_splits = 1;
  p.tiles_per_split = n_tiles;
  if (items < sms && static_cast<long long>(B) * H * Sq <= 0x7fffffffLL) {
    constexpr long long kItem = 4000, kTile = 2200, kMerge = 6000;
    const long long rows = static_cast<long long>(B) * H * Sq;
    long long best = kItem + kTile * n_tiles;
    for (int s = 2; s <= std::min(n_tiles, 64); ++s) {
      const int per = (n_tiles + s - 1) / s, n = (n_tiles + per - 1) / per;
      const long long cost = (items * n + sms - 1) / sms * (kItem + kTile * per) + kMerge +
                             rows * n * (fa::kNope + 1) * 8 / 7000;
      if (cost < best) {
        best = cost;
        p.n_splits = n;
        p.tiles_per_split = per;
      }
    }
  }
  if (p.n_splits > 1) {
    const size_t rows = static_cast<size_t>(p.n_splits) * B * H * Sq;
    p.o_bytes = up256(rows * fa::kNope * sizeof(float));
    p.bytes = p.o_bytes + up256(rows * sizeof(float));
  }
  return p;
}

}  // namespace

extern "C" {

size_t fa_expanded_workspace_bytes(int B, int H, int Sq, int Skv) {
  return sizes_ok(B, H, Sq, Skv) ? make_plan(B, H, Sq, Skv, fa::device_sms()).bytes : 0;
}

fa_status_t fa_fwd_expanded(const void* q, const void* kv, const void* k_rope, void* o, float* lse,
                            int B, int H, int Sq, int Skv, float scale, int causal, int dtype,
                            void* workspace, size_t workspace_bytes, fa_stream_t stream) {
  if (!q || !kv || !k_rope || !o || !lse) return FA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(kv) || !aligned16(k_rope) || !aligned16(o) || !aligned16(lse))
    return FA_ERR_INVALID_ARG;
  if (!sizes_ok(B, H, Sq, Skv)) return FA_ERR_INVALID_ARG;
  if (!(scale > 0.f) || !std::isfinite(scale)) return FA_ERR_INVALID_ARG;
  if (dtype != FA_F16 && dtype != FA_BF16) return FA_ERR_UNSUPPORTED;
  if (reinterpret_cast<uintptr_t>(workspace) & 255u) return FA_ERR_WORKSPACE;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  fa::LaunchEnv env{};
  fa_status_t st = fa::launch_env(s, &env);
  if (st != FA_OK) return st;
  Plan plan = make_plan(B, H, Sq, Skv, env.sm_count);
  std::unique_lock<std::mutex> hold;
  if (plan.bytes > 0 && !workspace && !env.captured) {
    if ((st = fa::library_workspace(s, plan.bytes, &workspace, &hold)) != FA_OK) return st;
    workspace_bytes = plan.bytes;
  }
  if (plan.n_splits > 1 && (!workspace || workspace_bytes < plan.bytes)) {  // no room: no split
    plan.n_splits = 1;
    plan.tiles_per_split = (Skv + fa::kBN - 1) / fa::kBN;
  }
  const long long items = static_cast<long long>(plan.n_qtiles) * B * H * plan.n_splits;
  if (items > 0x7fffffffLL) return FA_ERR_INVALID_ARG;
  const size_t rows = static_cast<size_t>(B) * H * Sq;
  fa::ExpandedParams ep{};
  fa::PrefillParams& p = ep.a;
  p.lse = lse;
  p.o = o;
  p.status = env.status;
  p.timeout_ns = env.timeout_ns;
  p.BH = B * H;
  p.Sq = Sq;
  p.Skv = Skv;
  p.n_qtiles = plan.n_qtiles;
  p.n_items = static_cast<int>(items);
  p.causal = causal ? 1 : 0;
  p.lpt = 1;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.rescale_tau = 8.f;
  p.n_splits = plan.n_splits;
  p.tiles_per_split = plan.tiles_per_split;
  ep.H = H;
  if (plan.n_splits > 1) {
    p.part_o = static_cast<float*>(workspace);
    p.part_lse = reinterpret_cast<float*>(static_cast<char*>(workspace) + plan.o_bytes);
  }
  const bool bf16 = dtype == FA_BF16;
  CUtensorMap tq, tk, tv, tr;
  if ((st = fa::encode_rows(&tq, q, fa::ExpandedLayout::kDq, Sq, B * H, fa::kBM, bf16)) != FA_OK) return st;
  if ((st = fa::encode_rows(&tk, kv, 2 * fa::kNope, Skv, B * H, fa::kBN, bf16)) != FA_OK) return st;
  if ((st = fa::encode_rows(&tv, kv, 2 * fa::kNope, Skv, B * H, 64, bf16)) != FA_OK) return st;
  if ((st = fa::encode_rows(&tr, k_rope, fa::kLatentRope, Skv, B, fa::kBN, bf16)) != FA_OK) return st;
  p.sched = fa::take_sched_slot(env);
  const int grid = static_cast<int>(std::min<long long>(items, env.sm_count > 0 ? env.sm_count : 1));
  const cudaError_t e =
      plan.n_splits > 1 ? (bf16 ? fa::launch<true, true>(tq, tk, tv, tr, ep, grid, s)
                                : fa::launch<false, true>(tq, tk, tv, tr, ep, grid, s))
                        : (bf16 ? fa::launch<true, false>(tq, tk, tv, tr, ep, grid, s)
                                : fa::launch<false, false>(tq, tk, tv, tr, ep, grid, s));
  if (e != cudaSuccess) return FA_ERR_CUDA;
  if (plan.n_splits > 1) {
    const fa::MergeParams m{p.part_o, p.part_lse, o, lse, static_cast<long long>(rows), plan.n_splits};
    if (fa::launch_merge(fa::kNope, bf16, m, s) != cudaSuccess) return FA_ERR_CUDA;
  }
  return FA_OK;
}

}  // extern "C"
