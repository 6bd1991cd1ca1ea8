// fa_score_api.cu -- fa_fwd_score: argument checks, the plan of rows, tiles and
// key ranges, the tanh coefficients, and the launches.
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <mutex>

#include "fa_host.h"
#include "fa_merge.h"
#include "fa_score.h"

namespace fa {

#define FA_SCORE_FORM(n)                                                                     \
  cudaError_t score_num_regs_##n(int* regs);                                                 \
  cudaError_t launch_score_##n(const CUtensorMap&, const CUtensorMap&, const CUtensorMap&,   \
                               const CUtensorMap&, const ScoreParams&, int, cudaStream_t);
FA_SCORE_FORM(d128_bf16)
FA_SCORE_FORM(d128_f16)
FA_SCORE_FORM(d64_bf16)
FA_SCORE_FORM(d64_f16)
#undef FA_SCORE_FORM

cudaError_t score_num_regs(int D, bool bf16, int* regs) {
  if (D == 128) return bf16 ? score_num_regs_d128_bf16(regs) : score_num_regs_d128_f16(regs);
  return bf16 ? score_num_regs_d64_bf16(regs) : score_num_regs_d64_f16(regs);
}
cudaError_t launch_score(int D, bool bf16, const CUtensorMap& q, const CUtensorMap& k,
                         const CUtensorMap& v, const CUtensorMap& o, const ScoreParams& p,
                         int grid, cudaStream_t stream) {
  if (D == 128)
    return bf16 ? launch_score_d128_bf16(q, k, v, o, p, grid, stream)
                : launch_score_d128_f16(q, k, v, o, p, grid, stream);
  return bf16 ? launch_score_d64_bf16(q, k, v, o, p, grid, stream)
              : launch_score_d64_f16(q, k, v, o, p, grid, stream);
}

}  // namespace fa

namespace {

// Query tokens up to which the heads of a group are rows of one tile: a tile
// of one head would be at most half full.
constexpr int kPackTokens = 128;

size_t up256(size_t n) { return (n + 255) / 256 * 256; }

// How the work is cut where its items are fewer than the SMs: into key ranges,
// and into items of 128 rows whose key tiles the two stages share (halves)
// instead of 128 rows a stage.  The smallest estimated time wins, in twentieths
// of the time of a key tile of 256 rows (1.7 us): rounds of one item an SM, each
// the tiles of a range, 20 to begin it and, split, 120 for 256 rows of 128
// channels of partials written and read again; and 30 for the merge.  A tile of
// an item in halves takes 12.  A split has to gain an eighth.  Measured, us, all
// causal, with a cap: 8 heads of one token over 700 keys 12.6 whole, 9.9 split; of
// 128 over 2048 23.0 and 12.8; 2 x 8 heads of 1021 x 1500 27.6 with 256 rows, 19.9
// in halves; 16 of 1024 x 4096 52.6 (in 2 ranges) and 39.0; 8 of 2048 x 2048 34.1
// and 23.5 (105 in 16 ranges).  Several items an SM, D = 128, 256 rows and halves:
// 352 heads of 300 42.4 and 35.7; 128 of 800 47.5 and 45.4; 640 of 300 x 1000 167 and
// 169 (D = 64 153 and 118); and where 256 rows are taken, 1024 heads of 400 111 and
// 138, 1024 of 148 x 1000 138 and 183, but 1024 of 300 102 and 90: a last item of few
// rows costs more than the rounds say.  Every key tile counts as visible, those that
// documents rule out included: their ids are the device's to read.
struct Cut {
  int halves, splits;
  long long cost;
};

Cut cut_items(int row_heads, int rows, bool halves, int D, int n_tiles, int sm_count) {
  const int item_rows = halves ? fa::kBM : fa::kRowsPerCta;
  const long long n = static_cast<long long>(row_heads) * ((rows + item_rows - 1) / item_rows);
  const long long sms = sm_count > 0 ? sm_count : 152;
  const int tile = halves ? 12 : 20;
  const int part = 120 * std::min(rows, item_rows) * D / (256 * 128);
  Cut c{halves ? 1 : 0, 1, (n + sms - 1) / sms * (tile * n_tiles + 20)};
  if (n >= sms) return c;
  long long best = c.cost * 7 / 8;
  for (int s = 2; s <= std::min(n_tiles, 64); ++s) {
    const int tiles = (n_tiles + s - 1) / s, ranges = (n_tiles + tiles - 1) / tiles;
    const long long cost = (n * ranges + sms - 1) / sms * (tile * tiles + 20 + part) + 30;
    if (cost < best) {
      best = c.cost = cost;
      c.splits = ranges;
    }
  }
  return c;
}

struct Plan {
  int packed, row_heads, rows, halves, n_qtiles, n_key_tiles, n_stages;
  int n_splits, tiles_per_split;
  size_t doc_bytes, split_bytes;  // the workspace's two parts, documents first
};

Plan make_plan(int B, int H, int Hkv, int Sq, int Skv, int D, bool documents, int sm_count) {
  Plan p{};
  const int group = H / Hkv;
  p.packed = group > 1 && Sq <= kPackTokens ? 1 : 0;
  p.row_heads = p.packed ? B * Hkv : B * H;
  p.rows = p.packed ? group * Sq : Sq;
  p.n_key_tiles = (Skv + fa::kBN - 1) / fa::kBN;
  p.n_stages = (p.rows + fa::kBM - 1) / fa::kBM;
  Cut cut = cut_items(p.row_heads, p.rows, p.rows <= fa::kBM, D, p.n_key_tiles, sm_count);
  if (p.rows > fa::kBM) {
    const Cut one = cut_items(p.row_heads, p.rows, true, D, p.n_key_tiles, sm_count);
    if (one.cost < cut.cost) cut = one;
  }
  p.halves = cut.halves;
  const int item_rows = p.halves ? fa::kBM : fa::kRowsPerCta;
  p.n_qtiles = (p.rows + item_rows - 1) / item_rows;
  const long long all_rows = static_cast<long long>(p.row_heads) * p.rows;
  const int s = all_rows > 0x7fffffffLL ? 1 : cut.splits;  // the merge's grid
  p.tiles_per_split = (p.n_key_tiles + s - 1) / s;
  p.n_splits = (p.n_key_tiles + p.tiles_per_split - 1) / p.tiles_per_split;
  if (documents)
    p.doc_bytes = up256(static_cast<size_t>(B) * p.n_key_tiles * sizeof(int)) +
                  up256(static_cast<size_t>(B) * p.n_key_tiles * sizeof(int2)) +
                  up256(static_cast<size_t>(B) * p.n_stages * sizeof(int2));
  if (p.n_splits > 1) {
    const size_t rows = static_cast<size_t>(p.n_splits) * static_cast<size_t>(all_rows);
    p.split_bytes = up256(rows * D * sizeof(float)) + up256(rows * sizeof(float));
  }
  return p;
}

bool sizes_ok(int B, int H, int Hkv, int Sq, int Skv) {
  return B >= 1 && H >= 1 && Hkv >= 1 && Sq >= 1 && Skv >= 1 && H % Hkv == 0 &&
         static_cast<long long>(B) * H < 65536 && Sq <= (1 << 24) && Skv <= (1 << 24);
}

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// cap tanh(s scale / cap) log2(e) = s (c0 + c1 s^2 + c2 s^4 + c3 s^6) while
// |s scale / cap| <= y_max.  The terms are the minimax fit (exchange algorithm)
// of y + a1 y^3 + a2 y^5 + a3 y^7 to tanh on [0, 0.5]: off by 2e-7 and 1.0e-6 of
// the value at most, by less than 1e-8 up to 0.05, where most scores are.
void plan_cap(fa::ScoreParams& p, double scale, double cap, bool bf16) {
  static const double kTanh[fa::kCapTerms] = {1.0, -0.33326461, 0.13185862, -0.0442293};
  // |y| up to which the first three alone are within 2e-7 (1.4e-6 of the value)
  constexpr double kThreeMax = 0.145;
  constexpr double kLog2e = 1.4426950408889634;
  const double k = scale / cap;
  double c[fa::kCapTerms], y_max = fa::kCapPolyMax;
  bool held = scale < 1e36;  // fp32 holds the terms of s
  for (int i = 0; i < fa::kCapTerms; ++i) {
    c[i] = std::pow(k, 2 * i) * scale;
    held = held && c[i] < 1e36 && (c[i] > 1e-36 || i == fa::kCapTerms - 1);
  }
  if (c[fa::kCapTerms - 1] <= 1e-36) {  // the cap is far above the scores
    c[fa::kCapTerms - 1] = 0.0;
    y_max = kThreeMax;
  }
  held = held && y_max / k > 1e-18 && y_max / k < 1e18;
  // else the terms of s scale, which caps of 1e-6 ... 1e6 keep within fp32, behind
  // a product more, where the exponentials are
  if (!held) {
    y_max = fa::kCapPolyMax;
    for (int i = 0; i < fa::kCapTerms; ++i) c[i] = std::pow(cap, -2 * i);
  }
  for (int i = 0; i < fa::kCapTerms; ++i) p.cap_poly[i] = static_cast<float>(kTanh[i] * kLog2e * c[i]);
  p.cap_mul = held ? 1.f : static_cast<float>(scale);
  // the product in fp32: |t| <= cap_t_max exactly where t^2 <= cap_u_max
  p.cap_t_max = static_cast<float>(held ? y_max / k : y_max * cap);
  p.cap_u_max = p.cap_t_max * p.cap_t_max;
  p.cap_u_fast = held ? p.cap_u_max : -1.f;
  p.cap_arg = static_cast<float>(2.0 * kLog2e * (held ? k : 1.0 / cap));
  p.cap_log2 = static_cast<float>(cap * kLog2e);
  p.capped = 1;
  // |x| <= 72.5 (a cap of 50) leaves 2^x, its sums and products normal
  p.cap_fixed = held && bf16 && !p.slopes && p.cap_log2 <= 72.5f ? 1 : 0;
}

}  // namespace

extern "C" size_t fa_score_workspace_bytes(int B, int H, int Hkv, int Sq, int Skv, int D,
                                           int documents) {
  if (!sizes_ok(B, H, Hkv, Sq, Skv) || (D != 64 && D != 128)) return 0;
  const Plan p = make_plan(B, H, Hkv, Sq, Skv, D, documents != 0, fa::device_sms());
  return p.doc_bytes + p.split_bytes;
}

extern "C" int fa_score_item_rows(int B, int H, int Hkv, int Sq, int Skv, int D) {
  if (!sizes_ok(B, H, Hkv, Sq, Skv) || (D != 64 && D != 128)) return 0;
  return make_plan(B, H, Hkv, Sq, Skv, D, false, fa::device_sms()).halves ? fa::kBM : fa::kRowsPerCta;
}

extern "C" int fa_score_key_ranges(int B, int H, int Hkv, int Sq, int Skv, int D) {
  if (!sizes_ok(B, H, Hkv, Sq, Skv) || (D != 64 && D != 128)) return 0;
  return make_plan(B, H, Hkv, Sq, Skv, D, false, fa::device_sms()).n_splits;
}

extern "C" fa_status_t fa_fwd_score(const void* q, const void* k, const void* v, void* o,
                                    float* lse, int B, int H, int Hkv, int Sq, int Skv, int D,
                                    float scale, int causal, int dtype, float softcap,
                                    const float* slopes, const int* doc_q, const int* doc_k,
                                    const int* prefix, void* workspace, size_t workspace_bytes,
                                    fa_stream_t stream) {
  // the checks that fa_fwd makes, then those of what is new
  if (!sizes_ok(B, H, Hkv, Sq, Skv)) return FA_ERR_INVALID_ARG;
  if (!fa::softcap_ok(softcap)) return FA_ERR_INVALID_ARG;
  if ((doc_q == nullptr) != (doc_k == nullptr)) return FA_ERR_INVALID_ARG;
  if (prefix && !causal) return FA_ERR_INVALID_ARG;
  if (!aligned4(slopes) || !aligned4(doc_q) || !aligned4(doc_k) || !aligned4(prefix))
    return FA_ERR_INVALID_ARG;
  fa_status_t st = fa::check_args(q, k, v, o, lse, B, H, Sq, Skv, D, scale, dtype);
  if (st != FA_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  fa::LaunchEnv env{};
  if ((st = fa::launch_env(s, &env)) != FA_OK) return st;
  const bool bf16 = dtype == FA_BF16;
  {
    // the kernel's register split assumes 128 registers a thread
    static std::mutex mu;
    static bool ok[2][2] = {};
    std::lock_guard<std::mutex> lock(mu);
    if (!ok[D == 128][bf16]) {
      int regs = 0;
      if (fa::score_num_regs(D, bf16, &regs) != cudaSuccess) return FA_ERR_CUDA;
      if (regs != 128) return FA_ERR_UNSUPPORTED;
      ok[D == 128][bf16] = true;
    }
  }

  Plan plan = make_plan(B, H, Hkv, Sq, Skv, D, doc_k != nullptr, env.sm_count);
  if (reinterpret_cast<uintptr_t>(workspace) & 255u) return FA_ERR_WORKSPACE;
  size_t have = workspace ? workspace_bytes : 0;
  const size_t need = plan.doc_bytes + plan.split_bytes;
  std::unique_lock<std::mutex> hold;
  if (!workspace && need > 0 && !env.captured) {
    if ((st = fa::library_workspace(s, need, &workspace, &hold)) != FA_OK) return st;
    have = need;
  }
  if (have < plan.doc_bytes) return FA_ERR_WORKSPACE;
  if (have < plan.doc_bytes + plan.split_bytes) {
    plan.n_splits = 1;
    plan.tiles_per_split = plan.n_key_tiles;
  }

  fa::ScoreParams p{};
  p.lse = lse;
  p.status = env.status;
  p.timeout_ns = env.timeout_ns;
  p.H = H;
  p.Hkv = Hkv;
  p.group = H / Hkv;
  p.Sq = Sq;
  p.Skv = Skv;
  p.packed = plan.packed;
  p.row_heads = plan.row_heads;
  p.rows = plan.rows;
  p.halves = plan.halves;
  p.n_qtiles = plan.n_qtiles;
  p.causal = causal ? 1 : 0;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.slopes = slopes;
  if (softcap > 0.f) plan_cap(p, scale, softcap, bf16);
  p.prefix = prefix;
  p.n_splits = plan.n_splits;
  p.tiles_per_split = plan.tiles_per_split;
  char* ws = static_cast<char*>(workspace);
  if (doc_k) {
    fa::DocParams dp{};
    dp.doc_q = doc_q;
    dp.doc_k = doc_k;
    dp.tile_doc = reinterpret_cast<int*>(ws);
    ws += up256(static_cast<size_t>(B) * plan.n_key_tiles * sizeof(int));
    dp.tile_range = reinterpret_cast<int2*>(ws);
    ws += up256(static_cast<size_t>(B) * plan.n_key_tiles * sizeof(int2));
    dp.stage_tiles = reinterpret_cast<int2*>(ws);
    ws += up256(static_cast<size_t>(B) * plan.n_stages * sizeof(int2));
    dp.B = B;
    dp.Sq = Sq;
    dp.Skv = Skv;
    dp.rows = plan.rows;
    dp.n_key_tiles = plan.n_key_tiles;
    dp.n_stages = plan.n_stages;
    p.doc_q = doc_q;
    p.doc_k = doc_k;
    p.tile_doc = dp.tile_doc;
    p.stage_tiles = dp.stage_tiles;
    p.n_key_tiles = plan.n_key_tiles;
    p.n_stages = plan.n_stages;
    if (fa::launch_doc_tiles(dp, s) != cudaSuccess) return FA_ERR_CUDA;
  }
  const size_t rows = static_cast<size_t>(plan.row_heads) * static_cast<size_t>(plan.rows);
  if (plan.n_splits > 1) {
    p.part_o = reinterpret_cast<float*>(ws);
    p.part_lse = reinterpret_cast<float*>(ws + up256(plan.n_splits * rows * D * sizeof(float)));
  }
  const long long n_items = static_cast<long long>(plan.n_qtiles) * plan.row_heads * plan.n_splits;
  if (n_items > 0x7fffffffLL) return FA_ERR_INVALID_ARG;
  p.n_items = static_cast<int>(n_items);

  const int kv_heads = B * Hkv;
  CUtensorMap tq, tk, tv, to;
  if ((st = fa::encode_rows(&tq, q, D, plan.rows, plan.row_heads, fa::kBM, bf16)) != FA_OK) return st;
  if ((st = fa::encode_rows(&tk, k, D, Skv, kv_heads, fa::kBN, bf16)) != FA_OK) return st;
  if ((st = fa::encode_rows(&tv, v, D, Skv, kv_heads, fa::kBN, bf16)) != FA_OK) return st;
  if ((st = fa::encode_rows(&to, o, D, plan.rows, plan.row_heads, 32, bf16)) != FA_OK) return st;
  p.sched = fa::take_sched_slot(env);
  const int grid = static_cast<int>(std::min<long long>(n_items, env.sm_count > 0 ? env.sm_count : 1));
  if (fa::launch_score(D, bf16, tq, tk, tv, to, p, grid, s) != cudaSuccess) return FA_ERR_CUDA;
  if (plan.n_splits > 1) {
    const fa::MergeParams m{p.part_o, p.part_lse, o, lse, static_cast<long long>(rows),
                            plan.n_splits};
    if (fa::launch_merge(D, bf16, m, s) != cudaSuccess) return FA_ERR_CUDA;
  }
  return FA_OK;
}
