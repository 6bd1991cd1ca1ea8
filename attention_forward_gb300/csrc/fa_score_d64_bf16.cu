// fa_score_d64_bf16.cu -- the score-modifying kernel's forms for head dimension
// 64, bf16.
#include "fa_score_launch.cuh"

namespace fa {

cudaError_t score_num_regs_d64_bf16(int* regs) { return score_regs<64, true>(regs); }

cudaError_t launch_score_d64_bf16(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                                const CUtensorMap& o, const ScoreParams& p, int grid,
                                cudaStream_t stream) {
  return score_launch<64, true>(q, k, v, o, p, grid, stream);
}

}  // namespace fa
