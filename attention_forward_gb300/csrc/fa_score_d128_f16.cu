// fa_score_d128_f16.cu -- the score-modifying kernel's forms for head dimension
// 128, fp16.
#include "fa_score_launch.cuh"

namespace fa {

cudaError_t score_num_regs_d128_f16(int* regs) { return score_regs<128, false>(regs); }

cudaError_t launch_score_d128_f16(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                                const CUtensorMap& o, const ScoreParams& p, int grid,
                                cudaStream_t stream) {
  return score_launch<128, false>(q, k, v, o, p, grid, stream);
}

}  // namespace fa
