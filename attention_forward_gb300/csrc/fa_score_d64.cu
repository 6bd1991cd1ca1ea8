// fa_score_d64.cu -- instantiations and launcher of the score-modifying kernel
// for head dimension 64.
#include "fa_score_launch.cuh"

namespace fa {

cudaError_t score_num_regs_d64(bool bf16, int* regs) {
  return bf16 ? score_regs<64, true>(regs) : score_regs<64, false>(regs);
}

cudaError_t launch_score_d64(bool bf16, const CUtensorMap& q, const CUtensorMap& k,
                             const CUtensorMap& v, const CUtensorMap& o, const ScoreParams& p,
                             int grid, cudaStream_t stream) {
  return bf16 ? score_launch<64, true>(q, k, v, o, p, grid, stream)
              : score_launch<64, false>(q, k, v, o, p, grid, stream);
}

}  // namespace fa
