// fa_score_d128.cu -- instantiations and launcher of the score-modifying kernel
// for head dimension 128.
#include "fa_score_launch.cuh"

namespace fa {

cudaError_t score_num_regs_d128(bool bf16, int* regs) {
  return bf16 ? score_regs<128, true>(regs) : score_regs<128, false>(regs);
}

cudaError_t launch_score_d128(bool bf16, const CUtensorMap& q, const CUtensorMap& k,
                             const CUtensorMap& v, const CUtensorMap& o, const ScoreParams& p,
                             int grid, cudaStream_t stream) {
  return bf16 ? score_launch<128, true>(q, k, v, o, p, grid, stream)
              : score_launch<128, false>(q, k, v, o, p, grid, stream);
}

}  // namespace fa
