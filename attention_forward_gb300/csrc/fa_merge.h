// fa_merge.h -- merge of split-key partials (internal).
#pragma once
#include <cuda_runtime.h>

namespace fa {

struct MergeParams {
  const float* part_o;    // [n_splits, rows, D] fp32, O / l of each key range
  const float* part_lse;  // [n_splits, rows]; -inf with O = 0: a range without keys
  void* o;                // [rows, D] 16-bit
  float* lse;             // [rows]
  long long rows;
  int n_splits;
};

// Launched to overlap the end of the kernel that writes the partials: it waits
// for that grid before it reads them.
cudaError_t launch_merge(int D, bool bf16, const MergeParams& p, cudaStream_t stream);

}  // namespace fa
