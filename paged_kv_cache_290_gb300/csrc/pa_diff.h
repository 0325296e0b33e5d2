// Launch interface of differential attention (pa_diff.cu, pa_diff_chunk.cu).
#pragma once

#include "pa_kernels.h"

namespace pa {

// AttnArgs as in pa_attention (num_q_heads counts both maps' heads; num_kv_heads both maps' keys;
// group = num_q_heads / num_kv_heads), with `out` [T, Hq / 2, 2 d], and
struct DiffArgs : AttnArgs {
  const float* lam;      // [.., Hq / 2]
  int64_t lam_stride;    // elements between tokens (0: the same for every token)
  const float* norm_w;   // [2 d], or nullptr: no norm
  float eps;
  float out_scale;
  int part_tokens;       // keys per split-context partition
  int num_pairs;         // num_kv_heads / 2
};

cudaError_t launch_diff_rows(const DiffArgs& a, const CUtensorMap& kmap, const CUtensorMap& vmap,
                             cudaStream_t stream);
cudaError_t launch_diff_merge(const DiffArgs& a, cudaStream_t stream);

}  // namespace pa
