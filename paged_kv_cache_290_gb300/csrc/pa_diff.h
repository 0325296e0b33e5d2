// Launch interface of differential attention (pa_diff.cu, pa_diff_chunk.cu).
#pragma once

#include "pa_kernels.h"

namespace pa {

constexpr int kChunkKeys = 128;  // keys per tile of the chunk kernels

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
  int group_inv;         // 65536 / group + 1
  int stages;            // units in flight per warp of the rows kernel
  int max_seq_len;       // the hint's
  int tile_q;            // query rows of a chunk tile: 128 / group
  int chunk_tiles;       // chunk tiles of the longest chunk
  uint32_t pairs_inv;    // ceil(2^32 / num_pairs)
  int key_splits;        // ranges of the keys that the chunk kernel's CTAs share out
  float* chunk_o;        // partials of the chunk kernel: [T, Hq, key_splits, 2 d]
  float* chunk_m;        // [T, Hq, key_splits], log2 units
  float* chunk_l;
};

cudaError_t launch_diff_rows(const DiffArgs& a, const CUtensorMap& kmap, const CUtensorMap& vmap,
                             cudaStream_t stream);
cudaError_t launch_diff_merge(const DiffArgs& a, cudaStream_t stream);
cudaError_t launch_diff_chunk(const DiffArgs& a, const CUtensorMap& kmap, const CUtensorMap& vmap,
                              cudaStream_t stream);
cudaError_t launch_diff_chunk_merge(const DiffArgs& a, cudaStream_t stream);

}  // namespace pa
