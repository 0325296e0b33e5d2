// Device helper shared by the kernels of query chunks: which sequence a grid row serves.
#pragma once

#include "pa_common.cuh"
#include "pa_kernels.h"

namespace pa {

// Grid row z of a prefill launch serves the z-th sequence with more than one query row (a
// block-wide ballot scan of query_start_loc, all threads of the CTA), so decode rows cost the
// launch nothing.  Returns that sequence, or -1 past the last one; more such sequences than
// grid rows (or, when the decode launch was skipped on the hint's word, a one-row sequence) is
// a hint error.
template <int kThreads>
__device__ __forceinline__ int find_prefill_seq(const AttnArgs& a, int* warp_count,
                                                int* chosen_seq, int target, bool first) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) *chosen_seq = -1;
  int found = 0;  // prefill sequences seen so far
  for (int s0 = 0; s0 < a.num_seqs; s0 += kThreads) {
    const int si = s0 + tid;
    const int ql = si < a.num_seqs ? a.query_start_loc[si + 1] - a.query_start_loc[si] : 0;
    const bool pf = ql > 1;
    const unsigned bal = __ballot_sync(0xffffffffu, pf);
    if (a.decode_skipped && __any_sync(0xffffffffu, ql == 1) && lane == 0 && first)
      atomicOr(a.err, kErrHint);
    if (lane == 0) warp_count[warp] = __popc(bal);
    __syncthreads();
    int rank = found + __popc(bal & ((1u << lane) - 1u)), total = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
      rank += w < warp ? warp_count[w] : 0;
      total += warp_count[w];
    }
    if (pf && rank == target) *chosen_seq = si;
    found += total;
    __syncthreads();
  }
  __syncthreads();
  if (found > a.prefill_seqs && first && tid == 0) atomicOr(a.err, kErrHint);
  return *chosen_seq;
}

}  // namespace pa
