// Device code that the rows kernel, the chunk kernels and the merges of differential attention share.
#pragma once

#include "pa_common.cuh"
#include "pa_diff.h"

namespace pa {

// The two element-type values of a word.
template <bool BF>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
  if constexpr (BF)
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  else
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

// A block's search for its chunk: the descriptor found (s = -1: none).
template <int kThreads>
struct ChunkScan {
  int warp_count[kThreads / 32];
  int s, row0, q_len, L;
};

// The sequence of rank z among those with more than one query row: longest first while the batch
// has at most 128 sequences (the longest CTAs then start first and the grid's tail is short: 4 x
// 512 rows behind 2k to 7.5k keys 206 against 215 us in batch order), else in batch order.  Every
// thread holds one sequence's descriptor, and the chosen one is handed on through shared memory,
// without a second round of loads.  keys: 128 words of shared memory.  All threads of the block
// call it.  `first` (one block of the grid): more such sequences than grid rows, or, when no rows
// kernel was launched on the hint's word, a one-row sequence, is reported.
template <int kThreads>
__device__ __forceinline__ void find_chunk(const DiffArgs& a, ChunkScan<kThreads>& sc, int* keys,
                                           int z, bool first) {
  static_assert(kThreads >= 128, "a batch that is sorted fits one round");
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) sc.s = -1;
  int found = 0;
  const bool sorted = a.num_seqs <= 128;
  for (int s0 = 0; s0 < a.num_seqs; s0 += kThreads) {
    const int si = s0 + tid;
    const bool in = si < a.num_seqs;
    const int row0 = in ? a.query_start_loc[si] : 0;
    const int q_len = in ? a.query_start_loc[si + 1] - row0 : 0;
    const int L = in ? a.seq_lens[si] : 0;
    const unsigned bal = __ballot_sync(0xffffffffu, q_len > 1);
    if (a.decode_skipped && first && __any_sync(0xffffffffu, q_len == 1) && lane == 0)
      atomicOr(a.err, kErrHint);
    if (lane == 0) sc.warp_count[warp] = __popc(bal);
    const int key = q_len > 1 ? max(L, 0) : -1;
    if (sorted && tid < 128) keys[tid] = key;
    __syncthreads();
    int rank = found + __popc(bal & ((1u << lane) - 1u));
    if (!sorted || first) {
#pragma unroll
      for (int w = 0; w < kThreads / 32; ++w) {
        rank += w < warp ? sc.warp_count[w] : 0;
        found += sc.warp_count[w];
      }
    }
    if (sorted && q_len > 1) {
      rank = 0;
      for (int j = 0; j < a.num_seqs; ++j)  // the same word for every thread: a broadcast
        rank += keys[j] > key || (keys[j] == key && j < tid);
    }
    if (q_len > 1 && rank == z) {
      sc.s = si;
      sc.row0 = row0;
      sc.q_len = q_len;
      sc.L = L;
    }
    __syncthreads();
  }
  __syncthreads();
  if (first && tid == 0 && found > a.prefill_seqs) atomicOr(a.err, kErrHint);
}

}  // namespace pa
