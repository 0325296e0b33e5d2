// Differential attention over a paged KV cache: rows of decode steps and short chunks, the merges,
// and the entry point.  Longer chunks: pa_diff_chunk.cu.
//
// Heads come in pairs.  Of q, heads 2p and 2p + 1 are the queries of the two softmax maps of
// differential head p; of the pool, K heads 2j and 2j + 1 are the two maps' keys and V heads
// 2j, 2j + 1 the two halves of one 2d-wide value (so the pool is what the scatter-write fills).
// With j = p / (Hq / Hkv):
//   y = softmax(s q_2p K_2j^T) V_j - lambda_p softmax(s q_2p+1 K_2j+1^T) V_j,
//   out = c y                                   or, with a norm weight w of 2d values,
//   out = c y rsqrt(mean(y^2) + eps) w.
// The subtraction is of two normalised sums, both float32; nothing is rounded before `out`.
//
// Rows kernel: CTA = (sequence, kv-head pair, 4 or 8 columns, partition of the keys), a column being
// a (query row, head).  One read of the four heads' K/V units serves all of its columns and both
// maps.  Bound by HBM: 32 rows behind 8192 keys (64 + 8 heads of 128) 167.8 us = 6.41 TB/s, 0.96 of
// the measured copy rate; 64 rows behind 512 to 4096 keys 94.7 us = 6.58 TB/s.
//   * a warp streams 16-token units (K1, K2, Va, Vb: 4 x 16 x d values, two copies) through its
//     own ring of 2 TMA stages, or 3 or 6 where a small grid leaves the SM's shared memory free
//     (one sequence of 4096 keys: 17 -> 11 us with the partitions below);
//   * S^T = K Q^T (m16n8k16: 16 tokens x 8 columns); P^T through movmatrix; O^T += V^T P^T over
//     2d rows.  NT = 1 packs 4 columns of both maps into one 8-wide tile (columns 0-3 map 1,
//     4-7 map 2: each K's product with the whole tile, of which its own half is kept, so that one
//     P V product serves both maps); NT = 2 has 8 columns, a tile per map.
//   * online softmax per column as in the decode kernel (a reference maximum raised only past
//     2^8), scores masked by a select, V rows past the sequence's end zeroed.  Each weight goes into
//     the product as two numbers, its rounding and the rest, so only `out` is rounded.
// A sequence within one partition is finished in the CTA; otherwise (m, l, O / l) partials of
// both maps go to the workspace and the merge kernel joins them (log-sum-exp), subtracts and
// normalises.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <string>

#include "pa.h"
#include "pa_common.cuh"
#include "pa_diff.cuh"
#include "pa_host.h"

namespace pa {
namespace {

constexpr int kSms = 152;

template <int D, int NT>
struct RowsCfg {
  static constexpr int kWarps = D == 128 ? 2 : 4;
  static constexpr int kThreads = kWarps * 32;
  static constexpr int kHalves = D / 64;
  static constexpr int kBoxBytes = 16 * 128;
  static constexpr int kHeadBytes = kHalves * kBoxBytes;  // one head's K (or V) of a unit
  static constexpr int kStageBytes = 4 * kHeadBytes;      // K1, K2, Va, Vb
  static constexpr int kMaxStages = 6;                    // per warp; the launch chooses 2, 3 or 6
  static_assert(2 * kWarps * kStageBytes == 64 * 1024, "three CTAs of two stages fit an SM");
  static constexpr int kMaxUnits = 64;                    // units of the longest partition
  static constexpr int kDK = D / 16;
  static constexpr int kMT = 2 * D / 16;                  // 16-row tiles of O^T
  static constexpr int kCols = 4 * NT;                    // columns per map
  static constexpr int kMergeBytes = kWarps * 8 * NT * (2 * D + 2) * 4;
  static constexpr int smem_bytes(int stages) { return kWarps * stages * kStageBytes + 1024; }
  static_assert(kMergeBytes <= 2 * kWarps * kStageBytes, "the warps' sums fit the rings");
  static constexpr float kRaiseLog2 = 8.f;
};

// y of one differential head (kV consecutive dims per lane, a warp per head) -> out.
template <int D, bool BF>
__device__ __forceinline__ void finish_head(const DiffArgs& a, float (&y)[2 * D / 32], int64_t row,
                                            int head, int lane) {
  constexpr int kV = 2 * D / 32;
  float f = a.out_scale;
  if (a.norm_w) {
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < kV; ++i) ss += y[i] * y[i];
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
    f *= rsqrtf(ss * (1.f / (2 * D)) + a.eps);
#pragma unroll
    for (int i = 0; i < kV; ++i) y[i] *= __ldg(a.norm_w + lane * kV + i);
  }
  uint32_t w[kV / 2];
#pragma unroll
  for (int i = 0; i < kV / 2; ++i) w[i] = pack2<BF>(y[2 * i] * f, y[2 * i + 1] * f);
  __half* dst = a.out + (row * (a.num_q_heads / 2) + head) * (2 * D) + lane * kV;
  if constexpr (kV == 8)
    *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
  else
    *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
}

template <int D, int BS, int NT, bool BF>
__global__ void __launch_bounds__(RowsCfg<D, NT>::kThreads)
    diff_rows_kernel(const __grid_constant__ CUtensorMap kmap,
                     const __grid_constant__ CUtensorMap vmap, const DiffArgs a) {
  using C = RowsCfg<D, NT>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bars[C::kWarps][C::kMaxStages];
  __shared__ int32_t unit_row[C::kMaxUnits];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));

  // Grid x = (partition, column group), y = kv-head pair, z = sequence.  A column is a (query
  // row, head of the pair's group), row-major.
  const int ncg = a.col_groups;
  const int cg = static_cast<int>(blockIdx.x) % ncg;
  const int part = static_cast<int>(blockIdx.x) / ncg;
  const int j = blockIdx.y, s = blockIdx.z;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const bool lead = blockIdx.x == 0;
  grid_launch_dependents();
  // Every CTA waits for the grid before it on the stream, even one that leaves early, so that
  // the stream's order stays transitive.
  auto leave = [] { grid_dependency_wait(); };

  const int row0 = a.query_start_loc[s];
  const int row_end = a.query_start_loc[s + 1];
  const int L = a.seq_lens[s];
  const int tok_begin = part * a.part_tokens;
  int32_t unit_blk[(C::kMaxUnits + C::kThreads - 1) / C::kThreads];
#pragma unroll
  for (int i = 0; i < static_cast<int>(sizeof(unit_blk) / 4); ++i) {
    const int u = tid + i * C::kThreads, col = (tok_begin + u * 16) / BS;
    unit_blk[i] = u * 16 < a.part_tokens && col < a.max_blocks
                      ? a.block_tables[static_cast<int64_t>(s) * a.bt_stride + col]
                      : 0;
  }
  const int q_len = row_end - row0;
  if (q_len < 1 || q_len > a.verify_rows) {
    // Longer than the hint's max_query_len: nobody's, unless chunk kernels were launched.
    if (q_len > 1 && a.prefill_seqs == 0 && lead && j == 0 && tid == 0) atomicOr(a.err, kErrHint);
    return leave();
  }
  if (row0 < 0 || row0 + q_len > a.num_tokens || L < q_len || (L + BS - 1) / BS > a.max_blocks) {
    if (lead && tid == 0) atomicOr(a.err, kErrDescriptor);
    return leave();
  }
  const int nparts = (L + a.part_tokens - 1) / a.part_tokens;
  const int ncols = q_len * a.group, col0 = cg * C::kCols;
  if (nparts > a.max_parts || (ncols + C::kCols - 1) / C::kCols > ncg) {
    if (lead && tid == 0) atomicOr(a.err, kErrHint);
    return leave();
  }
  if (col0 >= ncols || part >= nparts) return leave();
  const int ctx = L - q_len;  // row i sees keys 0 .. ctx + i
  const int my_cols = min(C::kCols, ncols - col0);

  const int tok_end = min(L, tok_begin + a.part_tokens);
  const int nunits = (tok_end - tok_begin + 15) >> 4;
  int bad = 0;
#pragma unroll
  for (int i = 0; i < static_cast<int>(sizeof(unit_blk) / 4); ++i) {
    const int u = tid + i * C::kThreads;
    if (u < nunits) {
      const int tok = tok_begin + u * 16;
      int y = 0;
      if (unit_blk[i] >= 0 && unit_blk[i] < a.num_blocks)
        y = (unit_blk[i] * a.num_kv_heads + 2 * j) * BS + (tok % BS);
      else
        bad = 1;
      unit_row[u] = y;
    }
  }
  if (lane == 0) {
    for (int st = 0; st < a.stages; ++st) mbar_init(smem_addr(&bars[warp][st]), 1);
    mbar_init_fence();
  }
  // A partition without a result says so in its cells (l = -1), and the merge leaves such rows.
  auto cell = [&](int cc, int m) {
    const int c = col0 + cc;
    return ((static_cast<int64_t>(s) * a.verify_rows + c / a.group) * a.num_q_heads +
            2 * (j * a.group + c % a.group) + m) * a.max_parts + part;
  };
  auto no_result = [&] {
    if (nparts > 1 && tid < 2 * my_cols) a.part_l[cell(tid >> 1, tid & 1)] = -1.f;
  };
  if (__syncthreads_or(bad)) {
    if (tid == 0) atomicOr(a.err, kErrBlockRange);
    leave();
    return no_result();
  }

  const int my_n = warp < nunits ? (nunits - warp + C::kWarps - 1) / C::kWarps : 0;
  const int stages = a.stages;
  const uint32_t ring = smem_addr(smem + warp * stages * C::kStageBytes);
  const uint32_t bar0 = smem_addr(&bars[warp][0]);
  const uint64_t pol = l2_policy_evict_first();  // read once
  auto issue = [&](int i, int st) {  // lane 0: unit i of this warp into stage st = i % stages
    const uint32_t bar = bar0 + st * 8;
    const uint32_t dst = ring + st * C::kStageBytes;
    const int y = unit_row[warp + i * C::kWarps];
    mbar_arrive_expect_tx(bar, C::kStageBytes);
    // one box each: [half][head][16 rows][128 B]
    tma_load_4d_hint(dst, &kmap, 0, y % BS, y / BS, 0, bar, pol);
    tma_load_4d_hint(dst + 2 * C::kHeadBytes, &vmap, 0, y % BS, y / BS, 0, bar, pol);
  };
  grid_dependency_wait();  // q and the pools now hold what the kernels before wrote
  if (lane == 0) {
    for (int i = 0; i < min(my_n, stages); ++i) issue(i, i);
  }

  // Q^T as the B operand: n index gq of tile nt is (map, column).
  const int gq = lane >> 2, cq = lane & 3;
  uint32_t qf[NT][C::kDK][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int map = NT == 1 ? gq >> 2 : nt, cc = NT == 1 ? gq & 3 : gq;
    const bool hv = cc < my_cols;
    const int c = col0 + (hv ? cc : 0);
    const __half* qrow = a.q + static_cast<int64_t>(row0 + c / a.group) * a.q_stride +
                         static_cast<int64_t>(2 * (j * a.group + c % a.group) + map) * D;
#pragma unroll
    for (int k = 0; k < C::kDK; ++k)
#pragma unroll
      for (int e = 0; e < 2; ++e)
        qf[nt][k][e] = hv ? __ldg(reinterpret_cast<const unsigned int*>(qrow + k * 16 + 8 * e +
                                                                        2 * cq))
                          : 0u;
  }
  // Last key that this lane's accumulator columns (2cq, 2cq + 1 of each tile) may see.
  int lim[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int cc = NT == 1 ? 2 * (cq & 1) + e : 2 * cq + e;
      lim[nt][e] = cc < my_cols ? ctx + (col0 + cc) / a.group : L - 1;
    }

  float o[NT][C::kMT][4];
  float m_run[NT][2], l_run[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int dt = 0; dt < C::kMT; ++dt) o[nt][dt][0] = o[nt][dt][1] = o[nt][dt][2] = o[nt][dt][3] = 0.f;
    m_run[nt][0] = m_run[nt][1] = -INFINITY;
    l_run[nt][0] = l_run[nt][1] = 0.f;
  }

  const int mi = lane >> 3, mr = lane & 7;
  int failed_at = -1;
  int st = 0, phase = 0;  // i % stages, i / stages & 1
  for (int i = 0; i < my_n; ++i) {
    const bool ok = mbar_wait_short(bar0 + st * 8, phase, a.err, a.wait_limit_ns);
    if (__any_sync(0xffffffffu, !ok)) {
      failed_at = i;
      break;
    }
    const int u = warp + i * C::kWarps;
    const int nvalid = min(16, tok_end - (tok_begin + u * 16));
    const uint32_t kb = ring + st * C::kStageBytes;
    const uint32_t vb = kb + 2 * C::kHeadBytes;

    // ---- S^T[16 tokens][8 columns] of each map
    float sacc[2][4];
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      sacc[m][0] = sacc[m][1] = sacc[m][2] = sacc[m][3] = 0.f;
      const int nt = NT == 1 ? 0 : m;
#pragma unroll
      for (int k = 0; k < C::kDK; ++k) {
        const int tok = mr + ((mi & 1) << 3);
        const int chunk = 2 * k + (mi >> 1);
        uint32_t af[4];
        ldsm_x4(kb + (chunk >> 3) * (2 * C::kBoxBytes) + m * C::kBoxBytes + swz128(tok, chunk & 7), af);
        mma_16816<BF>(sacc[m], af, qf[nt][k][0], qf[nt][k][1]);
      }
    }

    const int kp0 = tok_begin + u * 16 + gq, kp1 = kp0 + 8;
    const bool v0 = gq < nvalid, v1 = gq + 8 < nvalid;
    float sc[NT][4];
    bool raise = false;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float x[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        x[e] = (NT == 1 ? (cq < 2 ? sacc[0][e] : sacc[1][e]) : sacc[nt][e]) * a.scale_log2;
      sc[nt][0] = v0 && kp0 <= lim[nt][0] ? x[0] : -INFINITY;
      sc[nt][1] = v0 && kp0 <= lim[nt][1] ? x[1] : -INFINITY;
      sc[nt][2] = v1 && kp1 <= lim[nt][0] ? x[2] : -INFINITY;
      sc[nt][3] = v1 && kp1 <= lim[nt][1] ? x[3] : -INFINITY;
      raise |= fmaxf(sc[nt][0], sc[nt][2]) > m_run[nt][0] + C::kRaiseLog2;
      raise |= fmaxf(sc[nt][1], sc[nt][3]) > m_run[nt][1] + C::kRaiseLog2;
    }
    if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float mx = fmaxf(sc[nt][e], sc[nt][2 + e]);
          mx = warp_max_xor(mx, 4);
          mx = warp_max_xor(mx, 8);
          mx = warp_max_xor(mx, 16);
          const float mn = fmaxf(m_run[nt][e], mx);
          const float al = mn == -INFINITY ? 1.f : exp2f(m_run[nt][e] - mn);
          m_run[nt][e] = mn;
          l_run[nt][e] *= al;
#pragma unroll
          for (int dt = 0; dt < C::kMT; ++dt) {
            o[nt][dt][e] *= al;
            o[nt][dt][2 + e] *= al;
          }
        }
    }
    uint32_t pb0[NT], pb1[NT], lo0[NT], lo1[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      // a column with no visible key yet is still at m = -inf: subtract 0, so that p = 0, not NaN
      const float b0 = m_run[nt][0] == -INFINITY ? 0.f : m_run[nt][0];
      const float b1 = m_run[nt][1] == -INFINITY ? 0.f : m_run[nt][1];
      const float p00 = exp2f(sc[nt][0] - b0), p10 = exp2f(sc[nt][2] - b0);
      const float p01 = exp2f(sc[nt][1] - b1), p11 = exp2f(sc[nt][3] - b1);
      l_run[nt][0] += p00 + p10;
      l_run[nt][1] += p01 + p11;
      // P goes into the matrix product as two element-type numbers, the rounded weight and the
      // rounded rest: 2^-22 (fp16) or 2^-16 (bf16) of a weight is lost instead of 2^-11 or 2^-8,
      // which is the output's own rounding, counted twice by the difference of two maps.  The
      // second product is hidden behind HBM (32 sequences of 8k keys: 167 -> 169 us).
      const uint32_t h0 = pack2<BF>(p00, p01), h1 = pack2<BF>(p10, p11);
      const float2 f0 = unpack2<BF>(h0), f1 = unpack2<BF>(h1);
      pb0[nt] = movmatrix_trans(h0);
      pb1[nt] = movmatrix_trans(h1);
      lo0[nt] = movmatrix_trans(pack2<BF>(p00 - f0.x, p01 - f0.y));
      lo1[nt] = movmatrix_trans(pack2<BF>(p10 - f1.x, p11 - f1.y));
    }

    if (nvalid < 16) {  // V rows past the end: p is 0 there, but 0 * NaN is not
      constexpr int kRowChunks = 2 * C::kHalves * 8;  // of Va and Vb
      for (int c = lane; c < (16 - nvalid) * kRowChunks; c += 32) {
        const int row = nvalid + c / kRowChunks, k = c % kRowChunks;
        asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(
                         vb + (k >> 3) * C::kBoxBytes + row * 128 + (k & 7) * 16),
                     "r"(0)
                     : "memory");
      }
      __syncwarp();
    }
    // ---- O^T[2d][columns] += V^T[2d][16 tokens] P^T
#pragma unroll
    for (int dt = 0; dt < C::kMT; ++dt) {
      const int tok = mr + ((mi >> 1) << 3);
      const int chunk = 2 * dt + (mi & 1);  // of the 2d-wide row: head, half, 16-byte chunk
      const int half = (chunk >> 3) % C::kHalves, hd = (chunk >> 3) / C::kHalves;
      uint32_t af[4];
      ldsm_x4_trans(vb + half * (2 * C::kBoxBytes) + hd * C::kBoxBytes + swz128(tok, chunk & 7), af);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        mma_16816<BF>(o[nt][dt], af, pb0[nt], pb1[nt]);
        mma_16816<BF>(o[nt][dt], af, lo0[nt], lo1[nt]);
      }
    }

    __syncwarp();
    if (lane == 0 && i + stages < my_n) {
      fence_proxy_async();
      issue(i + stages, st);
    }
    if (++st == stages) {
      st = 0;
      phase ^= 1;
    }
  }

  if (failed_at >= 0 && lane == 0) {  // let the copies in flight land before leaving
    const int issued = min(my_n, failed_at + stages);
    for (int i = failed_at + 1; i < issued; ++i)
      mbar_wait(bar0 + (i % stages) * 8, (i / stages) & 1, a.err, a.wait_limit_ns);
  }

  // ---- join the warps
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float l = l_run[nt][e];
      l += __shfl_xor_sync(0xffffffffu, l, 4);
      l += __shfl_xor_sync(0xffffffffu, l, 8);
      l += __shfl_xor_sync(0xffffffffu, l, 16);
      l_run[nt][e] = l;
    }
  __syncthreads();  // every warp is done with its ring
  constexpr int H = 8 * NT;  // tile columns: index map * kCols + column
  float* sm_m = reinterpret_cast<float*>(smem);
  float* sm_l = sm_m + C::kWarps * H;
  float* sm_o = sm_l + C::kWarps * H;  // 16-byte aligned: kWarps * H is a multiple of 4
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int h = nt * 8 + 2 * cq + e;
      if (gq == 0) {
        sm_m[warp * H + h] = m_run[nt][e];
        sm_l[warp * H + h] = l_run[nt][e];
      }
      float* dst = sm_o + (warp * H + h) * (2 * D);
#pragma unroll
      for (int dt = 0; dt < C::kMT; ++dt) {
        dst[dt * 16 + gq] = o[nt][dt][e];
        dst[dt * 16 + gq + 8] = o[nt][dt][2 + e];
      }
    }
  if (__syncthreads_or(failed_at >= 0)) return no_result();

  constexpr int kV = 2 * D / 32;  // dims per lane
  for (int cc = warp; cc < my_cols; cc += C::kWarps) {
    const int c = col0 + cc;
    const int64_t row = row0 + c / a.group;
    const int head = j * a.group + c % a.group;
    float y[2][kV];
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      const int h = m * C::kCols + cc;
      float M = -INFINITY;
#pragma unroll
      for (int w = 0; w < C::kWarps; ++w) M = fmaxf(M, sm_m[w * H + h]);
      const float base = M == -INFINITY ? 0.f : M;  // the row sees no key of this partition
      float wsum = 0.f;
#pragma unroll
      for (int i = 0; i < kV; ++i) y[m][i] = 0.f;
#pragma unroll
      for (int w = 0; w < C::kWarps; ++w) {
        const float f = exp2f(sm_m[w * H + h] - base);
        wsum += f * sm_l[w * H + h];
#pragma unroll
        for (int i = 0; i < kV; ++i) y[m][i] += f * sm_o[(w * H + h) * (2 * D) + lane * kV + i];
      }
      const float inv = wsum > 0.f ? 1.f / wsum : 0.f;
#pragma unroll
      for (int i = 0; i < kV; ++i) y[m][i] *= inv;
      if (nparts > 1) {
        const int64_t pi = cell(cc, m);
        float* dst = a.part_o + pi * (2 * D) + lane * kV;
#pragma unroll
        for (int i = 0; i < kV; i += 4)
          *reinterpret_cast<float4*>(dst + i) =
              make_float4(y[m][i], y[m][i + 1], y[m][i + 2], y[m][i + 3]);
        if (lane == 0) {
          a.part_m[pi] = M;
          a.part_l[pi] = wsum;
        }
      }
    }
    if (nparts == 1) {
      const float lam = __ldg(a.lam + row * a.lam_stride + head);
      float z[kV];
#pragma unroll
      for (int i = 0; i < kV; ++i) z[i] = y[0][i] - lam * y[1][i];
      finish_head<D, BF>(a, z, row, head, lane);
    }
  }
}

// Joins n partials (m in log2 units, l, O / l) of one map of one row; a lane holds kV dims.  False
// when one of them says that it has no result (l < 0).  The first kBatch partials' sums are loaded
// with all the m and l, before any of them is used.
template <int kV>
__device__ __forceinline__ bool join(const float* po, const float* pm, const float* pl, int n,
                                     int lane, float (&y)[kV]) {
  constexpr int kBatch = 8;
  float4 x[kBatch][kV / 4];
  auto load = [&](int p0) {
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      if (p0 + i < n) {
        const float* src = po + static_cast<int64_t>(p0 + i) * (32 * kV) + lane * kV;
#pragma unroll
        for (int c = 0; c < kV / 4; ++c) x[i][c] = reinterpret_cast<const float4*>(src)[c];
      }
  };
  float mh = lane < n ? pm[lane] : -INFINITY, lh = lane < n ? pl[lane] : 0.f;  // partial `lane`
  load(0);
  float M = mh;
  bool lost = lh < 0.f;
  for (int p = lane + 32; p < n; p += 32) {
    M = fmaxf(M, pm[p]);
    lost |= pl[p] < 0.f;
  }
  if (__any_sync(0xffffffffu, lost)) return false;
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
  const float wh = exp2f(mh - M) * lh;
  float wsum = 0.f;
#pragma unroll
  for (int i = 0; i < kV; ++i) y[i] = 0.f;
  for (int p0 = 0; p0 < n; p0 += kBatch) {
    if (p0 > 0) load(p0);
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int p = p0 + i;  // the same for every lane
      if (p >= n) break;
      const float w = p < 32 ? __shfl_sync(0xffffffffu, wh, p) : exp2f(pm[p] - M) * pl[p];
      wsum += w;
#pragma unroll
      for (int c = 0; c < kV / 4; ++c) {
        y[4 * c] += w * x[i][c].x;
        y[4 * c + 1] += w * x[i][c].y;
        y[4 * c + 2] += w * x[i][c].z;
        y[4 * c + 3] += w * x[i][c].w;
      }
    }
  }
  const float inv = 1.f / wsum;
#pragma unroll
  for (int i = 0; i < kV; ++i) y[i] *= inv;
  return true;
}

// Two warps per (query row, differential head), one per map: the second map's hands its result
// over through shared memory, the first one's subtracts and finishes.  All threads of the block
// call it; `any`: this warp has a row.  c: the row's first partial of this warp's map.
template <int D, bool BF>
__device__ __forceinline__ void join_maps(const DiffArgs& a, bool any, const float* po,
                                          const float* pm, const float* pl, int64_t c, int n,
                                          int64_t row, int head) {
  constexpr int kV = 2 * D / 32;
  __shared__ float other[2][2 * D];
  __shared__ int lost[2];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, slot = warp >> 1, map = warp & 1;
  float y[kV];
  const bool ok = any && join<kV>(po + c * (2 * D), pm + c, pl + c, n, lane, y);
  if (map == 1) {
    if (ok) {
#pragma unroll
      for (int i = 0; i < kV; ++i) other[slot][i * 32 + lane] = y[i];
    }
    if (lane == 0) lost[slot] = !ok;
  }
  __syncthreads();
  if (map == 0 && ok && !lost[slot]) {
    const float lam = __ldg(a.lam + row * a.lam_stride + head);
#pragma unroll
    for (int i = 0; i < kV; ++i) y[i] -= lam * other[slot][i * 32 + lane];
    finish_head<D, BF>(a, y, row, head, lane);
  }
}

// Joins the rows kernel's partitions of both maps: two heads a block.
template <int D, bool BF>
__global__ void __launch_bounds__(128) diff_merge_kernel(const DiffArgs a) {
  grid_launch_dependents();
  const int s = blockIdx.y, qi = blockIdx.z;
  const int map = (threadIdx.x >> 5) & 1;
  const int head = blockIdx.x * 2 + (threadIdx.x >> 6);
  const int row0 = a.query_start_loc[s], row1 = a.query_start_loc[s + 1];
  const int L = a.seq_lens[s], q_len = row1 - row0;
  const int nparts = (L + a.part_tokens - 1) / a.part_tokens;
  const bool any = head < a.num_q_heads / 2 && q_len >= 1 && q_len <= a.verify_rows &&
                   qi < q_len && row0 >= 0 && row1 <= a.num_tokens && L >= q_len && nparts > 1 &&
                   nparts <= a.max_parts && (L + a.block_size - 1) / a.block_size <= a.max_blocks;
  grid_dependency_wait();
  const int64_t c = ((static_cast<int64_t>(s) * a.verify_rows + qi) * a.num_q_heads + 2 * head +
                     map) * a.max_parts;
  join_maps<D, BF>(a, any, a.part_o, a.part_m, a.part_l, c, nparts, row0 + qi, head);
}

// The same for the chunk kernel's partials: grid y = rank of the chunk's sequence, as in the chunk
// kernel, x over its (row, head)s.
template <int D, bool BF>
__global__ void __launch_bounds__(128) diff_chunk_merge_kernel(const DiffArgs a) {
  __shared__ ChunkScan<128> scan;
  __shared__ int keys[128];
  find_chunk(a, scan, keys, blockIdx.y, false);
  if (scan.s < 0) return;
  const int map = (threadIdx.x >> 5) & 1, heads = a.num_q_heads / 2;
  const int row0 = scan.row0, q_len = scan.q_len, L = scan.L;
  if (q_len > L || (L + a.block_size - 1) / a.block_size > a.max_blocks || row0 < 0 ||
      row0 + q_len > a.num_tokens || q_len > a.max_query_len || L > a.max_seq_len)
    return;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 2 + (threadIdx.x >> 6);
  const bool any = i < static_cast<int64_t>(q_len) * heads;
  const int ctx = L - q_len, tile_q = 128 / a.group;
  const int qi = any ? static_cast<int>(i / heads) : 0, head = static_cast<int>(i % heads);
  const int kend = ctx + min(q_len, (qi / tile_q + 1) * tile_q);
  const int tiles = (kend + kChunkKeys - 1) / kChunkKeys;
  const int per = (tiles + a.key_splits - 1) / a.key_splits;
  const int n = (tiles + per - 1) / per;  // ranges that hold keys
  const int64_t row = row0 + qi;
  const int64_t c = (row * a.num_q_heads + 2 * head + map) * a.key_splits;
  join_maps<D, BF>(a, any, a.chunk_o, a.chunk_m, a.chunk_l, c, n, row, head);
}

template <int D, int BS, int NT, bool BF>
cudaError_t launch_rows_t(const DiffArgs& a, const CUtensorMap& kmap, const CUtensorMap& vmap,
                          cudaStream_t stream) {
  using C = RowsCfg<D, NT>;
  auto kern = diff_rows_kernel<D, BS, NT, BF>;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = once_per_device(done, [&] {
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                C::smem_bytes(C::kMaxStages));
  });
  if (e != cudaSuccess) return e;
  DiffArgs b = a;
  b.col_groups = (a.verify_rows * a.group + C::kCols - 1) / C::kCols;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.max_parts) * b.col_groups, a.num_pairs, a.num_seqs);
  // Rings: what the SM's shared memory gives the CTAs that it holds.
  const int64_t ctas = static_cast<int64_t>(cfg.gridDim.x) * a.num_pairs * a.num_seqs;
  b.stages = ctas <= kSms ? 6 : ctas <= 2 * kSms ? 3 : 2;
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = C::smem_bytes(b.stages);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, kmap, vmap, b);
}

template <int D, int BS, bool BF>
cudaError_t launch_rows_g(const DiffArgs& a, const CUtensorMap& k, const CUtensorMap& v,
                          cudaStream_t st) {
  return a.verify_rows * a.group <= 4 ? launch_rows_t<D, BS, 1, BF>(a, k, v, st)
                                      : launch_rows_t<D, BS, 2, BF>(a, k, v, st);
}

template <int D, int BS>
cudaError_t launch_rows_b(const DiffArgs& a, const CUtensorMap& k, const CUtensorMap& v,
                          cudaStream_t st) {
  return a.bf16 ? launch_rows_g<D, BS, true>(a, k, v, st) : launch_rows_g<D, BS, false>(a, k, v, st);
}

}  // namespace

cudaError_t launch_diff_rows(const DiffArgs& a, const CUtensorMap& kmap, const CUtensorMap& vmap,
                             cudaStream_t stream) {
  if (a.head_dim == 128)
    return a.block_size == 16 ? launch_rows_b<128, 16>(a, kmap, vmap, stream)
                              : launch_rows_b<128, 32>(a, kmap, vmap, stream);
  return a.block_size == 16 ? launch_rows_b<64, 16>(a, kmap, vmap, stream)
                            : launch_rows_b<64, 32>(a, kmap, vmap, stream);
}

cudaError_t launch_diff_merge(const DiffArgs& a, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((a.num_q_heads / 2 + 1) / 2, a.num_seqs, a.verify_rows);
  cfg.blockDim = dim3(128);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (a.bf16)
    return a.head_dim == 128 ? cudaLaunchKernelEx(&cfg, diff_merge_kernel<128, true>, a)
                             : cudaLaunchKernelEx(&cfg, diff_merge_kernel<64, true>, a);
  return a.head_dim == 128 ? cudaLaunchKernelEx(&cfg, diff_merge_kernel<128, false>, a)
                           : cudaLaunchKernelEx(&cfg, diff_merge_kernel<64, false>, a);
}

cudaError_t launch_diff_chunk_merge(const DiffArgs& a, cudaStream_t stream) {
  const int64_t work = std::min<int64_t>(a.max_query_len, a.num_tokens) * (a.num_q_heads / 2);
  if ((work + 1) / 2 > INT32_MAX) return cudaErrorInvalidConfiguration;
  const dim3 grid(static_cast<unsigned>((work + 1) / 2), a.prefill_seqs);
  if (a.bf16)
    a.head_dim == 128 ? diff_chunk_merge_kernel<128, true><<<grid, 128, 0, stream>>>(a)
                      : diff_chunk_merge_kernel<64, true><<<grid, 128, 0, stream>>>(a);
  else
    a.head_dim == 128 ? diff_chunk_merge_kernel<128, false><<<grid, 128, 0, stream>>>(a)
                      : diff_chunk_merge_kernel<64, false><<<grid, 128, 0, stream>>>(a);
  return cudaGetLastError();
}

namespace {

// How a call is split, from its host-side facts alone, and the workspace that takes.
struct DiffPlan {
  bool chunks;       // sequences with several rows go to the chunk kernel
  bool rows;         // some sequences may go to the rows kernel
  int rows_per_seq;  // the rows kernel's most rows of a sequence
  int prefill_seqs;
  int part_tokens, parts, key_splits;
  size_t o, m, l, co, cm, cl, total;  // offsets of the regions
};

DiffPlan diff_plan(int64_t t, int64_t n, int64_t hq, int64_t hkv, int64_t d,
                   const pa_batch_hint& hint) {
  DiffPlan p{};
  const int64_t group = hq / hkv;
  // Short chunks (speculative verify, ends of prompts) go to the rows kernel too: always up to 8
  // columns (one group, which reads the keys once), and beyond while its grid of 256-key partitions
  // is small.  The chunk kernel takes 12 to 16 us for the smallest chunk.  One chunk of 16 rows
  // behind 1000 keys (32 + 8 heads of 128): rows 12.4, chunk 18.2 us; 32 rows 21.0 / 25.6; 64 rows
  // 34.2 / 25.6; heads of 64: 32 rows 13.9 / 25.0, 64 rows 21.2 / 25.2, 128 rows 25.8 / 25.8.
  const int64_t columns = hint.max_query_len * group;
  const int64_t units = n * (hkv / 2) * ((columns + 7) / 8) * ((hint.max_seq_len + int64_t{255}) / 256);
  const bool verify = columns <= 8 || units <= (d == 64 ? 4 : 2) * kSms;
  p.chunks = hint.max_query_len > 1 && !verify;
  p.rows = !(p.chunks && hint.num_prefill_seqs >= n);
  p.rows_per_seq = p.chunks ? 1 : hint.max_query_len;
  p.prefill_seqs = static_cast<int>(
      hint.num_prefill_seqs > 0 ? std::min<int64_t>(hint.num_prefill_seqs, n) : n);
  // Partitions of 128 to 1024 keys: the shortest with which the grid is at most two CTAs an SM, and
  // 512 where it is more than six even with 1024 (ragged lengths then even out).  Decode steps of
  // 32 + 8 heads of 128 in us, with partitions of 128 / 256 / 512 / 1024: 1 sequence of 4096 keys
  // 10.5 / 11.3 / 15.2 / 24.8; 4 of them 22.1 / 16.6 / 18.0 / 25.8; 8: 32.3 / 31.4 / 25.8 / 27.9;
  // 16: 52.1 / 49.4 / 51.1 / 45.8; 64 of 512 .. 4096 keys 107 / 96.5 / 94.6 / 97.2.
  const int64_t row_cols = p.rows_per_seq * group, per_cta = row_cols <= 4 ? 4 : 8;
  const int64_t row_ctas = n * (hkv / 2) * ((row_cols + per_cta - 1) / per_cta);
  auto parts_of = [&](int64_t tokens) { return (hint.max_seq_len + tokens - 1) / tokens; };
  p.part_tokens = 128;
  while (p.part_tokens < 1024 && row_ctas * parts_of(p.part_tokens) > 2 * kSms)
    p.part_tokens *= 2;
  if (row_ctas * parts_of(1024) > 6 * kSms) p.part_tokens = 512;
  p.parts = static_cast<int>(std::max<int64_t>(1, parts_of(p.part_tokens)));
  // Chunks too few to fill the SMs share out their keys too, 512 at least each, joined by the
  // merge kernel: a chunk of 32 rows behind 4000 keys (32 + 8 heads of 128) 52 -> 25 us, one of 10
  // rows (heads of 64) 62 -> 20 us.
  p.key_splits = 1;
  if (p.chunks) {
    const int64_t tile_q = 128 / group;
    const int64_t rows = std::min<int64_t>(hint.max_query_len, t);
    const int64_t ctas = (rows + tile_q - 1) / tile_q * (hkv / 2) * p.prefill_seqs *
                         (d == 128 ? 2 : 1);
    p.key_splits = static_cast<int>(
        std::max<int64_t>(1, std::min<int64_t>({kSms / ctas, parts_of(512), 32})));
  }
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  auto region = [&](size_t bytes) {
    const size_t at = p.total;
    p.total += up(bytes);
    return at;
  };
  if (p.rows && p.parts > 1) {
    const size_t cells = static_cast<size_t>(n) * p.rows_per_seq * hq * p.parts;
    p.o = region(cells * 2 * d * sizeof(float));
    p.m = region(cells * sizeof(float));
    p.l = region(cells * sizeof(float));
  }
  if (p.chunks && p.key_splits > 1) {
    const size_t cells = static_cast<size_t>(t) * hq * p.key_splits;
    p.co = region(cells * 2 * d * sizeof(float));
    p.cm = region(cells * sizeof(float));
    p.cl = region(cells * sizeof(float));
  }
  return p;
}

}  // namespace
}  // namespace pa

extern "C" {

size_t pa_diff_attention_workspace_size(int64_t num_tokens, int64_t num_seqs, int64_t num_q_heads,
                                        int64_t num_kv_heads, int64_t head_dim,
                                        const pa_batch_hint* hint) {
  if (!hint || num_tokens <= 0 || num_seqs <= 0 || num_kv_heads < 2 || num_kv_heads % 2 != 0 ||
      num_q_heads < num_kv_heads || num_q_heads % num_kv_heads != 0 ||
      num_q_heads / num_kv_heads > 16 || head_dim <= 0 || hint->max_query_len <= 0 ||
      hint->max_seq_len < 0)
    return 0;  // nothing to do, or refused by the call itself
  return pa::diff_plan(num_tokens, num_seqs, num_q_heads, num_kv_heads, head_dim, *hint).total;
}

int pa_diff_attention(const pa_tensor* q, const pa_tensor* k_cache, const pa_tensor* v_cache,
                      const pa_tensor* block_tables, const pa_tensor* seq_lens,
                      const pa_tensor* query_start_loc, float scale, const pa_diff* diff,
                      const pa_tensor* out, const pa_batch_hint* hint, void* workspace,
                      size_t workspace_bytes, void* stream) {
  using namespace pa;
  clear_last_error();
  int rc;
  if (k_cache && k_cache->dtype == PA_F8E4M3)
    return fail(PA_ERR_UNSUPPORTED, "differential attention over an FP8 pool is not built");
  const int dt = pool_dtype16(k_cache);
  if ((rc = check_pool(k_cache, v_cache, dt))) return rc;
  if ((rc = check_tensor(q, "q", dt, 3))) return rc;
  if ((rc = check_tensor(out, "out", dt, 3))) return rc;
  if ((rc = check_tensor(block_tables, "block_tables", PA_I32, 2))) return rc;
  if ((rc = check_tensor(seq_lens, "seq_lens", PA_I32, 1))) return rc;
  if ((rc = check_tensor(query_start_loc, "query_start_loc", PA_I32, 1))) return rc;
  if (!hint) return fail(PA_ERR_INVALID_ARG, "hint is NULL");
  if (!diff) return fail(PA_ERR_INVALID_ARG, "diff is NULL");
  const int64_t t = q->shape[0], hq = q->shape[1], d = q->shape[2];
  const int64_t hkv = k_cache->shape[1], n = seq_lens->shape[0];
  if (d != k_cache->shape[3]) return fail(PA_ERR_INVALID_ARG, "q head_dim differs from the pool's");
  if (hkv % 2 != 0 || hkv < 2)
    return fail(PA_ERR_INVALID_ARG, "num_kv_heads must be even: heads 2j and 2j + 1 are a pair");
  if (hq < 1 || hq % hkv != 0)
    return fail(PA_ERR_INVALID_ARG, "num_q_heads must be a positive multiple of num_kv_heads");
  const int64_t group = hq / hkv;
  if (group > 16) return fail(PA_ERR_UNSUPPORTED, "GQA group size above 16 not built");
  if (out->shape[0] != t || out->shape[1] != hq / 2 || out->shape[2] != 2 * d)
    return fail(PA_ERR_INVALID_ARG, "out must be [T, num_q_heads / 2, 2 * head_dim]");
  if ((rc = check_contiguous(out, "out"))) return rc;
  if (t > 0 && (q->stride[1] != d || (t > 1 && (q->stride[0] < hq * d || q->stride[0] % 8 != 0)) ||
                !aligned16(q->data) || !aligned16(out->data)))
    return fail(PA_ERR_INVALID_ARG,
                "q needs head stride head_dim, token stride >= heads*head_dim and a multiple of 8; "
                "q and out need 16-byte alignment");
  if (query_start_loc->shape[0] != n + 1)
    return fail(PA_ERR_INVALID_ARG, "query_start_loc must have num_seqs + 1 entries");
  if (block_tables->shape[0] != n)
    return fail(PA_ERR_INVALID_ARG, "block_tables must have num_seqs rows");
  if (n > 65535) return fail(PA_ERR_UNSUPPORTED, "more than 65535 sequences in one call");
  if (block_tables->shape[1] < 1 && n > 0)
    return fail(PA_ERR_INVALID_ARG, "block_tables needs at least one column");
  if (block_tables->shape[1] > INT32_MAX ||
      (n > 1 && block_tables->stride[0] < block_tables->shape[1]))
    return fail(PA_ERR_INVALID_ARG, "block_tables row stride must cover its columns");
  if (hint->max_query_len < 0 || hint->max_seq_len < 0 || hint->num_prefill_seqs < 0)
    return fail(PA_ERR_INVALID_ARG, "hint values must be non-negative");
  if (hint->shared_prefix_tokens != 0)
    return fail(PA_ERR_UNSUPPORTED, "differential attention has no shared-prefix pass");
  if (hint->max_query_len > hint->max_seq_len)
    return fail(PA_ERR_INVALID_ARG, "hint max_query_len exceeds max_seq_len");
  if (!(scale - scale == 0.f)) return fail(PA_ERR_INVALID_ARG, "scale must be finite");
  // lambda: one value per differential head, or per token and differential head
  const pa_tensor* lam = diff->lambda;
  if ((rc = check_tensor(lam, "lambda", PA_F32, lam && lam->ndim == 2 ? 2 : 1))) return rc;
  if (lam->shape[lam->ndim - 1] != hq / 2 || (lam->ndim == 2 && lam->shape[0] != t))
    return fail(PA_ERR_INVALID_ARG, "lambda must be [num_q_heads / 2] or [T, num_q_heads / 2]");
  const pa_tensor* w = diff->norm_weight;
  if (w) {
    if ((rc = check_tensor(w, "norm_weight", PA_F32, 1))) return rc;
    if (w->shape[0] != 2 * d || !aligned16(w->data))
      return fail(PA_ERR_INVALID_ARG,
                  "norm_weight must have 2 * head_dim values and 16-byte alignment");
    if (!(diff->eps >= 0.f && diff->eps < INFINITY))
      return fail(PA_ERR_INVALID_ARG, "eps must be finite and >= 0");
  }
  if (!(diff->out_scale - diff->out_scale == 0.f))
    return fail(PA_ERR_INVALID_ARG, "out_scale must be finite");

  if (t == 0 || n == 0 || hint->max_query_len == 0) return PA_OK;
  const DiffPlan plan = diff_plan(t, n, hq, hkv, d, *hint);
  if (plan.total > 0) {
    if (!workspace || workspace_bytes < plan.total)
      return fail(PA_ERR_WORKSPACE, "workspace needs " + std::to_string(plan.total) + " bytes");
    if (reinterpret_cast<uintptr_t>(workspace) & 255u)
      return fail(PA_ERR_WORKSPACE, "workspace must be 256-byte aligned");
  }

  DiffArgs a{};
  a.q = static_cast<const __half*>(q->data);
  a.q_stride = q->stride[0];
  a.out = static_cast<__half*>(out->data);
  a.block_tables = static_cast<const int32_t*>(block_tables->data);
  a.bt_stride = block_tables->stride[0];
  a.seq_lens = static_cast<const int32_t*>(seq_lens->data);
  a.query_start_loc = static_cast<const int32_t*>(query_start_loc->data);
  uint8_t* wsb = static_cast<uint8_t*>(workspace);
  a.part_o = reinterpret_cast<float*>(wsb + plan.o);
  a.part_m = reinterpret_cast<float*>(wsb + plan.m);
  a.part_l = reinterpret_cast<float*>(wsb + plan.l);
  a.chunk_o = reinterpret_cast<float*>(wsb + plan.co);
  a.chunk_m = reinterpret_cast<float*>(wsb + plan.cm);
  a.chunk_l = reinterpret_cast<float*>(wsb + plan.cl);
  a.num_seqs = static_cast<int>(n);
  a.num_tokens = t;
  a.num_q_heads = static_cast<int>(hq);
  a.num_kv_heads = static_cast<int>(hkv);
  a.num_pairs = static_cast<int>(hkv / 2);
  a.group = static_cast<int>(group);
  a.group_inv = 65536 / a.group + 1;
  a.head_dim = static_cast<int>(d);
  a.block_size = static_cast<int>(k_cache->shape[2]);
  a.max_blocks = static_cast<int>(block_tables->shape[1]);
  a.num_blocks = k_cache->shape[0];
  a.part_tokens = plan.part_tokens;
  a.max_parts = plan.parts;
  a.max_query_len = hint->max_query_len;
  a.max_seq_len = hint->max_seq_len;
  a.verify_rows = plan.rows_per_seq;
  a.prefill_seqs = plan.chunks ? plan.prefill_seqs : 0;
  a.decode_skipped = plan.rows ? 0 : 1;
  a.key_splits = plan.key_splits;
  a.scale_log2 = scale * 1.4426950408889634f;
  a.v_scale = 1.f;
  a.bf16 = dt == PA_BF16 ? 1 : 0;
  a.lam = static_cast<const float*>(lam->data);
  a.lam_stride = lam->ndim == 2 ? lam->stride[0] : 0;
  a.norm_w = w ? static_cast<const float*>(w->data) : nullptr;
  a.eps = diff->eps;
  a.out_scale = diff->out_scale;
  a.wait_limit_ns = wait_limit_ns();
  cudaError_t e = error_word(stream, &a.err);
  if (e != cudaSuccess) return cuda_fail(e, "error word");
  const int64_t rows = k_cache->shape[0] * hkv * k_cache->shape[2];
  const int64_t tiles = k_cache->shape[0] * hkv;
  // kmap: one head's 16 rows a box; kpair, vpair: both heads of a pair
  CUtensorMap kmap{}, kpair{}, vpair{};
  const int bs = a.block_size, di = a.head_dim;
  if (plan.chunks && (rc = make_pool_map(&kmap, k_cache->data, rows, di, dt))) return rc;
  if (plan.rows && (rc = make_pair_map(&kpair, k_cache->data, tiles, bs, di, dt))) return rc;
  if ((rc = make_pair_map(&vpair, v_cache->data, tiles, bs, di, dt))) return rc;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  auto chunks = [&](cudaStream_t on) -> int {
    cudaError_t ce = launch_diff_chunk(a, kmap, vpair, on);
    if (ce != cudaSuccess) return cuda_fail(ce, "diff chunk launch");
    if (a.key_splits > 1) ce = launch_diff_chunk_merge(a, on);
    return ce == cudaSuccess ? PA_OK : cuda_fail(ce, "diff chunk merge launch");
  };
  if (!plan.rows) return chunks(st);
  // Chunks beside rows: the chunks go first, on the side stream, joined back on every path.
  struct Join {
    SideStream* side = nullptr;
    cudaStream_t st = nullptr;
    cudaError_t done() {
      if (!side) return cudaSuccess;
      cudaError_t je = cudaEventRecord(side->join, side->stream);
      if (je == cudaSuccess) je = cudaStreamWaitEvent(st, side->join, 0);
      side = nullptr;
      return je;
    }
    ~Join() { done(); }
  } join;
  if (plan.chunks) {
    SideStream* side = nullptr;
    if ((e = side_stream(&side)) != cudaSuccess) return cuda_fail(e, "side stream");
    if ((e = cudaEventRecord(side->fork, st)) != cudaSuccess ||
        (e = cudaStreamWaitEvent(side->stream, side->fork, 0)) != cudaSuccess)
      return cuda_fail(e, "stream fork");
    join.side = side;
    join.st = st;
    if ((rc = chunks(side->stream))) return rc;
  }
  if ((e = launch_diff_rows(a, kpair, vpair, st)) != cudaSuccess) return cuda_fail(e, "diff launch");
  if (a.max_parts > 1 && (e = launch_diff_merge(a, st)) != cudaSuccess)
    return cuda_fail(e, "diff merge launch");
  if ((e = join.done()) != cudaSuccess) return cuda_fail(e, "stream join");
  return PA_OK;
}

}  // extern "C"
