// Differential attention of query chunks on the 5th-generation tensor cores (the mathematics is
// in pa_diff.cu).
//
// Work item = one CTA = (Q tile, softmax map, kv-head pair, sequence, range of the keys).  A Q
// tile is 128 rows, each a (query token, head of the pair's group) pair.  A map's result is 2d
// wide: with d = 128 its accumulator takes 256 of TMEM's 512 columns and two 128 x 128 score
// buffers the rest, so a CTA holds one map; the two maps of a row are two CTAs.  (Both maps in
// one CTA with half of V's width each would fit too, but every score and exponential would be
// computed twice: 8 tile products instead of 6 per 128 keys and row tile.)
//
// 640 threads:
//   * warps 16, 17 stream 128-key tiles of K (one head) and V (two heads, 2d columns) through the
//     block table into rings of 128-byte-swizzled tiles;
//   * lane 0 of warp 18 issues the MMAs: S(j) = Q K_j^T (M 128, N 128, K d) into buffer j % 2 and
//     O += P(j) V_j (M 128, N 2d, K 128), P(j) read from TMEM where it overwrote S(j).  Order:
//     S(0), S(1), then P(j) V_j, S(j + 2): the pipe computes one tile's products while the
//     other buffer's tile is in softmax;
//   * warps 0 .. 15 are the softmax: group j % 2 (256 threads) takes key tile j, a thread per
//     (row, half of the tile's columns).  O has one base m per row for both groups, raised only
//     when a tile's maximum passes it by more than 2^8 (then O is rescaled in TMEM, after the
//     P V before): a function of the tiles' maxima alone, so a group needs only the other
//     group's maxima of the tile before, known before that group's exponentials, and the two
//     groups' exponentials overlap.
// The sum l is of the rounded weights that the P V product uses: the rounding of a weight then
// cancels in part (measured against float64: 1.37 instead of 1.53 times the output's own
// rounding).
// Every wait is bounded; V rows past the last visible key are zeroed before their product.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "pa_chunk.cuh"
#include "pa_common.cuh"
#include "pa_diff.h"

namespace pa {
namespace {

template <int D>
struct ChunkCfg {
  static constexpr int kRows = 128, kKeys = 128;
  static constexpr int kHalves = D / 64;
  static constexpr int kTileBytes = kHalves * kKeys * 128;  // 128 rows of one head
  static constexpr int kQBytes = kTileBytes, kKBytes = kTileBytes, kVBytes = 2 * kTileBytes;
  static constexpr int kKStages = D == 128 ? 2 : 4, kVStages = D == 128 ? 2 : 4;
  static constexpr int kSmemBytes = kQBytes + kKStages * kKBytes + kVStages * kVBytes + 1024;
  static constexpr int kSoftmax = 512, kGroup = 256;
  static constexpr int kThreads = kSoftmax + 128;
  // launched at 96 registers a thread; the producer warpgroup falls to 64, softmax takes 104
  static constexpr int kRegsSoftmax = 104, kRegsOther = 64, kLaunchRegs = 96;
  static constexpr uint32_t kTmemCols = 512, kOCol = 256;
  static constexpr float kRescaleLog2 = 8.f;
  static_assert(kSmemBytes + 2048 <= 232448, "dynamic + static shared memory fit one SM");
  static_assert(kRegsSoftmax * kSoftmax + kRegsOther * 128 <= kLaunchRegs * kThreads,
                "register split exceeds the launch allocation");
};

// The sum of the two values that a packed pair holds, per lane of a packed float32 pair.
template <bool BF>
__device__ __forceinline__ uint64_t widen2(uint32_t pk) {
  if constexpr (BF) {
    return f32x2(__uint_as_float(pk << 16), __uint_as_float(pk & 0xffff0000u));
  } else {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&pk));
    return f32x2(f.x, f.y);
  }
}

// x rounded up to a float32 whose low 8 bits are 0 (NaN cannot occur: maxima ignore it).
__device__ __forceinline__ uint32_t round_up24(float x) {
  const uint32_t u = __float_as_uint(x);
  if (u & 0x80000000u) return u & 0xffffff00u;  // toward zero is up
  return u >= 0x7f800000u ? u : (u + 0xffu) & 0xffffff00u;
}

template <int D, int BS, bool BF>
__global__ void __launch_bounds__(ChunkCfg<D>::kThreads, 1)
    diff_chunk_kernel(const __grid_constant__ CUtensorMap kmap,
                      const __grid_constant__ CUtensorMap vmap, const DiffArgs a) {
  using C = ChunkCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t k_full[C::kKStages], k_empty[C::kKStages];
  __shared__ __align__(8) uint64_t v_full[C::kVStages], v_empty[C::kVStages];
  __shared__ __align__(8) uint64_t s_full[2], p_full[2], handed[2][4], pv_done, q_full, drain;
  __shared__ uint32_t tmem_base;
  __shared__ int warp_count[C::kThreads / 32];
  __shared__ int chosen_seq, softmax_stop;
  // [group][half][row]: maximum of the group's latest tile over each half of its columns, in the
  // scores' own unit, rounded up to the upper 24 bits of its float32 (what shared memory is left)
  __shared__ uint16_t max_hi[2][2][C::kRows];
  __shared__ uint8_t max_lo[2][2][C::kRows];

  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t q_s = smem_addr(smem);
  const uint32_t k_s = q_s + C::kQBytes;
  const uint32_t v_s = k_s + C::kKStages * C::kKBytes;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  const int map = blockIdx.x & 1, pair = blockIdx.y;
  const int nsplit = a.key_splits;
  const int split = blockIdx.z % nsplit, z = blockIdx.z / nsplit;
  const int nq = gridDim.x / 2;
  const int qt = nq - 1 - static_cast<int>(blockIdx.x) / 2;  // later tiles see more keys: first
  const int s = find_prefill_seq<C::kThreads>(a, warp_count, &chosen_seq, z,
                                              blockIdx.x == 0 && pair == 0 && blockIdx.z == 0);
  if (s < 0) return;
  const int tile_q = C::kRows / a.group;  // query tokens per tile
  const int row0 = a.query_start_loc[s];
  const int q_len = a.query_start_loc[s + 1] - row0;
  const int L = a.seq_lens[s];
  const bool lead = blockIdx.x == 0 && split == 0;
  if (q_len > L || (L + BS - 1) / BS > a.max_blocks || row0 < 0 || row0 + q_len > a.num_tokens) {
    if (lead && tid == 0) atomicOr(a.err, kErrDescriptor);
    return;
  }
  if (q_len > a.max_query_len || L > a.max_seq_len) {
    if (lead && tid == 0) atomicOr(a.err, kErrHint);
    return;
  }
  const int qbase = qt * tile_q;
  if (qbase >= q_len) return;
  const int ctx = L - q_len;
  const int kend = ctx + min(q_len, qbase + tile_q);  // keys [0, kend) are visible to some row
  const int all_tiles = (kend + C::kKeys - 1) / C::kKeys;
  const int per = (all_tiles + nsplit - 1) / nsplit;
  const int tile_first = split * per;
  const int ntiles = min(all_tiles - tile_first, per);
  if (ntiles <= 0) return;
  const int key_base = tile_first * C::kKeys;
  const int key_stop = min(kend, key_base + ntiles * C::kKeys);

  int bad = 0;
  for (int i = key_base / BS + tid; i < (key_stop + BS - 1) / BS; i += C::kThreads) {
    const int32_t blk = a.block_tables[static_cast<int64_t>(s) * a.bt_stride + i];
    if (blk < 0 || blk >= a.num_blocks) bad = 1;
  }
  // A tile without a result says so in its cells (l = -1), and the merge leaves such rows.
  auto no_result = [&](int row) {
    if (row < tile_q * a.group && qbase + row / a.group < q_len)
      a.chunk_l[(static_cast<int64_t>(row0 + qbase + row / a.group) * a.num_q_heads +
                 2 * (pair * a.group + row % a.group) + map) * nsplit + split] = -1.f;
  };
  if (__syncthreads_or(bad)) {
    if (tid == 0) atomicOr(a.err, kErrBlockRange);
    if (tid < C::kRows) no_result(tid);
    return;
  }

  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_addr(&tmem_base)),
                 "r"(C::kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (tid == 0) {
    for (int i = 0; i < C::kKStages; ++i) {
      mbar_init(smem_addr(&k_full[i]), 1);
      mbar_init(smem_addr(&k_empty[i]), 1);
    }
    for (int i = 0; i < C::kVStages; ++i) {
      mbar_init(smem_addr(&v_full[i]), 1);
      mbar_init(smem_addr(&v_empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_addr(&s_full[i]), 1);
      mbar_init(smem_addr(&p_full[i]), C::kGroup);
      for (int k = 0; k < 4; ++k) mbar_init(smem_addr(&handed[i][k]), 64);
    }
    mbar_init(smem_addr(&pv_done), 1);
    mbar_init(smem_addr(&q_full), C::kSoftmax);
    mbar_init(smem_addr(&drain), 1);
    mbar_init_fence();
    softmax_stop = 0;
  }
  tmem_fence_before_sync();
  __syncthreads();
  tmem_fence_after_sync();
  const uint32_t tmem = tmem_base;

  constexpr int kKWarp = C::kSoftmax / 32, kVWarp = kKWarp + 1, kMmaWarp = kKWarp + 2;
  if (warp >= kKWarp) {
    // ================================================ producer / MMA warpgroup
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kRegsOther));
    if (warp == kKWarp || warp == kVWarp) {
      const bool is_v = warp == kVWarp;
      const CUtensorMap* tm = is_v ? &vmap : &kmap;
      const int stages = is_v ? C::kVStages : C::kKStages, heads = is_v ? 2 : 1;
      const int stage_bytes = is_v ? C::kVBytes : C::kKBytes;
      const int head0 = 2 * pair + (is_v ? 0 : map);
      uint64_t* full = is_v ? v_full : k_full;
      uint64_t* empty = is_v ? v_empty : k_empty;
      const uint32_t ring = is_v ? v_s : k_s;
      // lane u fetches unit u (16 keys) of a tile; its block id is read a tile ahead
      auto units_of = [&](int j) {
        return min(C::kKeys / 16, (key_stop - (key_base + j * C::kKeys) + 15) >> 4);
      };
      auto block_of = [&](int j) {
        return lane < units_of(j) ? a.block_tables[static_cast<int64_t>(s) * a.bt_stride +
                                                   (key_base + j * C::kKeys + 16 * lane) / BS]
                                  : 0;
      };
      int issued = 0, next = block_of(0);
      for (int j = 0; j < ntiles; ++j) {
        const int st = j % stages, round = j / stages, blk = next;
        if (j + 1 < ntiles) next = block_of(j + 1);
        bool ok = true;
        if (lane == 0 && round > 0)
          ok = mbar_wait(smem_addr(&empty[st]), (round - 1) & 1, a.err, a.wait_limit_ns);
        if (!__shfl_sync(0xffffffffu, ok ? 1 : 0, 0)) break;
        const int units = units_of(j);
        const uint32_t bar = smem_addr(&full[st]);
        if (lane == 0) mbar_arrive_expect_tx(bar, units * heads * C::kHalves * 2048);
        __syncwarp();
        if (lane < units) {
          const int y = (blk * a.num_kv_heads + head0) * BS + (key_base + 16 * lane) % BS;
          const uint32_t dst = ring + st * stage_bytes + lane * 2048;
          for (int h = 0; h < heads; ++h)
#pragma unroll
            for (int c = 0; c < C::kHalves; ++c)
              tma_load_2d(dst + (h * C::kHalves + c) * (C::kKeys * 128), tm, c * 64, y + h * BS,
                          bar);
        }
        issued = j + 1;
      }
      if (lane == 0)  // no copy lands after the CTA retires
        for (int j = max(0, issued - stages); j < issued; ++j)
          mbar_wait(smem_addr(&full[j % stages]), (j / stages) & 1, a.err, a.wait_limit_ns);
    } else if (warp == kMmaWarp && lane == 0) {
      constexpr uint32_t kIdS = umma_idesc_f16(C::kRows, C::kKeys, 0, 0, BF);
      constexpr uint32_t kIdO = umma_idesc_f16(C::kRows, 2 * D, 0, 1, BF);
      auto issue_s = [&](int j) {
        const int st = j % C::kKStages;
        if (!mbar_wait(smem_addr(&k_full[st]), (j / C::kKStages) & 1, a.err, a.wait_limit_ns))
          return false;
        tmem_fence_after_sync();
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint32_t off = (k >> 2) * (C::kKeys * 128) + (k & 3) * 32;
          umma_f16(tmem + (j & 1) * 128, umma_sdesc(q_s + off, 16, 1024),
                   umma_sdesc(k_s + st * C::kKBytes + off, 16, 1024), kIdS, k > 0);
        }
        umma_commit(smem_addr(&s_full[j & 1]));
        umma_commit(smem_addr(&k_empty[st]));
        return true;
      };
      bool ok = mbar_wait(smem_addr(&q_full), 0, a.err, a.wait_limit_ns) && issue_s(0) &&
                (ntiles < 2 || issue_s(1));
      for (int j = 0; ok && j < ntiles; ++j) {
        const int vst = j % C::kVStages;
        ok = mbar_wait(smem_addr(&p_full[j & 1]), (j >> 1) & 1, a.err, a.wait_limit_ns) &&
             mbar_wait(smem_addr(&v_full[vst]), (j / C::kVStages) & 1, a.err, a.wait_limit_ns);
        if (!ok) break;
        tmem_fence_after_sync();
        const uint32_t vb = v_s + vst * C::kVBytes;
#pragma unroll
        for (int k = 0; k < C::kKeys / 16; ++k)
          umma_f16_tmem_a(tmem + C::kOCol, tmem + (j & 1) * 128 + k * 8,
                          umma_sdesc(vb + k * 16 * 128, C::kKeys * 128, 1024), kIdO,
                          (j > 0 || k > 0));
        umma_commit(smem_addr(&v_empty[vst]));
        umma_commit(smem_addr(&pv_done));
        if (j + 2 < ntiles) ok = issue_s(j + 2);
      }
      umma_commit(smem_addr(&drain));
      mbar_wait(smem_addr(&drain), 0, a.err, a.wait_limit_ns);
    }
  } else {
    // ================================================ softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kRegsSoftmax));
    constexpr int kHalfKeys = C::kKeys / 2;
    const int g = warp >> 3, h = (warp >> 2) & 1, quarter = warp & 3;
    const int r = quarter * 32 + lane;  // TMEM lane = row of the tile
    const uint32_t pair_bar = 1 + g * 4 + quarter;
    const int qi = r / a.group, hg = r % a.group;
    const int tok = qbase + qi;
    const bool rv = qi < tile_q && tok < q_len;
    const int pos = ctx + (rv ? tok : qbase);  // padding rows mirror the tile's first row
    const int head = pair * a.group + hg;      // differential head
    const uint32_t lane_addr = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t sbuf = tmem + lane_addr + g * 128;
    const uint32_t obuf = tmem + lane_addr + C::kOCol;

    {  // a quarter of the Q row -> shared memory, 128B-swizzled K-major
      const __half* qrow = a.q + static_cast<int64_t>(row0 + (rv ? tok : 0)) * a.q_stride +
                           static_cast<int64_t>(2 * head + map) * D;
#pragma unroll
      for (int cc = 0; cc < D / 32; ++cc) {
        const int c = (g * 2 + h) * (D / 32) + cc;
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (rv) v = __ldg(reinterpret_cast<const uint4*>(qrow + c * 8));
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                         q_s + (c >> 3) * (C::kRows * 128) + swz128(r, c & 7)),
                     "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
                     : "memory");
      }
      fence_proxy_async();
      mbar_arrive(smem_addr(&q_full));
    }

    bool stopped = false;
    float m_run = -INFINITY, l_run = 0.f;  // m in the scores' unit
    const int min_pos = ctx + qbase;
    const bool prescale = !(a.scale_log2 > 0.f);
    const float mul = prescale ? 1.f : a.scale_log2;  // exponent = fma(score, mul, -m mul)
    for (int j = g; j < ntiles; j += 2) {
      const bool got = __all_sync(
          0xffffffffu, mbar_wait(smem_addr(&s_full[g]), (j >> 1) & 1, a.err, a.wait_limit_ns));
      uint32_t sv[2][32];
      float mloc = -INFINITY;
      const int key0 = key_base + j * C::kKeys + h * kHalfKeys;
      if (got) {
        tmem_fence_after_sync();
        tmem_ld32(sbuf + h * kHalfKeys, sv[0]);
        tmem_ld32(sbuf + h * kHalfKeys + 32, sv[1]);
        tmem_wait_ld();
        tmem_regs_ready(sv[0]);
        tmem_regs_ready(sv[1]);
        const bool masked = key0 + kHalfKeys - 1 > min_pos;
        if (prescale || masked) {
#pragma unroll
          for (int c = 0; c < kHalfKeys; ++c) {
            float v = __uint_as_float(sv[c >> 5][c & 31]);
            if (prescale) v *= a.scale_log2;
            if (masked && key0 + c > pos) v = -INFINITY;
            sv[c >> 5][c & 31] = __float_as_uint(v);
          }
        }
        float m2[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int c = 0; c < kHalfKeys; c += 2)
          m2[(c >> 1) & 1] = fmax3(m2[(c >> 1) & 1], __uint_as_float(sv[c >> 5][c & 31]),
                                   __uint_as_float(sv[c >> 5][(c & 31) + 1]));
        mloc = fmaxf(m2[0], m2[1]);
      }
      // The other group's maxima of tile j - 1 (its threads wait for this read, through `handed`,
      // before they store those of tile j + 1).
      auto row_max = [&](int gg) {
        auto at = [&](int hh) {
          return __uint_as_float(static_cast<uint32_t>(max_hi[gg][hh][r]) << 16 |
                                 static_cast<uint32_t>(max_lo[gg][hh][r]) << 8);
        };
        return fmaxf(at(0), at(1));
      };
      float before = -INFINITY;
      if (j > 0) {
        if (!__all_sync(0xffffffffu, mbar_wait(smem_addr(&handed[g ^ 1][quarter]),
                                               ((j - 1) >> 1) & 1, a.err, a.wait_limit_ns)))
          stopped = true;  // nothing more is written; the pair leaves together below
        before = row_max(g ^ 1);
      }
      const uint32_t up = round_up24(mloc);
      max_hi[g][h][r] = static_cast<uint16_t>(up >> 16);
      max_lo[g][h][r] = static_cast<uint8_t>(up >> 8);
      // Both halves read the same stored maxima, so they take the same base; and both have read
      // their scores before either stores P over them.
      tmem_fence_before_sync();
      if (bar_sync_or(pair_bar, 64, !got || stopped)) {
        stopped = true;
        break;
      }
      tmem_fence_after_sync();
      const float mx = row_max(g);
      mbar_arrive(smem_addr(&handed[g][quarter]));
      // The base is a function of the maxima so far, so every thread of the row computes the same
      // one: after tile j - 1 (the other group's), then after tile j.
      auto raises = [&](float m, float x) {
        return (x - m) * mul > C::kRescaleLog2 || (m == -INFINITY && x > -INFINITY);
      };
      const float m_prev = j > 0 && raises(m_run, before) ? before : m_run;
      float m_new = m_prev, alpha = 1.f;
      if (raises(m_prev, mx)) {
        alpha = ex2_approx((m_prev - mx) * mul);  // 0 when m_prev is -inf
        m_new = mx;
      }
      if (j > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
        // rare: O so far, its last product done, goes over to the new base
        if (!__all_sync(0xffffffffu, mbar_wait(smem_addr(&pv_done), (j - 1) & 1, a.err,
                                               a.wait_limit_ns)))
          stopped = true;
        tmem_fence_after_sync();
#pragma unroll
        for (int c0 = 0; c0 < D; c0 += 16) {
          uint32_t t[16];
          tmem_ld16(obuf + h * D + c0, t);
          tmem_wait_ld();
          tmem_regs_ready(t);
#pragma unroll
          for (int c = 0; c < 16; ++c) t[c] = __float_as_uint(__uint_as_float(t[c]) * alpha);
          tmem_st16(obuf + h * D + c0, t);
        }
      }
      // this thread's sum is still against its group's base of two tiles ago
      if (m_new != m_run) l_run *= ex2_approx((m_run - m_new) * mul);
      m_run = m_new;

      const float neg_m = m_run == -INFINITY ? 0.f : -m_run * mul;
      const uint64_t mul2 = f32x2(mul, mul), negm2 = f32x2(neg_m, neg_m);
      uint64_t ps2[2] = {f32x2(0.f, 0.f), f32x2(0.f, 0.f)};
#pragma unroll
      for (int q8 = 0; q8 < kHalfKeys / 16; ++q8) {
        uint32_t pk[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const int k = q8 * 16 + 2 * c;
          float x0, x1;
          f32x2_split(ffma2(f32x2(__uint_as_float(sv[k >> 5][k & 31]),
                                  __uint_as_float(sv[k >> 5][(k & 31) + 1])),
                            mul2, negm2),
                      x0, x1);
          pk[c] = pack2<BF>(ex2_approx(x0), ex2_approx(x1));
          ps2[c & 1] = fadd2(ps2[c & 1], widen2<BF>(pk[c]));
        }
        tmem_st8(sbuf + h * (kHalfKeys / 2) + q8 * 8, pk);
      }
      float s0, s1, s2, s3;
      f32x2_split(ps2[0], s0, s1);
      f32x2_split(ps2[1], s2, s3);
      l_run += (s0 + s1) + (s2 + s3);

      const int tile0 = key_base + j * C::kKeys;
      if (j == ntiles - 1 && tile0 + C::kKeys > key_stop) {
        // V rows past the last visible key may hold any bits: the thread of (row, half) clears
        // that row of V head h once the tile has landed
        const int vst = j % C::kVStages;
        const bool landed =
            mbar_wait(smem_addr(&v_full[vst]), (j / C::kVStages) & 1, a.err, a.wait_limit_ns);
        if (landed && tile0 + r >= key_stop) {
          const uint32_t vrow = v_s + vst * C::kVBytes + h * C::kTileBytes + r * 128;
#pragma unroll
          for (int c = 0; c < C::kHalves * 8; ++c)
            asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(
                             vrow + (c >> 3) * (C::kKeys * 128) + (c & 7) * 16),
                         "r"(0u)
                         : "memory");
        }
        fence_proxy_async();
        if (!landed) stopped = true;
      }
      tmem_wait_st();
      tmem_fence_before_sync();
      // a thread that gave up hands over nothing; its pair leaves at the next tile's meeting
      if (!stopped) mbar_arrive(smem_addr(&p_full[g]));
    }

    // ---- join the four (group, half) sums of each row; every softmax thread meets here
    bool ok = !stopped;
    if (ok) ok = mbar_wait(smem_addr(&drain), 0, a.err, a.wait_limit_ns);
    float* red = reinterpret_cast<float*>(smem);  // Q and the rings are done once drained
    if (!ok) softmax_stop = 1;
    asm volatile("bar.sync 9, %0;" ::"n"(C::kSoftmax) : "memory");
    ok = !*reinterpret_cast<volatile int*>(&softmax_stop);
    if (ok) {
      red[(g * 2 + h) * C::kRows + r] = l_run;
      if (h == 0) red[(4 + g) * C::kRows + r] = m_run;
    }
    asm volatile("bar.sync 9, %0;" ::"n"(C::kSoftmax) : "memory");
    if (!ok) {
      if (g == 0 && h == 0) no_result(r);
    } else {
      tmem_fence_after_sync();
      const float m0 = red[4 * C::kRows + r], m1 = ntiles > 1 ? red[5 * C::kRows + r] : -INFINITY;
      const float m = fmaxf(m0, m1), base = m == -INFINITY ? 0.f : m;
      const float l = (red[r] + red[C::kRows + r]) * ex2_approx((m0 - base) * mul) +
                      (red[2 * C::kRows + r] + red[3 * C::kRows + r]) * ex2_approx((m1 - base) * mul);
      const float inv = l > 0.f ? 1.f / l : 0.f;
      const int64_t cell =
          (static_cast<int64_t>(row0 + tok) * a.num_q_heads + 2 * head + map) * nsplit + split;
      if (rv && g == 0 && h == 0) {
        a.chunk_m[cell] = m * mul;
        a.chunk_l[cell] = l;
      }
      constexpr int kCols = 2 * D / 4;  // output columns of this thread
      const int col0 = (g * 2 + h) * kCols;
#pragma unroll
      for (int c0 = 0; c0 < kCols; c0 += 16) {
        uint32_t t[16];
        tmem_ld16(obuf + col0 + c0, t);
        tmem_wait_ld();
        tmem_regs_ready(t);
        if (rv) {
#pragma unroll
          for (int c = 0; c < 16; c += 4)
            *reinterpret_cast<float4*>(a.chunk_o + cell * (2 * D) + col0 + c0 + c) =
                make_float4(__uint_as_float(t[c]) * inv, __uint_as_float(t[c + 1]) * inv,
                            __uint_as_float(t[c + 2]) * inv, __uint_as_float(t[c + 3]) * inv);
        }
      }
    }
  }

  tmem_fence_before_sync();
  __syncthreads();
  tmem_fence_after_sync();
  if (warp == 0)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                 "r"(C::kTmemCols)
                 : "memory");
}

template <int D, int BS, bool BF>
cudaError_t launch_t(const DiffArgs& a, const CUtensorMap& kmap, const CUtensorMap& vmap,
                     cudaStream_t stream) {
  using C = ChunkCfg<D>;
  auto kern = diff_chunk_kernel<D, BS, BF>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       C::kSmemBytes);
  if (e != cudaSuccess) return e;
  // setmaxnreg.inc takes registers the CTA was launched with: never launch a build below the split
  cudaFuncAttributes attr{};
  if ((e = cudaFuncGetAttributes(&attr, kern)) != cudaSuccess) return e;
  if (attr.numRegs * C::kThreads < C::kRegsSoftmax * C::kSoftmax + C::kRegsOther * 128 ||
      attr.numRegs * C::kThreads > 65536)
    return cudaErrorInvalidConfiguration;
  const int tile_q = C::kRows / a.group;
  const dim3 grid(2 * ((a.max_query_len + tile_q - 1) / tile_q), a.num_pairs,
                  a.prefill_seqs * a.key_splits);
  kern<<<grid, C::kThreads, C::kSmemBytes, stream>>>(kmap, vmap, a);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_d(const DiffArgs& a, const CUtensorMap& k, const CUtensorMap& v,
                     cudaStream_t st) {
  if (a.block_size == 16)
    return a.bf16 ? launch_t<D, 16, true>(a, k, v, st) : launch_t<D, 16, false>(a, k, v, st);
  return a.bf16 ? launch_t<D, 32, true>(a, k, v, st) : launch_t<D, 32, false>(a, k, v, st);
}

}  // namespace

cudaError_t launch_diff_chunk(const DiffArgs& a, const CUtensorMap& kmap, const CUtensorMap& vmap,
                              cudaStream_t stream) {
  return a.head_dim == 128 ? launch_d<128>(a, kmap, vmap, stream)
                           : launch_d<64>(a, kmap, vmap, stream);
}

}  // namespace pa
