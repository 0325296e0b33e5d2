// Differential attention of query chunks on the 5th-generation tensor cores (the mathematics is
// in pa_diff.cu).
//
// A Q tile is 128 rows, each a (query token, head of the kv-head pair's group) pair; key tiles are
// 128 keys.  Per softmax map and key tile: S = Q K^T (M 128, N 128, K d), P = 2^(S - m) in the
// element type, O += P V (M 128, N 2d, K 128), with S, P and O in TMEM (512 columns).
//   * d = 64 (diff_chunk_both_kernel): a CTA holds both maps: two score buffers, two 128-column
//     accumulators.  V is loaded once for both, and the CTA finishes its rows alone.
//   * d = 128 (diff_chunk_map_kernel): one map's accumulator takes 256 columns and its two score
//     buffers the rest, so a CTA holds one map and a cluster of two CTAs a Q tile; at the end
//     each CTA copies half of its rows' sums into the other's shared memory and finishes the
//     other 64 rows.  (Both maps in one CTA with half of V's width each would fit too, but
//     every score and exponential would be computed twice: 8 tile products instead of 6.)
//
// 640 threads in both:
//   * warps 16, 17 stream K and V tiles through the block table into rings of 128-byte-swizzled
//     tiles;
//   * lane 0 of warp 18 issues the MMAs, P read from TMEM where it overwrote S: the pipe computes
//     one score buffer's products while the other buffer is in softmax;
//   * warps 0 .. 15 are the softmax: all of them take every score buffer in turn, a thread per
//     (row, quarter of the tile's columns), while the pipe works on the other buffer.  The base m
//     of a row is raised only when weights against it grow large (then O is rescaled in TMEM).
// Every wait is bounded; V rows past the last visible key are zeroed before their product.
//
// Bound by the tensor pipe and the softmax about it: a key tile takes 1.10 us a map at d = 128 and
// 1.35 us for both maps at d = 64 (its products alone, with the rests below, 1.17 us each at the
// measured rate of large matrix products); and by what surrounds the key loop, about 10 us a CTA
// (search 2, first loads and first tile 4, last products and end 5, overlapping little), in which
// the pipe idles, since an SM holds one CTA.  4 x 512 rows behind up to 7.5k keys (32 + 8 heads of
// 128): 182 us = 1200 TFLOP/s, 0.63 of the measured burst; a prompt of 4001 rows (32 + 8 heads of
// 64): 107 us.  At d = 128 the key loop's speed hangs on its spills: versions with 32 more bytes
// spilled took 5% longer.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "pa_common.cuh"
#include "pa_diff.cuh"
#include "pa_host.h"

namespace pa {
namespace {

// What both kernels share.  Registers: launched at 96 a thread; the producer warpgroup falls to 64
// and the softmax warps take 104.
struct ChunkCfg {
  static constexpr int kRows = 128, kKeys = 128;
  static constexpr int kSoftmax = 512, kThreads = kSoftmax + 128;
  static constexpr int kRegsSoftmax = 104, kRegsOther = 64, kLaunchRegs = 96;
  static constexpr uint32_t kTmemCols = 512, kOCol = 256;
  static_assert(kRegsSoftmax * kSoftmax + kRegsOther * 128 <= kLaunchRegs * kThreads,
                "register split exceeds the launch allocation");
};

struct BothCfg : ChunkCfg {                       // d = 64
  static constexpr int kTileBytes = 128 * 128;    // 128 rows of one head
  static constexpr int kStageBytes = 2 * kTileBytes;  // K1 and K2, or the two halves of V
  static constexpr int kKStages = 2, kVStages = 3;
  static constexpr int kSmemBytes = 2 * kTileBytes + (kKStages + kVStages) * kStageBytes + 1024;
  static_assert(kSmemBytes + 4096 <= 232448, "dynamic + static shared memory fit one SM");
};

struct MapCfg : ChunkCfg {                        // d = 128
  static constexpr int kTileBytes = 2 * 128 * 128;  // 128 rows of one head
  static constexpr int kVBytes = 2 * kTileBytes;    // both heads
  static constexpr int kKStages = 2, kVStages = 2;
  static constexpr int kSmemBytes = kTileBytes + kKStages * kTileBytes + kVStages * kVBytes + 1024;
  static_assert(kSmemBytes + 2048 <= 232448, "dynamic + static shared memory fit one SM");
  static_assert(kVStages * kVBytes >= 64 * 2 * 128 * 4, "64 rows of the other map fit V's ring");
};

// One arrival for the whole warp, after every lane's accesses before it.
__device__ __forceinline__ void warp_arrive(uint32_t bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

// row / group and row % group of a tile row (0 .. 127, group 1 .. 16) by a multiplication: exact
// there for inv = 65536 / group + 1.
__device__ __forceinline__ int token_of(const DiffArgs& a, int row) {
  return (row * a.group_inv) >> 16;
}
__device__ __forceinline__ int head_of(const DiffArgs& a, int row) {
  return row - token_of(a, row) * a.group;
}

// The chunk tile of a CTA: its rows and keys.
struct Tile {
  int s, row0, q_len, ctx, qbase, tile_q;
  int kend;        // keys [0, kend) are visible to some row
  int key_base;    // this CTA's keys: [key_base, key_stop), in ntiles 128-key tiles
  int key_stop, ntiles;
};

// The CTA's place: grid x is (tile from the last on, kv-head pair), z (rank of the chunk, key range).
struct Place {
  int pair, back, z, split;
};
__device__ __forceinline__ Place place_of(const DiffArgs& a, unsigned x) {
  Place p;
  p.back = static_cast<int>(a.num_pairs > 1 ? __umulhi(x, a.pairs_inv) : x);
  p.pair = static_cast<int>(x) - p.back * a.num_pairs;
  p.z = blockIdx.z;
  p.split = 0;
  if (a.key_splits > 1) {
    p.split = p.z % a.key_splits;
    p.z /= a.key_splits;
  }
  return p;
}

// Finds and checks the tile; false when the CTA has none (errors are reported).  All threads of
// the block call it.  keys: 128 words that nothing uses yet (of Q's tile, which only generic
// stores fill).
template <int BS>
__device__ __forceinline__ bool find_tile(const DiffArgs& a, ChunkScan<ChunkCfg::kThreads>& sc,
                                          int* keys, const Place& at, Tile& t) {
  const bool lead = blockIdx.x == 0 && at.split == 0, first = blockIdx.x == 0 && blockIdx.z == 0;
  const int qt = a.chunk_tiles - 1 - at.back, split = at.split;
  const int tid = threadIdx.x;
  find_chunk(a, sc, keys, at.z, first);
  t.s = sc.s;
  if (t.s < 0) return false;
  t.tile_q = a.tile_q;
  t.row0 = sc.row0;
  t.q_len = sc.q_len;
  const int L = sc.L;
  if (t.q_len > L || (L + BS - 1) / BS > a.max_blocks || t.row0 < 0 ||
      t.row0 + t.q_len > a.num_tokens) {
    if (lead && tid == 0) atomicOr(a.err, kErrDescriptor);
    return false;
  }
  if (t.q_len > a.max_query_len || L > a.max_seq_len) {
    if (lead && tid == 0) atomicOr(a.err, kErrHint);
    return false;
  }
  t.qbase = qt * t.tile_q;
  if (t.qbase >= t.q_len) return false;
  t.ctx = L - t.q_len;
  t.kend = t.ctx + min(t.q_len, t.qbase + t.tile_q);
  const int all_tiles = (t.kend + 127) / 128;
  // (divisions cost a CTA's start 0.2 us each; so the host's inverses, and none for one range)
  const int per =
      a.key_splits > 1 ? (all_tiles + a.key_splits - 1) / a.key_splits : all_tiles;
  t.ntiles = min(all_tiles - split * per, per);
  if (t.ntiles <= 0) return false;
  t.key_base = split * per * 128;
  t.key_stop = min(t.kend, t.key_base + t.ntiles * 128);
  return true;
}

// A producer warp: streams 128-key tiles of `heads` heads from head0 on into a ring; lane u
// fetches unit u (16 keys), whose block id it reads a tile ahead.  K (kPairs false): one box per
// head and 64 columns, into [head][half][128 keys][128 B].  V (kPairs true): one box of both
// heads, into [unit][half][head][16 keys][128 B].  Before returning it waits for its last
// copies, so none lands after the CTA retires.  A block id outside the pool is reported, sets
// *stop (no row of the tile is written then) and block 0 is fetched in its place.
template <int D, int BS, bool kPairs>
__device__ __forceinline__ void stream_heads(const DiffArgs& a, const Tile& t,
                                             const CUtensorMap* tm, int head0, int heads,
                                             int stages, uint64_t* full, uint64_t* empty,
                                             uint32_t ring, int* stop) {
  constexpr int kHalves = D / 64, kPart = 128, kUnits = kPart / 16;
  const int lane = threadIdx.x & 31;
  const int pieces = (t.key_stop - t.key_base + kPart - 1) / kPart;
  const int stage_bytes = heads * kHalves * kPart * 128;
  auto units_of = [&](int j) {
    return min(kUnits, (t.key_stop - (t.key_base + j * kPart) + 15) >> 4);
  };
  auto block_of = [&](int j) {
    return lane < units_of(j) ? a.block_tables[static_cast<int64_t>(t.s) * a.bt_stride +
                                               (t.key_base + j * kPart + 16 * lane) / BS]
                              : 0;
  };
  int issued = 0, next = block_of(0);
  for (int j = 0; j < pieces; ++j) {
    const int st = j % stages, round = j / stages;
    int blk = next;
    if (blk < 0 || blk >= a.num_blocks) {
      atomicOr(a.err, kErrBlockRange);
      *reinterpret_cast<volatile int*>(stop) = 1;
      blk = 0;
    }
    if (j + 1 < pieces) next = block_of(j + 1);
    bool ok = true;
    if (lane == 0 && round > 0)
      ok = mbar_wait_short(smem_addr(&empty[st]), (round - 1) & 1, a.err, a.wait_limit_ns);
    if (!__shfl_sync(0xffffffffu, ok ? 1 : 0, 0)) break;
    const int units = units_of(j);
    const uint32_t bar = smem_addr(&full[st]);
    if (lane == 0) mbar_arrive_expect_tx(bar, units * heads * kHalves * 2048);
    __syncwarp();
    if (lane < units) {
      const int off = (t.key_base + j * kPart + 16 * lane) % BS;
      const uint32_t dst = ring + st * stage_bytes;
      if constexpr (kPairs) {
        tma_load_4d(dst + lane * (2 * kHalves * 2048), tm, 0, off, blk * a.num_kv_heads + head0, 0,
                    bar);
      } else {
        const int y = (blk * a.num_kv_heads + head0) * BS + off;
        for (int h = 0; h < heads; ++h)
#pragma unroll
          for (int c = 0; c < kHalves; ++c)
            tma_load_2d(dst + (h * kHalves + c) * (kPart * 128) + lane * 2048, tm, c * 64,
                        y + h * BS, bar);
      }
    }
    issued = j + 1;
  }
  if (lane == 0)
    for (int j = max(0, issued - stages); j < issued; ++j)
      mbar_wait_short(smem_addr(&full[j % stages]), (j / stages) & 1, a.err, a.wait_limit_ns);
}

// A thread's 32 scores from TMEM, scaled where the scale cannot go into the exponent, masked.
__device__ __forceinline__ void load_scores(uint32_t addr, uint32_t (&sv)[32], bool prescale,
                                            float scale_log2, bool masked, int key0, int pos) {
  tmem_ld32(addr, sv);
  tmem_wait_ld();
  tmem_regs_ready(sv);
  if (prescale || masked) {
#pragma unroll
    for (int c = 0; c < 32; ++c) {
      float v = __uint_as_float(sv[c]);
      if (prescale) v *= scale_log2;
      if (masked && key0 + c > pos) v = -INFINITY;
      sv[c] = __float_as_uint(v);
    }
  }
}

// Their weights 2^(score mul + neg_m), rounded to the element type for the matrix product (at most
// 2^-11 (fp16) or 2^-8 (bf16) of each weight, at random over the keys), two keys a word; returns
// the unrounded weights' sum.  (Summing the rounded weights instead changes the result's error by
// under 1%.)  What the rounding took off the first 8 goes into `rest` in the same form and through a
// product of its own: a quarter of the weights enter to twice the bits.  The result's error against
// 64 bits falls from 1.53 to 1.46 times that of the output's own rounding (bf16, 32 + 8 heads of
// 128; the maps' difference magnifies it), for 1.03 -> 1.10 us a tile at d = 128 and 1.21 -> 1.35 at
// d = 64; all of them would take twice the products of P and V.
template <bool BF>
__device__ __forceinline__ float weigh(const uint32_t (&sv)[32], uint32_t (&pk)[16],
                                       uint32_t (&rest)[4], float mul, float neg_m) {
  const uint64_t mul2 = f32x2(mul, mul), negm2 = f32x2(neg_m, neg_m);
  uint64_t ps2[2] = {f32x2(0.f, 0.f), f32x2(0.f, 0.f)};
#pragma unroll
  for (int k = 0; k < 32; k += 2) {
    float x0, x1;
    f32x2_split(ffma2(f32x2(__uint_as_float(sv[k]), __uint_as_float(sv[k + 1])), mul2, negm2), x0,
                x1);
    const float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
    ps2[(k >> 1) & 1] = fadd2(ps2[(k >> 1) & 1], f32x2(p0, p1));
    pk[k >> 1] = pack2<BF>(p0, p1);
    if (k < 8) {
      const float2 w = unpack2<BF>(pk[k >> 1]);
      rest[k >> 1] = pack2<BF>(p0 - w.x, p1 - w.y);
    }
  }
  float s0, s1, s2, s3;
  f32x2_split(ps2[0], s0, s1);
  f32x2_split(ps2[1], s2, s3);
  return (s0 + s1) + (s2 + s3);
}

// Columns [0, n) at `addr` of this thread's lane times f.
__device__ __forceinline__ void rescale(uint32_t addr, int n, float f) {
  for (int c0 = 0; c0 < n; c0 += 16) {
    uint32_t t[16];
    tmem_ld16(addr + c0, t);
    tmem_wait_ld();
    tmem_regs_ready(t);
#pragma unroll
    for (int c = 0; c < 16; ++c) t[c] = __float_as_uint(__uint_as_float(t[c]) * f);
    tmem_st16(addr + c0, t);
  }
}

// Clears 64 columns (`half`) of row r of head h of a V tile (a whole 128-byte row of it, so the
// swizzle does not matter).
template <int kHalves>
__device__ __forceinline__ void clear_v_row(uint32_t tile, int r, int half, int h) {
  const uint32_t row =
      tile + (r >> 4) * (2 * kHalves * 2048) + half * 4096 + h * 2048 + (r & 15) * 128;
#pragma unroll
  for (int c = 0; c < 8; ++c)
    asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(row + c * 16), "r"(0u)
                 : "memory");
}

// x rounded up to a float32 whose low 8 bits are 0 (NaN cannot occur: maxima ignore it).
__device__ __forceinline__ uint32_t round_up24(float x) {
  const uint32_t u = __float_as_uint(x);
  if (u & 0x80000000u) return u & 0xffffff00u;  // toward zero is up
  return u >= 0x7f800000u ? u : (u + 0xffu) & 0xffffff00u;
}

// Shared maxima of a tile: [column quarter][row], the upper 24 bits of a float32 rounded up, in
// two arrays (what shared memory the d = 128 kernel has left).
struct Maxima {
  uint16_t hi[4][ChunkCfg::kRows];
  uint8_t lo[4][ChunkCfg::kRows];
};

// One score buffer's softmax by the 512 threads: this thread's row r, columns 32 cq .. + 31 of S at
// sbuf (fresh: the first, for which there is no base).  The weights are taken against the row's base
// m so far.  Only where that does not do (no
// base yet, or a thread's 32 weights sum to more than 2^10, so one is above 2^5: they stay far below
// fp16's 2^16) are the maxima of the threads that want it exchanged, O brought to the new base by
// `rebase` and the weights taken again, from the scores still in TMEM; a row that does not want one
// keeps its base, so no row's result depends on the rows beside it.  So the usual tile computes no
// maximum, and the one meeting of the row's four threads only asks whether anyone wants a new base.
// P goes where the thread's own scores were: 16 columns from 32 cq on.  The rests of the first 8
// weights of quarters 0 and 1 stand together behind P of quarter 0, those of 2 and 3 behind quarter
// 2's.  False, for all four of a row's warps, when one of them had no scores (its wait gave up).
template <bool BF, typename Rebase>
__device__ __forceinline__ bool soften(uint32_t sbuf, bool got, Maxima& mx, int r, int cq,
                                       uint32_t meet_bar, bool prescale, float scale_log2,
                                       bool masked, int key0, int pos, float mul, bool fresh,
                                       float& m_run, float& l_run, Rebase rebase) {
  uint32_t pk[16], rest[4];
  float sum = 0.f;
  // Unrolled, so that the usual tile runs straight through (a 4001-row prompt 111 -> 105 us).
#pragma unroll 2
  for (int turn = 0; turn < 2; ++turn) {
    uint32_t sv[32];
    if (got && !(turn == 0 && fresh)) {
      tmem_fence_after_sync();
      load_scores(sbuf + 32 * cq, sv, prescale, scale_log2, masked, key0, pos);
      sum = weigh<BF>(sv, pk, rest, mul, m_run == -INFINITY ? 0.f : -m_run * mul);
    }
    const bool wants = m_run == -INFINITY || !(sum <= 1024.f);  // at first: everyone
    // (the second time: everyone's scores are read before anyone's rests are stored)
    if (!bar_sync_or(meet_bar, 128, turn == 0 && (!got || wants))) break;
    uint32_t up = 0x7fffff00u;  // NaN: this thread has given up (a maximum itself is never NaN)
    if (got) {
      tmem_fence_after_sync();
      load_scores(sbuf + 32 * cq, sv, prescale, scale_log2, masked, key0, pos);
      float top = -INFINITY;
#pragma unroll
      for (int c = 0; c < 32; ++c) top = fmaxf(top, __uint_as_float(sv[c]));
      up = round_up24(wants ? top : -INFINITY);
    }
    mx.hi[cq][r] = static_cast<uint16_t>(up >> 16);
    mx.lo[cq][r] = static_cast<uint8_t>(up >> 8);
    bar_sync_or(meet_bar, 128, false);
    float top = m_run;
    bool lost = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t hi = mx.hi[i][r];
      lost |= hi == 0x7fffu;
      top = fmaxf(top, __uint_as_float(hi << 16 | static_cast<uint32_t>(mx.lo[i][r]) << 8));
    }
    bar_sync_or(meet_bar, 128, false);  // the maxima are read before a later tile's are stored
    if (__any_sync(0xffffffffu, lost)) return false;
    if (__any_sync(0xffffffffu, top != m_run)) {
      const float alpha = top == m_run ? 1.f : ex2_approx((m_run - top) * mul);
      rebase(alpha);
      l_run *= alpha;  // alpha is 0, and l, when m_run is still -inf
      m_run = top;
    }
  }
  l_run += sum;
  tmem_st16(sbuf + 32 * cq, pk);
  tmem_st4(sbuf + 64 * (cq >> 1) + 16 + 4 * (cq & 1), rest);
  return true;
}

__device__ __forceinline__ void alloc_tmem(uint32_t* base, uint32_t cols) {  // one warp
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                   smem_addr(base)),
               "r"(cols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void free_tmem(uint32_t base, uint32_t cols) {  // the same warp
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(base), "r"(cols)
               : "memory");
}

// Four normalised partial sums.
__device__ __forceinline__ void store4(float* dst, const uint32_t (&t)[32], int c, float inv) {
  *reinterpret_cast<float4*>(dst) =
      make_float4(__uint_as_float(t[c]) * inv, __uint_as_float(t[c + 1]) * inv,
                  __uint_as_float(t[c + 2]) * inv, __uint_as_float(t[c + 3]) * inv);
}

// o1 - lambda o2, each step rounded on its own: equal maps cancel to 0 at lambda 1.
__device__ __forceinline__ float difference(float o1, float o2, float lam) {
  return __fsub_rn(o1, __fmul_rn(lam, o2));
}

// kCols consecutive columns of a row's y from col0 on -> out, the row's sum of squares known.
template <int D, bool BF, int kCols>
__device__ __forceinline__ void finish_columns(const DiffArgs& a, float (&y)[kCols], float sum,
                                               __half* out, int col0) {
  float f = a.out_scale;
  if (a.norm_w) {
    f *= rsqrtf(sum * (1.f / (2 * D)) + a.eps);
#pragma unroll
    for (int c = 0; c < kCols; c += 4) {
      const float4 w = __ldg(reinterpret_cast<const float4*>(a.norm_w + col0 + c));
      y[c] *= w.x;
      y[c + 1] *= w.y;
      y[c + 2] *= w.z;
      y[c + 3] *= w.w;
    }
  }
#pragma unroll
  for (int c = 0; c < kCols; c += 8)
    *reinterpret_cast<uint4*>(out + col0 + c) =
        make_uint4(pack2<BF>(y[c] * f, y[c + 1] * f), pack2<BF>(y[c + 2] * f, y[c + 3] * f),
                   pack2<BF>(y[c + 4] * f, y[c + 5] * f), pack2<BF>(y[c + 6] * f, y[c + 7] * f));
}

// All 512 softmax threads meet.
__device__ __forceinline__ void softmax_sync() { asm volatile("bar.sync 9, 512;" ::: "memory"); }

// All threads of both CTAs of the cluster meet; their shared-memory accesses before the arrival
// are visible after the wait.
__device__ __forceinline__ void cluster_arrive() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  __syncwarp();
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_sync() {
  cluster_arrive();
  cluster_wait();
}

// An arrival on another CTA's mbarrier, and the (bounded) wait for it there.
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t remote_bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(remote_bar)
               : "memory");
}
__device__ __forceinline__ bool mbar_wait_cluster(uint32_t bar, uint32_t parity, unsigned* err,
                                                  uint64_t limit_ns) {
  uint64_t t0 = 0;
  for (uint32_t it = 0; it < (1u << 28); ++it) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    if (ok) return true;
    if ((it & 63u) == 63u) {
      const uint64_t now = global_timer_ns();
      if (t0 == 0) t0 = now;
      if (now - t0 > limit_ns) break;
    }
  }
  atomicOr(err, kErrTimeout);
  return false;
}

// The address of `addr` (of this CTA's shared memory) in the CTA of cluster rank `rank`.
__device__ __forceinline__ uint32_t cluster_addr(uint32_t addr, int rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}

template <int BS, bool BF>
__global__ void __launch_bounds__(BothCfg::kThreads, 1)
    diff_chunk_both_kernel(const __grid_constant__ CUtensorMap kmap,
                           const __grid_constant__ CUtensorMap vmap, const DiffArgs a) {
  using C = BothCfg;
  constexpr int D = 64;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t k_full[C::kKStages], k_empty[C::kKStages];
  __shared__ __align__(8) uint64_t v_full[C::kVStages], v_empty[C::kVStages];
  __shared__ __align__(8) uint64_t s_full[2], p_full[2], q_full, drain;
  __shared__ uint32_t tmem_base;
  __shared__ ChunkScan<C::kThreads> scan;
  __shared__ int softmax_stop;
  __shared__ Maxima maxima[2];  // per map

  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t q_s = smem_addr(smem);  // both maps' Q tiles
  const uint32_t k_s = q_s + 2 * C::kTileBytes;
  const uint32_t v_s = k_s + C::kKStages * C::kStageBytes;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  const Place at = place_of(a, blockIdx.x);
  const int nsplit = a.key_splits, pair = at.pair, split = at.split;
  // Barriers and TMEM are set up while the search for the tile waits for its loads.
  if (warp == 0) alloc_tmem(&tmem_base, C::kTmemCols);
  if (tid == 32) {  // beside the warp that allocates
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
      mbar_init(smem_addr(&p_full[i]), C::kSoftmax / 32);
    }
    mbar_init(smem_addr(&q_full), C::kSoftmax / 32);
    mbar_init(smem_addr(&drain), 1);
    mbar_init_fence();
    softmax_stop = 0;
  }
  tmem_fence_before_sync();
  Tile tile;
  if (!find_tile<BS>(a, scan, reinterpret_cast<int*>(smem), at, tile)) {
    if (warp == 0) free_tmem(tmem_base, C::kTmemCols);
    return;
  }
  tmem_fence_after_sync();
  // the cell of a row's partial, when the keys are split
  auto cell = [&](int row, int map) {
    return (static_cast<int64_t>(tile.row0 + tile.qbase + token_of(a, row)) * a.num_q_heads +
            2 * (pair * a.group + head_of(a, row)) + map) * nsplit + split;
  };
  auto real_row = [&](int row) {
    return row < tile.tile_q * a.group && tile.qbase + token_of(a, row) < tile.q_len;
  };
  // A range without a result says so (l = -1), and the merge leaves such rows alone.
  auto no_result = [&](int row, int map) {
    if (nsplit > 1 && real_row(row)) a.chunk_l[cell(row, map)] = -1.f;
  };
  // This thread's share of Q: a quarter of each map's row.
  uint4 qv[2][D / 32];
  if (warp < C::kSoftmax / 32) {
    const int r = (warp & 3) * 32 + lane;
    const bool rv = real_row(r);
    const __half* qrow =
        a.q + static_cast<int64_t>(tile.row0 + tile.qbase + (rv ? token_of(a, r) : 0)) * a.q_stride +
        static_cast<int64_t>(2 * (pair * a.group + head_of(a, r))) * D + (warp >> 2) * (D / 4);
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int c = 0; c < D / 32; ++c)
        qv[t][c] = rv ? __ldg(reinterpret_cast<const uint4*>(qrow + t * D) + c)
                      : make_uint4(0u, 0u, 0u, 0u);
  }
  const uint32_t tmem = tmem_base;
  const int ntiles = tile.ntiles;

  constexpr int kKWarp = C::kSoftmax / 32, kVWarp = kKWarp + 1, kMmaWarp = kKWarp + 2;
  if (warp >= kKWarp) {
    // ================================================ producer / MMA warpgroup
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kRegsOther));
    if (warp == kKWarp) {
      stream_heads<D, BS, false>(a, tile, &kmap, 2 * pair, 2, C::kKStages, k_full, k_empty, k_s,
                                 &softmax_stop);
    } else if (warp == kVWarp) {
      stream_heads<D, BS, true>(a, tile, &vmap, 2 * pair, 2, C::kVStages, v_full, v_empty, v_s,
                                 &softmax_stop);
    } else if (warp == kMmaWarp) {
      const bool leader = elect_one();
      constexpr uint32_t kIdS = umma_idesc_f16(C::kRows, C::kKeys, 0, 0, BF);
      constexpr uint32_t kIdO = umma_idesc_f16(C::kRows, 2 * D, 0, 1, BF);
      // The pipe queues almost nothing, so a wait between two products idles it for the wait's own
      // latency even when the barrier is long complete.  So each barrier is tested while products
      // issued before are still running, and waited for only when that test failed.
      auto k_bar = [&](int j) { return smem_addr(&k_full[j % C::kKStages]); };
      auto v_bar = [&](int j) { return smem_addr(&v_full[j % C::kVStages]); };
      auto need = [&](bool seen, uint32_t bar, int phase) {
        const bool ok = seen || __all_sync(0xffffffffu, mbar_wait_short(bar, phase & 1, a.err,
                                                                        a.wait_limit_ns));
        tmem_fence_after_sync();
        return ok;
      };
      // S_t(j); tests P of the product to follow halfway
      bool p_seen = false, v_seen = false, k_seen = false;
      auto test = [&](uint32_t bar, int phase) {
        return __all_sync(0xffffffffu, mbar_test(bar, phase & 1)) != 0;
      };
      auto issue_s = [&](int t, int j, uint32_t next_p, int next_phase) {
        const uint32_t qb = q_s + t * C::kTileBytes;
        const uint32_t kb = k_s + (j % C::kKStages) * C::kStageBytes + t * C::kTileBytes;
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          if (k == D / 16 - 1 && next_phase >= 0) p_seen = test(next_p, next_phase);
          umma_f16_if(leader, tmem + t * 128, umma_sdesc(qb + k * 32, 16, 1024),
                   umma_sdesc(kb + k * 32, 16, 1024), kIdS, k > 0);
        }
        umma_commit_if(leader, smem_addr(&s_full[t]));
      };
      bool ok = need(false, smem_addr(&q_full), 0) && need(false, k_bar(0), 0);
      if (ok) {
        issue_s(0, 0, 0, -1);
        issue_s(1, 0, 0, -1);
        umma_commit_if(leader, smem_addr(&k_empty[0]));
      }
      for (int j = 0; ok && j < ntiles; ++j) {
        const int vst = j % C::kVStages;
        const uint32_t vb = v_s + vst * C::kStageBytes;
        const bool more = j + 1 < ntiles;
        ok = need(v_seen, v_bar(j), j / C::kVStages);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          ok = ok && need(p_seen, smem_addr(&p_full[t]), j);
          if (!ok) break;
          p_seen = false;
#pragma unroll
          for (int k = 0; k < C::kKeys / 16 + 2; ++k) {
            // the last two: the rests of 8 keys each of two quarters, 32 keys apart in V
            const int rest = k - C::kKeys / 16;
            if (k == 6 && more) {
              if (t == 0)
                k_seen = test(k_bar(j + 1), (j + 1) / C::kKStages & 1);
              else
                v_seen = test(v_bar(j + 1), (j + 1) / C::kVStages & 1);
            }
            umma_f16_tmem_a_if(leader, tmem + C::kOCol + t * 128,
                               tmem + t * 128 +
                                   (rest < 0 ? (k >> 1) * 32 + (k & 1) * 8 : rest * 64 + 16),
                               rest < 0 ? umma_sdesc(vb + k * 4096, 2048, 1024)
                                        : umma_sdesc(vb + rest * 4 * 4096, 2048, 2 * 4096),
                               kIdO, (j > 0 || k > 0));
          }
          if (t == 1) umma_commit_if(leader, smem_addr(&v_empty[vst]));
          if (more) {
            if (t == 0) ok = need(k_seen, k_bar(j + 1), (j + 1) / C::kKStages);
            if (ok) issue_s(t, j + 1, smem_addr(&p_full[t ^ 1]), t == 0 ? j : j + 1);
          }
        }
        if (ok && more) umma_commit_if(leader, smem_addr(&k_empty[(j + 1) % C::kKStages]));
      }
      umma_commit_if(leader, smem_addr(&drain));
      mbar_wait_short(smem_addr(&drain), 0, a.err, a.wait_limit_ns);
    }
  } else {
    // ================================================ softmax: both maps' tiles in turn
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kRegsSoftmax));
    const int cq = warp >> 2, quarter = warp & 3;
    const int r = quarter * 32 + lane;  // TMEM lane = row of the tile
    const bool rv = real_row(r);
    const int tok = tile.qbase + (rv ? token_of(a, r) : 0);
    const int head = pair * a.group + head_of(a, r);
    const int pos = tile.ctx + tok;  // padding rows mirror the tile's first row
    const uint32_t lane_addr = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t obuf = tmem + lane_addr + C::kOCol;

    // Q -> shared memory, 128B-swizzled K-major
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int c = 0; c < D / 32; ++c)
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                         q_s + t * C::kTileBytes + swz128(r, cq * (D / 32) + c)),
                     "r"(qv[t][c].x), "r"(qv[t][c].y), "r"(qv[t][c].z), "r"(qv[t][c].w)
                     : "memory");
    fence_proxy_async();
    warp_arrive(smem_addr(&q_full));

    bool stopped = false;
    float m_run[2] = {-INFINITY, -INFINITY}, l_run[2] = {0.f, 0.f};  // m in the scores' unit
    const bool prescale = !(a.scale_log2 > 0.f);
    const float mul = prescale ? 1.f : a.scale_log2;
    for (int j = 0; j < ntiles && !stopped; ++j) {
      const int key0 = tile.key_base + j * C::kKeys + cq * 32;
      const bool masked = key0 + 31 > tile.ctx + tile.qbase;
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        // S(j) of this map done; it was issued after P V of tile j - 1, so O is settled too
        const bool got = __all_sync(0xffffffffu, mbar_wait_short(smem_addr(&s_full[t]), j & 1,
                                                                 a.err, a.wait_limit_ns));
        auto rebase = [&](float alpha) {
          if (j > 0) rescale(obuf + t * 128 + cq * (D / 2), D / 2, alpha);
        };
        if (!soften<BF>(tmem + lane_addr + t * 128, got, maxima[t], r, cq, 1 + quarter, prescale,
                        a.scale_log2, masked, key0, pos, mul, j == 0,
                        m_run[t], l_run[t], rebase)) {
          stopped = true;  // the row's four warps leave together
          break;
        }
        const int tile0 = tile.key_base + j * C::kKeys;
        if (t == 0 && j == ntiles - 1 && tile0 + C::kKeys > tile.key_stop) {
          // V rows past the last visible key may hold any bits: they are cleared before the first
          // product of their tile, once it has landed (row r of head cq per thread)
          const int vst = j % C::kVStages;
          if (!mbar_wait_short(smem_addr(&v_full[vst]), (j / C::kVStages) & 1, a.err,
                               a.wait_limit_ns))
            softmax_stop = 1;  // no row is written
          else if (cq < 2 && tile0 + r >= tile.key_stop)
            clear_v_row<1>(v_s + vst * C::kStageBytes, r, 0, cq);
          fence_proxy_async();
        }
        tmem_wait_st();
        tmem_fence_before_sync();
        warp_arrive(smem_addr(&p_full[t]));
      }
    }

    // ---- the row's sums of both maps; every softmax thread meets here
    const int64_t row = tile.row0 + tok;
    const float lam = __ldg(a.lam + row * a.lam_stride + head);  // used after the waits below
    bool ok = !stopped;
    if (ok) ok = mbar_wait_short(smem_addr(&drain), 0, a.err, a.wait_limit_ns);
    float* red = reinterpret_cast<float*>(smem);  // Q and the rings are done once drained
    if (!ok) softmax_stop = 1;
    softmax_sync();
    ok = !*reinterpret_cast<volatile int*>(&softmax_stop);
    if (ok) {
      red[cq * C::kRows + r] = l_run[0];
      red[(4 + cq) * C::kRows + r] = l_run[1];
    }
    softmax_sync();
    if (!ok) {
      if (cq < 2) no_result(r, cq);
    } else {
      tmem_fence_after_sync();
      float inv[2];
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        const float* p = red + 4 * m * C::kRows + r;
        const float l = (p[0] + p[C::kRows]) + (p[2 * C::kRows] + p[3 * C::kRows]);
        inv[m] = l > 0.f ? 1.f / l : 0.f;  // 0: the row sees no key of this range
        if (nsplit > 1 && rv && cq == m) {
          a.chunk_m[cell(r, m)] = m_run[m] * mul;
          a.chunk_l[cell(r, m)] = l;
        }
      }
      constexpr int kCols = 2 * D / 4;  // this thread's columns of y
      const int col0 = cq * kCols;
      uint32_t o0[kCols], o1[kCols];
      tmem_ld32(obuf + col0, o0);
      tmem_ld32(obuf + 128 + col0, o1);
      tmem_wait_ld();
      tmem_regs_ready(o0);
      tmem_regs_ready(o1);
      if (nsplit > 1) {
        if (rv) {
#pragma unroll
          for (int c = 0; c < kCols; c += 4) {
            store4(a.chunk_o + cell(r, 0) * (2 * D) + col0 + c, o0, c, inv[0]);
            store4(a.chunk_o + cell(r, 1) * (2 * D) + col0 + c, o1, c, inv[1]);
          }
        }
      } else {
        float y[kCols], ss = 0.f;
#pragma unroll
        for (int c = 0; c < kCols; ++c) {
          y[c] = difference(__fmul_rn(__uint_as_float(o0[c]), inv[0]),
                            __fmul_rn(__uint_as_float(o1[c]), inv[1]), lam);
          ss += y[c] * y[c];
        }
        float* sq = red + 8 * C::kRows;
        sq[cq * C::kRows + r] = ss;
        softmax_sync();
        const float sum = (sq[r] + sq[C::kRows + r]) + (sq[2 * C::kRows + r] + sq[3 * C::kRows + r]);
        if (rv)
          finish_columns<D, BF, kCols>(a, y, sum,
                                       a.out + (row * (a.num_q_heads / 2) + head) * (2 * D), col0);
      }
    }
  }

  tmem_fence_before_sync();
  __syncthreads();
  tmem_fence_after_sync();
  if (warp == 0) free_tmem(tmem, C::kTmemCols);
}

// d = 128: the CTAs of a cluster are the two maps of one Q tile.
template <int BS, bool BF>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(MapCfg::kThreads, 1)
    diff_chunk_map_kernel(const __grid_constant__ CUtensorMap kmap,
                          const __grid_constant__ CUtensorMap vmap, const DiffArgs a) {
  using C = MapCfg;
  constexpr int D = 128;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t k_full[C::kKStages], k_empty[C::kKStages];
  __shared__ __align__(8) uint64_t v_full[C::kVStages], v_empty[C::kVStages];
  __shared__ __align__(8) uint64_t s_full[2], p_full[2], pv_done, q_full, drain;
  __shared__ uint32_t tmem_base;
  // the other CTA's rings may be written; the other map's rows have arrived
  __shared__ __align__(8) uint64_t peer_free, rows_in;
  __shared__ ChunkScan<C::kThreads> scan;
  __shared__ int softmax_stop;
  __shared__ Maxima maxima;

  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t q_s = smem_addr(smem);
  const uint32_t k_s = q_s + C::kTileBytes;
  const uint32_t v_s = k_s + C::kKStages * C::kTileBytes;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  const Place at = place_of(a, blockIdx.x >> 1);
  const int map = blockIdx.x & 1, nsplit = a.key_splits;  // map = cluster rank
  const int pair = at.pair, split = at.split;
  // Barriers and TMEM are set up while the search for the tile waits for its loads.
  if (warp == 0) alloc_tmem(&tmem_base, C::kTmemCols);
  if (tid == 32) {  // beside the warp that allocates
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
      mbar_init(smem_addr(&p_full[i]), C::kSoftmax / 32);
    }
    mbar_init(smem_addr(&pv_done), 1);
    mbar_init(smem_addr(&q_full), C::kSoftmax / 32);
    mbar_init(smem_addr(&drain), 1);
    mbar_init(smem_addr(&rows_in), 1);
    mbar_init(smem_addr(&peer_free), 1);
    mbar_init_fence();
    softmax_stop = 0;
  }
  tmem_fence_before_sync();
  Tile tile;
  // both CTAs of the cluster see the same tile: they leave early together or not at all
  if (!find_tile<BS>(a, scan, reinterpret_cast<int*>(smem), at, tile)) {
    if (warp == 0) free_tmem(tmem_base, C::kTmemCols);
    return;
  }
  tmem_fence_after_sync();
  cluster_arrive();  // this CTA's barriers are set up
  auto cell = [&](int row) {
    return (static_cast<int64_t>(tile.row0 + tile.qbase + token_of(a, row)) * a.num_q_heads +
            2 * (pair * a.group + head_of(a, row)) + map) * nsplit + split;
  };
  auto real_row = [&](int row) {
    return row < tile.tile_q * a.group && tile.qbase + token_of(a, row) < tile.q_len;
  };
  auto no_result = [&](int row) {
    if (nsplit > 1 && real_row(row)) a.chunk_l[cell(row)] = -1.f;
  };
  // This thread's share of Q: a quarter of a row.
  uint4 qv[D / 32];
  if (warp < C::kSoftmax / 32) {
    const int r = (warp & 3) * 32 + lane;
    const bool rv = real_row(r);
    const __half* qrow =
        a.q + static_cast<int64_t>(tile.row0 + tile.qbase + (rv ? token_of(a, r) : 0)) * a.q_stride +
        static_cast<int64_t>(2 * (pair * a.group + head_of(a, r)) + map) * D + (warp >> 2) * (D / 4);
#pragma unroll
    for (int c = 0; c < D / 32; ++c)
      qv[c] = rv ? __ldg(reinterpret_cast<const uint4*>(qrow) + c) : make_uint4(0u, 0u, 0u, 0u);
  }
  const uint32_t tmem = tmem_base;
  const int ntiles = tile.ntiles;

  constexpr int kKWarp = C::kSoftmax / 32, kVWarp = kKWarp + 1, kMmaWarp = kKWarp + 2;
  if (warp >= kKWarp) {
    // ================================================ producer / MMA warpgroup
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kRegsOther));
    if (warp == kKWarp) {
      stream_heads<D, BS, false>(a, tile, &kmap, 2 * pair + map, 1, C::kKStages, k_full, k_empty,
                                 k_s, &softmax_stop);
    } else if (warp == kVWarp) {
      stream_heads<D, BS, true>(a, tile, &vmap, 2 * pair, 2, C::kVStages, v_full, v_empty, v_s,
                                 &softmax_stop);
    } else if (warp == kMmaWarp) {
      const bool leader = elect_one();
      constexpr uint32_t kIdS = umma_idesc_f16(C::kRows, C::kKeys, 0, 0, BF);
      constexpr uint32_t kIdO = umma_idesc_f16(C::kRows, 2 * D, 0, 1, BF);
      // As in the other kernel: barriers are tested while products still run.
      auto k_bar = [&](int j) { return smem_addr(&k_full[j % C::kKStages]); };
      auto v_bar = [&](int j) { return smem_addr(&v_full[j % C::kVStages]); };
      auto need = [&](bool seen, uint32_t bar, int phase) {
        const bool ok = seen || __all_sync(0xffffffffu, mbar_wait_short(bar, phase & 1, a.err,
                                                                        a.wait_limit_ns));
        tmem_fence_after_sync();
        return ok;
      };
      bool p_seen = false, v_seen = false, k_seen = false;
      auto test = [&](uint32_t bar, int phase) {
        return __all_sync(0xffffffffu, mbar_test(bar, phase & 1)) != 0;
      };
      auto issue_s = [&](int j, bool look) {  // look: test V and P of tile j - 1, the products to follow
        const int st = j % C::kKStages;
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          if (k == 4 && look) v_seen = test(v_bar(j - 1), (j - 1) / C::kVStages & 1);
          if (k == 6 && look) p_seen = test(smem_addr(&p_full[(j - 1) & 1]), (j - 1) >> 1 & 1);
          const uint32_t off = (k >> 2) * (C::kKeys * 128) + (k & 3) * 32;
          umma_f16_if(leader, tmem + (j & 1) * 128, umma_sdesc(q_s + off, 16, 1024),
                   umma_sdesc(k_s + st * C::kTileBytes + off, 16, 1024), kIdS, k > 0);
        }
        umma_commit_if(leader, smem_addr(&s_full[j & 1]));
        umma_commit_if(leader, smem_addr(&k_empty[st]));
      };
      bool ok = need(false, smem_addr(&q_full), 0) && need(false, k_bar(0), 0);
      if (ok) issue_s(0, false);
      if (ok && ntiles > 1) {
        ok = need(false, k_bar(1), 1 / C::kKStages);
        if (ok) issue_s(1, false);
      }
      for (int j = 0; ok && j < ntiles; ++j) {
        const int vst = j % C::kVStages;
        const bool more = j + 2 < ntiles;
        ok = need(v_seen, v_bar(j), j / C::kVStages) &&
             need(p_seen, smem_addr(&p_full[j & 1]), j >> 1);
        if (!ok) break;
        v_seen = p_seen = false;
        const uint32_t vb = v_s + vst * C::kVBytes;
#pragma unroll
        for (int k = 0; k < C::kKeys / 16 + 2; ++k) {
          // the last two: the rests of 8 keys each of two quarters, 32 keys apart in V
          const int rest = k - C::kKeys / 16;
          if (k == 6 && more) k_seen = test(k_bar(j + 2), (j + 2) / C::kKStages & 1);
          umma_f16_tmem_a_if(leader, tmem + C::kOCol,
                             tmem + (j & 1) * 128 +
                                 (rest < 0 ? (k >> 1) * 32 + (k & 1) * 8 : rest * 64 + 16),
                             rest < 0 ? umma_sdesc(vb + k * 8192, 2048, 1024)
                                      : umma_sdesc(vb + rest * 4 * 8192, 2048, 2 * 8192),
                             kIdO, (j > 0 || k > 0));
        }
        umma_commit_if(leader, smem_addr(&v_empty[vst]));
        if (more) {
          ok = need(k_seen, k_bar(j + 2), (j + 2) / C::kKStages);
          if (ok) issue_s(j + 2, true);
        } else {
          umma_commit_if(leader, smem_addr(&pv_done));
        }
      }
      umma_commit_if(leader, smem_addr(&drain));
      mbar_wait_short(smem_addr(&drain), 0, a.err, a.wait_limit_ns);
    }
  } else {
    // ================================================ softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kRegsSoftmax));
    const int cq = warp >> 2, quarter = warp & 3;
    const int r = quarter * 32 + lane;  // TMEM lane = row of the tile
    const bool rv = real_row(r);
    const int pos = tile.ctx + tile.qbase + (rv ? token_of(a, r) : 0);  // padding rows: the first row's
    const uint32_t lane_addr = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t obuf = tmem + lane_addr + C::kOCol;

    // Q -> shared memory, 128B-swizzled K-major
#pragma unroll
    for (int cc = 0; cc < D / 32; ++cc) {
      const int c = cq * (D / 32) + cc;
      asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                       q_s + (c >> 3) * (C::kRows * 128) + swz128(r, c & 7)),
                   "r"(qv[cc].x), "r"(qv[cc].y), "r"(qv[cc].z), "r"(qv[cc].w)
                   : "memory");
    }
    fence_proxy_async();
    warp_arrive(smem_addr(&q_full));

    bool stopped = false;
    float m_run = -INFINITY, l_run = 0.f;  // m in the scores' unit
    const bool prescale = !(a.scale_log2 > 0.f);
    const float mul = prescale ? 1.f : a.scale_log2;
    for (int j = 0; j < ntiles; ++j) {
      const bool got = __all_sync(0xffffffffu, mbar_wait_short(smem_addr(&s_full[j & 1]), j >> 1 & 1,
                                                               a.err, a.wait_limit_ns));
      const int key0 = tile.key_base + j * C::kKeys + cq * 32;
      // O so far, its last product done, goes over to the new base.  P V of tile j - 1 is done when
      // S(j + 1), issued after it, is; the last tile has its own barrier.
      auto rebase = [&](float alpha) {
        if (j == 0) return;
        const bool more = j + 1 < ntiles;
        const bool done = __all_sync(
            0xffffffffu, mbar_wait_short(smem_addr(more ? &s_full[(j + 1) & 1] : &pv_done),
                                         more ? (j + 1) >> 1 & 1 : 0, a.err, a.wait_limit_ns));
        tmem_fence_after_sync();
        if (done) rescale(obuf + cq * (D / 2), D / 2, alpha);
        if (!done) softmax_stop = 1;  // no row is written
      };
      if (!soften<BF>(tmem + lane_addr + (j & 1) * 128, got, maxima, r, cq, 1 + quarter, prescale,
                      a.scale_log2, key0 + 31 > tile.ctx + tile.qbase, key0, pos, mul, j == 0,
                      m_run, l_run, rebase)) {
        stopped = true;  // the row's four warps leave together
        break;
      }
      const int tile0 = tile.key_base + j * C::kKeys;
      if (j == ntiles - 1 && tile0 + C::kKeys > tile.key_stop) {
        // V rows past the last visible key may hold any bits: each thread clears 64 columns of row r
        // once the tile has landed
        const int vst = j % C::kVStages;
        if (!mbar_wait_short(smem_addr(&v_full[vst]), (j / C::kVStages) & 1, a.err,
                             a.wait_limit_ns))
          softmax_stop = 1;  // no row is written
        else if (tile0 + r >= tile.key_stop)
          clear_v_row<2>(v_s + vst * C::kVBytes, r, cq >> 1, cq & 1);
        fence_proxy_async();
      }
      tmem_wait_st();
      tmem_fence_before_sync();
      warp_arrive(smem_addr(&p_full[j & 1]));
    }
    // The norm weights go where Q was (every S is done), for the rows that this CTA finishes.
    if (a.norm_w && tid < 2 * D / 4)
      reinterpret_cast<float4*>(smem + 8192)[tid] =
          __ldg(reinterpret_cast<const float4*>(a.norm_w) + tid);
    bool ok = !stopped;
    if (ok) ok = mbar_wait_short(smem_addr(&drain), 0, a.err, a.wait_limit_ns);
    if (!ok) softmax_stop = 1;
    softmax_sync();
    if (!*reinterpret_cast<volatile int*>(&softmax_stop)) {
      float* red = reinterpret_cast<float*>(smem);  // Q is done once drained
      red[cq * C::kRows + r] = l_run;
      if (cq == 0) red[4 * C::kRows + r] = m_run;
    }
  }
  __syncthreads();
  cluster_wait();  // so are the other CTA's

  // ---- the row's sum; then rows change sides: CTA `map` finishes rows 64 map .. 64 map + 63
  const int ch = warp >> 2, quarter = warp & 3, r = quarter * 32 + lane;  // softmax warps
  const bool mine = (quarter >> 1) == map, softmax = warp < kKWarp;
  const bool rv = softmax && real_row(r);
  const uint32_t obuf = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + C::kOCol;
  const float* red = reinterpret_cast<const float*>(smem);
  const bool ok = !softmax_stop;
  constexpr int kCols = 2 * D / 4;  // this thread's columns: kCols ch .. of O
  // O's 64-column pieces are in V's order (half, head); of y: (head, half)
  const int out0 = ((ch & 1) * 2 + (ch >> 1)) * 64;
  const float mul = a.scale_log2 > 0.f ? a.scale_log2 : 1.f;
  float inv = 0.f;
  tmem_fence_after_sync();
  if (softmax && ok) {
    const float l = (red[r] + red[C::kRows + r]) + (red[2 * C::kRows + r] + red[3 * C::kRows + r]);
    inv = l > 0.f ? 1.f / l : 0.f;  // 0: the row sees no key of this range
    if (nsplit > 1 && rv && ch == 0) {
      a.chunk_m[cell(r)] = red[4 * C::kRows + r] * mul;
      a.chunk_l[cell(r)] = l;
    }
  }
  if (nsplit > 1) {
    if (softmax && !ok && ch == 0) no_result(r);
    if (softmax && ok) {
#pragma unroll
      for (int c0 = 0; c0 < kCols; c0 += 32) {
        uint32_t t[32];
        tmem_ld32(obuf + ch * kCols + c0, t);
        tmem_wait_ld();
        tmem_regs_ready(t);
        if (rv) {
#pragma unroll
          for (int c = 0; c < 32; c += 4)
            store4(a.chunk_o + cell(r) * (2 * D) + out0 + c0 + c, t, c, inv);
        }
      }
    }
  } else {
    // Normalised sums -> shared memory, [row of the half][64 chunks of 16 bytes], a chunk's place
    // XORed with the row (conflict-free both ways): the rows this CTA finishes where K was, the
    // others in V's second stage, from which one bulk copy takes them to the other CTA's first.
    // This CTA's rings are done with: the other one may send.
    if (tid == 0) {
      mbar_arrive_expect_tx(smem_addr(&rows_in), 64 * 2 * D * 4);
      mbar_arrive_cluster(cluster_addr(smem_addr(&peer_free), map ^ 1));
    }
    const uint32_t own_s = k_s, out_s = v_s + C::kVBytes, in_s = v_s;
    // column of y of chunk 8 i + sub: O's 64-column pieces are in V's order (half, head)
    auto out_column = [](int i, int sub) {
      const int piece = i >> 1;
      return ((piece & 1) * 2 + (piece >> 1)) * 64 + ((i & 1) * 8 + sub) * 4;
    };
    auto chunk_at = [&](uint32_t base, int row, int c) {
      return base + row * (2 * D * 4) + ((c ^ (row & 7)) << 4);
    };
    // eight threads per row, 32 columns each (every eighth chunk)
    const int row = tid >> 3, sub = tid & 7, rr = 64 * map + row;
    const bool real = softmax && real_row(rr);
    const int64_t token = tile.row0 + tile.qbase + (real ? token_of(a, rr) : 0);
    const int dhead = pair * a.group + (real ? head_of(a, rr) : 0);
    const float lam = real ? __ldg(a.lam + token * a.lam_stride + dhead) : 0.f;
    if (softmax && ok) {
#pragma unroll
      for (int c0 = 0; c0 < kCols; c0 += 32) {
        uint32_t t[32];
        tmem_ld32(obuf + ch * kCols + c0, t);
        tmem_wait_ld();
        tmem_regs_ready(t);
#pragma unroll
        for (int c = 0; c < 32; c += 4)
          asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(
                           chunk_at(mine ? own_s : out_s, r & 63, (ch * kCols + c0 + c) / 4)),
                       "f"(__uint_as_float(t[c]) * inv), "f"(__uint_as_float(t[c + 1]) * inv),
                       "f"(__uint_as_float(t[c + 2]) * inv), "f"(__uint_as_float(t[c + 3]) * inv)
                       : "memory");
      }
      if (!mine) {
        // the 32 rows of this quarter go over as soon as its four warps have stored them
        fence_proxy_async();  // the bulk copy reads what these threads wrote
        asm volatile("bar.sync %0, 128;" ::"r"(1 + quarter) : "memory");
        const uint32_t at = (quarter & 1) * (32 * 2 * D * 4);
        if (ch == 0 && lane == 0 &&
            mbar_wait_cluster(smem_addr(&peer_free), 0, a.err, a.wait_limit_ns))
          asm volatile(
              "cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], "
              "%2, [%3];" ::"r"(cluster_addr(in_s + at, map ^ 1)),
              "r"(out_s + at), "r"(32 * 2 * D * 4),
              "r"(cluster_addr(smem_addr(&rows_in), map ^ 1))
              : "memory");
      }
      softmax_sync();  // this CTA's own rows are stored
    }
    // A CTA that failed sends nothing: the other one's wait runs out and its rows stay unwritten.
    if (softmax && ok && __all_sync(0xffffffffu, mbar_wait_short(smem_addr(&rows_in), 0, a.err,
                                                                 a.wait_limit_ns))) {
      float y[32], ss = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float4 x, p;
        asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                     : "=f"(x.x), "=f"(x.y), "=f"(x.z), "=f"(x.w)
                     : "r"(chunk_at(own_s, row, i * 8 + sub))
                     : "memory");
        asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                     : "=f"(p.x), "=f"(p.y), "=f"(p.z), "=f"(p.w)
                     : "r"(chunk_at(in_s, row, i * 8 + sub))
                     : "memory");
        if (map) {
          const float4 t = x;
          x = p;
          p = t;
        }
        y[4 * i] = difference(x.x, p.x, lam);
        y[4 * i + 1] = difference(x.y, p.y, lam);
        y[4 * i + 2] = difference(x.z, p.z, lam);
        y[4 * i + 3] = difference(x.w, p.w, lam);
      }
      float f = a.out_scale;
      if (a.norm_w) {
#pragma unroll
        for (int i = 0; i < 32; ++i) ss += y[i] * y[i];
#pragma unroll
        for (int off = 1; off < 8; off <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
        f *= rsqrtf(ss * (1.f / (2 * D)) + a.eps);
      }
      __half* out = a.out + (token * (a.num_q_heads / 2) + dhead) * (2 * D);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (a.norm_w) {
          const float4 w = reinterpret_cast<const float4*>(smem + 8192)[out_column(i, sub) / 4];
          y[4 * i] *= w.x;
          y[4 * i + 1] *= w.y;
          y[4 * i + 2] *= w.z;
          y[4 * i + 3] *= w.w;
        }
        if (real)
          *reinterpret_cast<uint2*>(out + out_column(i, sub)) = make_uint2(
              pack2<BF>(y[4 * i] * f, y[4 * i + 1] * f), pack2<BF>(y[4 * i + 2] * f, y[4 * i + 3] * f));
      }
    }
    cluster_sync();  // the copy out of this CTA's shared memory is done
  }

  tmem_fence_before_sync();
  __syncthreads();
  tmem_fence_after_sync();
  if (warp == 0) free_tmem(tmem, C::kTmemCols);
}

template <typename C, typename K>
cudaError_t launch_t(K kern, std::atomic<uint64_t>& done, const DiffArgs& a,
                     const CUtensorMap& kmap, const CUtensorMap& vmap, int ctas_per_tile,
                     cudaStream_t stream) {
  cudaError_t e = once_per_device(done, [&] {
    cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                           C::kSmemBytes);
    if (err != cudaSuccess) return err;
    // setmaxnreg.inc takes registers the CTA was launched with: never launch a build below the
    // split
    cudaFuncAttributes attr{};
    if ((err = cudaFuncGetAttributes(&attr, kern)) != cudaSuccess) return err;
    return attr.numRegs * C::kThreads < C::kRegsSoftmax * C::kSoftmax + C::kRegsOther * 128 ||
                   attr.numRegs * C::kThreads > 65536
               ? cudaErrorInvalidConfiguration
               : cudaSuccess;
  });
  if (e != cudaSuccess) return e;
  // Grid x: Q tiles, the last of a chunk (with the most keys) first, every pair of one before the
  // next: longest first over all pairs, so that the grid's tail is short (2432 rows, 32 + 8 heads
  // of 64, 49 us against 58 with one pair after the other; 4 x 512 rows, heads of 128, 177
  // against 180).
  DiffArgs b = a;
  b.tile_q = C::kRows / a.group;
  const int64_t rows = std::min<int64_t>(a.max_query_len, a.num_tokens);
  const int64_t tiles = (rows + b.tile_q - 1) / b.tile_q, ctas = tiles * a.num_pairs;
  // x / num_pairs as a multiplication: exact while x num_pairs < 2^32
  if (ctas * a.num_pairs > UINT32_MAX || ctas * ctas_per_tile > INT32_MAX)
    return cudaErrorInvalidConfiguration;
  b.chunk_tiles = static_cast<int>(tiles);
  b.pairs_inv = static_cast<uint32_t>(((uint64_t{1} << 32) + a.num_pairs - 1) / a.num_pairs);
  const dim3 grid(static_cast<unsigned>(ctas * ctas_per_tile), 1, a.prefill_seqs * a.key_splits);
  kern<<<grid, C::kThreads, C::kSmemBytes, stream>>>(kmap, vmap, b);
  return cudaGetLastError();
}

template <int BS, bool BF>
cudaError_t launch_d(const DiffArgs& a, const CUtensorMap& k, const CUtensorMap& v,
                     cudaStream_t st) {
  static std::atomic<uint64_t> map_done{0}, both_done{0};
  return a.head_dim == 128
             ? launch_t<MapCfg>(diff_chunk_map_kernel<BS, BF>, map_done, a, k, v, 2, st)
             : launch_t<BothCfg>(diff_chunk_both_kernel<BS, BF>, both_done, a, k, v, 1, st);
}

}  // namespace

cudaError_t launch_diff_chunk(const DiffArgs& a, const CUtensorMap& kmap, const CUtensorMap& vmap,
                              cudaStream_t stream) {
  if (a.block_size == 16)
    return a.bf16 ? launch_d<16, true>(a, kmap, vmap, stream)
                  : launch_d<16, false>(a, kmap, vmap, stream);
  return a.bf16 ? launch_d<32, true>(a, kmap, vmap, stream)
                : launch_d<32, false>(a, kmap, vmap, stream);
}

}  // namespace pa
