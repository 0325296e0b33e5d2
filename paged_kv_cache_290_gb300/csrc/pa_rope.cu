// Rotary positions with several axes, fused with the scatter-write of the step's K/V.
//
// Pair i of a head's R/2 rotated pairs turns by theta = position[axis_i][t] * f_i:
//   a' = (a cos theta - b sin theta) * factor,   b' = (b cos theta + a sin theta) * factor,
// with (a, b) = dims (i, i + R/2), or (2i, 2i + 1) when `adjacent`; dims R .. d-1 pass through.
// Rotated q goes to q_out, rotated k and plain v into their pages: k never exists rotated
// outside the cache, so its extra write and read are saved.
//
// Angles without far-position loss: f_i / 2 pi is held as a 64-bit fraction of a turn F_i, and
// position * F_i modulo 2^64 is the exact fraction of a turn of the angle (integer arithmetic,
// any sign); only then is it rounded to float32 for sincospif.  A float32 product position * f_i
// would be off by a hundredth of a radian at position 10^5.
//
// Bound by HBM for long chunks and by the launch for a decode step.  A CTA takes kTokens tokens:
// its threads compute the tokens' kTokens * R/2 (cos, sin) into shared memory, one sincospif for
// all heads, while their first loads are in flight; then each walks over (token, head)s with two
// 16-byte loads and stores each, one task's loads in flight while another's is turned.  Four
// CTAs an SM (64 registers): 8192 tokens of 64 + 8 heads of 128, bf16, 60 us = 5.6 TB/s, 0.84 of
// the measured copy rate (with 1 / 4 / 8 tokens a CTA 67 / 62 / 66 us; five CTAs of 48
// registers 76; 128, 384 or 512 threads 60 to 76); into an E4M3 pool three CTAs of 80 (8192 tokens
// of 32 + 8 heads 50 us; two CTAs 62).  K/V go to scattered slots, 256 bytes each.
// A decode step of 64 tokens (32 + 8 heads): 2.8 us on the device.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <string>

#include "pa.h"
#include "pa_common.cuh"
#include "pa_host.h"
#include "pa_kernels.h"

namespace pa {
namespace {

constexpr int kMaxPairs = 64;
constexpr int kThreads = 256;

struct RopeArgs {
  const __half* q;
  const __half* k;
  const __half* v;
  __half* q_out;
  int64_t q_stride, k_stride, v_stride, qo_stride;  // elements between tokens
  const int64_t* positions;
  int64_t pos_stride;  // elements between axes
  const int64_t* slot_mapping;
  void* k_cache;
  void* v_cache;
  float k_inv, v_inv;  // E4M3 pools: 1 / scale
  float factor;
  int64_t num_tokens;
  int64_t num_slots;
  int hq, hkv, block_size;
  int pairs;     // R / 2, a multiple of 8
  int adjacent;
  unsigned* err;
  uint64_t turn[kMaxPairs];  // fraction of a turn per position, times 2^64
  uint8_t axis[kMaxPairs];
};

template <bool BF>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
  if constexpr (BF) {
    return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w));
  } else {
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
  }
}

template <bool BF>
__device__ __forceinline__ void unpack8(const uint4& w, float (&x)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = unpack2<BF>(u[i]);
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}

template <bool BF>
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack2<BF>(x[0], x[1]), pack2<BF>(x[2], x[3]), pack2<BF>(x[4], x[5]),
                    pack2<BF>(x[6], x[7]));
}

// 8 values -> 8 E4M3 codes of x * inv (round to nearest even, saturating; NaN stays NaN).
__device__ __forceinline__ uint2 codes8(const float (&x)[8], float inv) {
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) c[i] = e4m3x2_from_f32(x[2 * i] * inv, x[2 * i + 1] * inv);
  return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

// Rotates the 8 pairs held in chunks x (first) and y (second): first = the a's and second the
// b's of the half layout; in the adjacent layout chunk x holds pairs 0..3, y pairs 4..7.
__device__ __forceinline__ void rotate8(float (&x)[8], float (&y)[8], const float* cos8,
                                        const float* sin8, bool adjacent) {
  float c[8], s[8];
#pragma unroll
  for (int i = 0; i < 8; i += 4) {
    const float4 cc = *reinterpret_cast<const float4*>(cos8 + i);
    const float4 ss = *reinterpret_cast<const float4*>(sin8 + i);
    c[i] = cc.x, c[i + 1] = cc.y, c[i + 2] = cc.z, c[i + 3] = cc.w;
    s[i] = ss.x, s[i + 1] = ss.y, s[i + 2] = ss.z, s[i + 3] = ss.w;
  }
  if (adjacent) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float a = x[2 * i], b = x[2 * i + 1];
      x[2 * i] = a * c[i] - b * s[i];
      x[2 * i + 1] = b * c[i] + a * s[i];
      const float e = y[2 * i], f = y[2 * i + 1];
      y[2 * i] = e * c[4 + i] - f * s[4 + i];
      y[2 * i + 1] = f * c[4 + i] + e * s[4 + i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float a = x[i], b = y[i];
      x[i] = a * c[i] - b * s[i];
      y[i] = b * c[i] + a * s[i];
    }
  }
}

// Thread = (head slot, column): a column is two 16-byte chunks of a head, 8 pairs.  A CTA covers
// tokens blockIdx.x * kTokens .. and heads blockIdx.y, blockIdx.y + gridDim.y, ... in units of
// kSlots heads; heads 0 .. hq-1 are q's, then k's, then v's.
template <int D, bool BF, bool F8, int kTokens>
__global__ void __launch_bounds__(kThreads, F8 ? 3 : 4) rope_and_cache_kernel(const __grid_constant__ RopeArgs a) {
  constexpr int kCols = D / 16, kSlots = kThreads / kCols;
  __shared__ __align__(16) float cos_s[kTokens][kMaxPairs], sin_s[kTokens][kMaxPairs];
  grid_launch_dependents();
  grid_dependency_wait();
  const int tid = threadIdx.x;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * kTokens;

  const int col = tid % kCols;
  const int rcols = a.pairs / 8;  // columns that rotate
  const bool rot = col < rcols;
  const bool adj = a.adjacent != 0;
  // the two chunks of this column in a q or k head (in a v head: col and col + kCols)
  const int ch0 = rot ? (adj ? 2 * col : col) : 2 * col;
  const int ch1 = rot ? (adj ? 2 * col + 1 : col + rcols) : 2 * col + 1;
  const int heads = a.hq + 2 * a.hkv;
  const int here = static_cast<int>(a.num_tokens - t0 < kTokens ? a.num_tokens - t0 : kTokens);

  // This thread's (token, head)s, one after the other.
  struct Task {
    uint4 w0, w1;
    int tt, h;     // token of the CTA, head
    int64_t slot;  // of a k or v head
    bool write;
  };
  int tt = 0, h = tid / kCols + static_cast<int>(blockIdx.y) * kSlots;
  auto settle = [&] {  // h past the token's heads goes on in the next token
    while (tt < here && h >= heads) {
      h -= heads;
      ++tt;
    }
  };
  auto load = [&](Task& q) {
    q.tt = tt;
    q.h = h;
    q.write = false;
    if (tt >= here) return;
    const int64_t t = t0 + tt;
    const bool is_q = h < a.hq, is_v = h >= a.hq + a.hkv;
    q.slot = is_q ? 0 : a.slot_mapping[t];
    q.write = q.slot >= 0 && q.slot < a.num_slots;
    if (q.write) {
      const int hh = is_q ? h : is_v ? h - a.hq - a.hkv : h - a.hq;
      const __half* src = (is_q ? a.q + t * a.q_stride : is_v ? a.v + t * a.v_stride
                                                             : a.k + t * a.k_stride) +
                          static_cast<int64_t>(hh) * D;
      q.w0 = *reinterpret_cast<const uint4*>(src + (is_v ? col : ch0) * 8);
      q.w1 = *reinterpret_cast<const uint4*>(src + (is_v ? col + kCols : ch1) * 8);
    } else if (q.slot >= 0 && h == a.hq && col == 0) {
      atomicOr(a.err, kErrSlotRange);  // once per token: its first k head
    }
    h += static_cast<int>(gridDim.y) * kSlots;
    settle();
  };
  auto finish = [&](Task& q) {
    if (!q.write) return;
    const int64_t t = t0 + q.tt;
    const bool is_q = q.h < a.hq, is_v = q.h >= a.hq + a.hkv;
    const int hh = is_q ? q.h : is_v ? q.h - a.hq - a.hkv : q.h - a.hq;
    const int x0 = is_v ? col : ch0, x1 = is_v ? col + kCols : ch1;
    const bool turns = rot && !is_v;
    float x[8], y[8];
    if (turns || (F8 && !is_q)) {
      unpack8<BF>(q.w0, x);
      unpack8<BF>(q.w1, y);
    }
    if (turns) {
      rotate8(x, y, &cos_s[q.tt][col * 8], &sin_s[q.tt][col * 8], adj);
      if (!F8 || is_q) {
        q.w0 = pack8<BF>(x);
        q.w1 = pack8<BF>(y);
      }
    }
    if (is_q) {
      __half* dst = a.q_out + t * a.qo_stride + static_cast<int64_t>(hh) * D;
      *reinterpret_cast<uint4*>(dst + x0 * 8) = q.w0;
      *reinterpret_cast<uint4*>(dst + x1 * 8) = q.w1;
    } else {
      const int64_t blk = q.slot / a.block_size;
      const int off = static_cast<int>(q.slot - blk * a.block_size);
      const int64_t base = ((blk * a.hkv + hh) * a.block_size + off) * D;
      void* pool = is_v ? a.v_cache : a.k_cache;
      if constexpr (F8) {
        // the float32 rotation goes straight to its code: one rounding
        const float inv = is_v ? a.v_inv : a.k_inv;
        uint8_t* dst = static_cast<uint8_t*>(pool) + base;
        *reinterpret_cast<uint2*>(dst + x0 * 8) = codes8(x, inv);
        *reinterpret_cast<uint2*>(dst + x1 * 8) = codes8(y, inv);
      } else {
        __half* dst = static_cast<__half*>(pool) + base;
        *reinterpret_cast<uint4*>(dst + x0 * 8) = q.w0;
        *reinterpret_cast<uint4*>(dst + x1 * 8) = q.w1;
      }
    }
  };

  // Two tasks in turn: one's loads are in flight while the other is turned and stored; the first
  // one's while the angles are computed.
  settle();
  Task even, odd;
  load(even);
  for (int i = tid; i < here * a.pairs; i += kThreads) {
    const int token = i / a.pairs, p = i % a.pairs;
    const int64_t pos = a.positions[a.axis[p] * a.pos_stride + t0 + token];
    // signed fraction of a turn, times 2^64; in half turns (sincospif's unit): times 2^-63
    const int64_t turn = static_cast<int64_t>(static_cast<uint64_t>(pos) * a.turn[p]);
    float sn, cs;
    sincospif(__ll2float_rn(turn) * 0x1p-63f, &sn, &cs);
    cos_s[token][p] = cs * a.factor;
    sin_s[token][p] = sn * a.factor;
  }
  __syncthreads();
  while (even.tt < here) {
    load(odd);
    finish(even);
    load(even);
    finish(odd);
  }
}

template <int D, bool BF, bool F8>
cudaError_t launch(const RopeArgs& a, int num_sms, cudaStream_t stream) {
  constexpr int kSlots = kThreads / (D / 16);
  const int units = (a.hq + 2 * a.hkv + kSlots - 1) / kSlots;  // head units of a token
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (a.num_tokens >= 4 * num_sms) {
    cfg.gridDim = dim3(static_cast<unsigned>((a.num_tokens + 1) / 2));
    return cudaLaunchKernelEx(&cfg, rope_and_cache_kernel<D, BF, F8, 2>, a);
  }
  const int64_t want = (2 * num_sms + a.num_tokens - 1) / a.num_tokens;
  cfg.gridDim = dim3(static_cast<unsigned>(a.num_tokens),
                     static_cast<unsigned>(std::max<int64_t>(1, std::min<int64_t>(units, want))));
  return cudaLaunchKernelEx(&cfg, rope_and_cache_kernel<D, BF, F8, 1>, a);
}

template <int D>
cudaError_t launch_d(const RopeArgs& a, bool bf, bool f8, int sms, cudaStream_t st) {
  if (f8) return launch<D, false, true>(a, sms, st);
  return bf ? launch<D, true, false>(a, sms, st) : launch<D, false, false>(a, sms, st);
}

// Bytes [lo, hi) that a [T, H, d] tensor of 16-bit values spans.
void span(const pa_tensor* x, uintptr_t* lo, uintptr_t* hi) {
  *lo = reinterpret_cast<uintptr_t>(x->data);
  *hi = *lo + 2 * static_cast<uintptr_t>((x->shape[0] - 1) * x->stride[0] +
                                         x->shape[1] * x->shape[2]);
}

}  // namespace
}  // namespace pa

extern "C" int pa_rope_and_cache(const pa_tensor* q, const pa_tensor* k, const pa_tensor* v,
                                 const pa_tensor* positions, const pa_rope* rope,
                                 const pa_tensor* k_cache, const pa_tensor* v_cache,
                                 const pa_tensor* slot_mapping, const pa_tensor* q_out,
                                 const pa_kv_scales* scales, void* stream) {
  using namespace pa;
  clear_last_error();
  int rc;
  const bool fp8 = k_cache && k_cache->dtype == PA_F8E4M3;
  if (fp8 && (rc = check_scales(scales))) return rc;
  const int dt = fp8 ? PA_F16 : pool_dtype16(k_cache);
  if ((rc = check_pool(k_cache, v_cache, fp8 ? PA_F8E4M3 : dt))) return rc;
  if ((rc = check_tensor(q, "q", dt, 3))) return rc;
  if ((rc = check_tensor(k, "k", dt, 3))) return rc;
  if ((rc = check_tensor(v, "v", dt, 3))) return rc;
  if ((rc = check_tensor(q_out, "q_out", dt, 3))) return rc;
  if ((rc = check_tensor(positions, "positions", PA_I64, 2))) return rc;
  if ((rc = check_tensor(slot_mapping, "slot_mapping", PA_I64, 1))) return rc;
  const int64_t t = q->shape[0], hq = q->shape[1], d = k_cache->shape[3];
  const int64_t hkv = k_cache->shape[1];
  if (hq < 1 || hq > 65535 || q->shape[2] != d)
    return fail(PA_ERR_INVALID_ARG, "q must be [T, num_q_heads, head_dim] matching the pool");
  for (int i = 0; i < 3; ++i)
    if (q_out->shape[i] != q->shape[i])
      return fail(PA_ERR_INVALID_ARG, "q_out must have q's shape");
  for (const pa_tensor* x : {k, v})
    if (x->shape[0] != t || x->shape[1] != hkv || x->shape[2] != d)
      return fail(PA_ERR_INVALID_ARG, "k and v must be [T, num_kv_heads, head_dim] matching the pool");
  if (t > 0)
    for (const pa_tensor* x : {q, k, v, q_out})
      if ((x->shape[1] > 1 && x->stride[1] != d) ||
          (t > 1 && (x->stride[0] < x->shape[1] * d || x->stride[0] % 8 != 0)) ||
          !aligned16(x->data))
        return fail(PA_ERR_INVALID_ARG,
                    "q / k / v / q_out need head stride head_dim, token stride >= heads*head_dim "
                    "and a multiple of 8, and 16-byte alignment");
  if (slot_mapping->shape[0] != t)
    return fail(PA_ERR_INVALID_ARG, "slot_mapping must have T entries");
  if (!rope || !rope->inv_freq) return fail(PA_ERR_INVALID_ARG, "rope or its inv_freq is NULL");
  if (rope->num_pairs < 8 || rope->num_pairs % 8 != 0 || 2 * rope->num_pairs > d)
    return fail(PA_ERR_INVALID_ARG,
                "num_pairs must be a multiple of 8 with 2 * num_pairs <= head_dim");
  if (positions->shape[0] < 1 || positions->shape[0] > 255 || positions->shape[1] != t)
    return fail(PA_ERR_INVALID_ARG, "positions must be [num_axes, T] with 1 to 255 axes");
  if (!(rope->factor - rope->factor == 0.f))
    return fail(PA_ERR_INVALID_ARG, "factor must be finite");
  RopeArgs a{};
  for (int i = 0; i < rope->num_pairs; ++i) {
    const double f = rope->inv_freq[i];
    const int32_t ax = rope->axis_of_pair ? rope->axis_of_pair[i] : 0;
    if (!std::isfinite(f)) return fail(PA_ERR_INVALID_ARG, "inv_freq must be finite");
    if (ax < 0 || ax >= positions->shape[0])
      return fail(PA_ERR_INVALID_ARG, "axis_of_pair names an axis that positions lacks");
    // whole turns per position change nothing: keep the fraction, as an integer over 2^64
    double turns = f * 0.15915494309189533577;  // 1 / (2 pi)
    turns -= std::floor(turns);
    a.turn[i] = turns < 1.0 ? static_cast<uint64_t>(turns * 0x1p64) : 0;
    a.axis[i] = static_cast<uint8_t>(ax);
  }
  if (t == 0) return PA_OK;
  if (t > INT32_MAX) return fail(PA_ERR_UNSUPPORTED, "2^31 or more tokens in one call");
  if (q_out->data != q->data || (t > 1 && q_out->stride[0] != q->stride[0])) {
    uintptr_t lo, hi, olo, ohi;
    span(q_out, &olo, &ohi);
    for (const pa_tensor* x : {q, k, v}) {
      span(x, &lo, &hi);
      if (lo < ohi && olo < hi)
        return fail(PA_ERR_INVALID_ARG, "q_out must be q itself or not overlap q, k or v");
    }
  }
  a.q = static_cast<const __half*>(q->data);
  a.k = static_cast<const __half*>(k->data);
  a.v = static_cast<const __half*>(v->data);
  a.q_out = static_cast<__half*>(q_out->data);
  a.q_stride = q->stride[0];
  a.k_stride = k->stride[0];
  a.v_stride = v->stride[0];
  a.qo_stride = q_out->stride[0];
  a.positions = static_cast<const int64_t*>(positions->data);
  a.pos_stride = positions->stride[0];
  a.slot_mapping = static_cast<const int64_t*>(slot_mapping->data);
  a.k_cache = k_cache->data;
  a.v_cache = v_cache->data;
  a.k_inv = fp8 ? 1.0f / scales->k_scale : 1.f;
  a.v_inv = fp8 ? 1.0f / scales->v_scale : 1.f;
  a.factor = rope->factor;
  a.num_tokens = t;
  a.num_slots = k_cache->shape[0] * k_cache->shape[2];
  a.hq = static_cast<int>(hq);
  a.hkv = static_cast<int>(hkv);
  a.block_size = static_cast<int>(k_cache->shape[2]);
  a.pairs = rope->num_pairs;
  a.adjacent = rope->adjacent ? 1 : 0;
  int sms = 0;
  cudaError_t e = error_word(stream, &a.err);
  if (e != cudaSuccess) return cuda_fail(e, "error word");
  if ((e = device_sm_count(&sms)) != cudaSuccess) return cuda_fail(e, "device attribute");
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  e = d == 128 ? launch_d<128>(a, dt == PA_BF16, fp8, sms, st)
               : launch_d<64>(a, dt == PA_BF16, fp8, sms, st);
  if (e != cudaSuccess) return cuda_fail(e, "rope_and_cache launch");
  return PA_OK;
}
