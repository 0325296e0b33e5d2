// Moves of whole pages inside the pool, in place, where a move's destination may be another
// move's source (chains and cycles, as a compaction makes them), and the block tables' new ids.
//
// Plan (host, once per list of moves).  Moves are put in chain order, each chain from its end:
// the move out of a page then comes before the move into it.  Consecutive moves form groups of
// kGroup, and groups form launches of at most kMaxMoves moves.  A CTA (one warp) owns the same
// slice of every page of a group: it copies the slices of all the group's sources into shared
// memory (bulk copies), waits for them, then copies them to the destinations, so inside a group
// any chain or cycle is safe.  Launches run one after the other.  What is left is a page that
// another group overwrites in the same launch, or that an earlier launch has overwritten: those
// sources (one or two per kGroup moves of a long chain, none where holes are filled) are first
// copied into the workspace and read from there.
//
// Bound by HBM: each moved byte is read and written once, plus staging (about 1 in kGroup of a
// chain's moves, read and written once more).  4096 pages of 8 layers put in order (2.1 GB, long
// cycles) 656 us = 6.55 TB/s of moved bytes read and written, 0.98 of the measured copy rate (with
// launches of 1024 moves 667 us, and with those, groups of 8 in registers, a thread per 16 bytes, 729,
// an eighth of the pages staged; 16 x 2 KB 680); 2 x 1501 holes of four E4M3 layers 62 us, 0.95.  The
// moves travel as kernel arguments: no upload, and a captured launch keeps its own copy.
#include <cuda_runtime.h>

#include <algorithm>
#include <new>
#include <string>
#include <type_traits>
#include <vector>

#include "pa.h"
#include "pa_common.cuh"
#include "pa_host.h"
#include "pa_kernels.h"

namespace pa {
namespace {

constexpr int kGroup = 32;
// Moves per launch, which travel as kernel arguments: 24 KB of the 32 KB there are (1501 holes 64.9
// us with 12 KB, 62.0 with 24).  A short list takes the small size, whose arguments stay below 4 KB
// (a launch of the small size costs 3.0 us on the host).
constexpr int kMaxMoves = 2048, kFewMoves = 256;
constexpr int kThreads = 256;  // of the renaming
// Moves and bytes of a page per CTA: a list with chains keeps the plan's groups together; one
// without takes smaller groups of longer slices, which start sooner (48 moves 1.3 us less, 1501
// holes of an FP8 pool 67 -> 64.5 us).
constexpr int kLooseGroup = 8, kSlice = 1024, kLooseSlice = 2048;
static_assert(kMaxMoves % kGroup == 0 && kFewMoves % kGroup == 0, "a group lies in one launch");

template <int N>
struct MoveArgs {
  uint4* k;
  uint4* v;
  uint4* stage;          // [slot][layer of the batch][K, V][chunks]
  int64_t layer_stride;  // chunks between layers of the pools
  int64_t chunks;        // 16-byte chunks of one page of K (or V)
  unsigned* err;
  int layer0, layers;    // the batch of layers this launch covers
  int group, slice;      // moves, and bytes of a page, of a CTA
  int n;
  int32_t* old_ids;      // long lists with tables: the move's old and new id by position, and a
  int32_t* new_ids;      // page's position
  int32_t* position;
  int base;              // position of this launch's first move
  int32_t* tables;       // short lists: [rows, cols], renamed by the grid's last z plane
  int64_t rows, stride;
  int cols;
  int32_t src[N];  // page id, or ~slot of the workspace
  int32_t dst[N];  // page id, or ~slot
  int32_t id[N];   // the moved page's old id
};

// Block tables after a short list of moves (at most kFewMoves): old ids and their new ones in a hash
// table in shared memory (2 kFewMoves places of (id, new id), which the moves fill at most by half),
// built by every block that renames.  Nothing here waits for the moves themselves.
template <int N>
__device__ __forceinline__ void rename_few(const MoveArgs<N>& a, int2* hash, int64_t first,
                                           int64_t step) {
  constexpr int kBits = 9;
  static_assert((1 << kBits) == 2 * kFewMoves, "half full at most");
  constexpr int kPlaces = 1 << kBits;
  auto place = [](int32_t id) { return (static_cast<uint32_t>(id) * 0x9E3779B1u) >> (32 - kBits); };
  for (int i = threadIdx.x; i < kPlaces; i += blockDim.x) hash[i] = make_int2(-1, -1);
  __syncthreads();
  for (int i = threadIdx.x; i < a.n; i += blockDim.x) {
    uint32_t p = place(a.id[i]);
    while (atomicCAS(&hash[p].x, -1, a.id[i]) != -1) p = (p + 1) % kPlaces;  // ids are distinct
    hash[p].y = a.dst[i];
  }
  __syncthreads();
  const int64_t total = a.rows * a.cols;
  for (int64_t i = first; i < total; i += step) {
    const int64_t row = total <= INT32_MAX ? static_cast<int>(i) / a.cols : i / a.cols;
    int32_t* e = a.tables + row * a.stride + (i - row * a.cols);
    const int32_t id = *e;
    if (id < 0) continue;  // padding
    for (uint32_t p = place(id); hash[p].x >= 0; p = (p + 1) % kPlaces)
      if (hash[p].x == id) {
        *e = hash[p].y;
        break;
      }
  }
}

// The renaming alone, where the tables are too long for the blocks that move.
__global__ void __launch_bounds__(kThreads)
    rename_few_kernel(const __grid_constant__ MoveArgs<kFewMoves> a) {
  __shared__ int2 hash[2 * kFewMoves];
  rename_few(a, hash, static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x,
             static_cast<int64_t>(gridDim.x) * kThreads);
}

template <int N>
__global__ void __launch_bounds__(32) move_kernel(const __grid_constant__ MoveArgs<N> a) {
  extern __shared__ __align__(128) uint8_t buf[];  // [move of the group][slice]
  __shared__ __align__(8) uint64_t full;
  const int g0 = static_cast<int>(blockIdx.y) * a.group, n = min(a.group, a.n - g0);
  const int lz = static_cast<int>(blockIdx.z) >> 1, kv = static_cast<int>(blockIdx.z) & 1;
  const int lane = threadIdx.x;
  if constexpr (N == kFewMoves)
    if (lz == a.layers) {
      const int64_t cta = blockIdx.y * gridDim.x + blockIdx.x;
      if (cta * 32 < a.rows * a.cols)
        rename_few(a, reinterpret_cast<int2*>(buf), cta * 32 + lane,
                   static_cast<int64_t>(gridDim.x) * gridDim.y * 32);
      return;
    }
  if (a.position && blockIdx.x == 0 && blockIdx.z == 0)
    for (int i = lane; i < n; i += 32) {
      a.old_ids[a.base + g0 + i] = a.id[g0 + i];
      a.new_ids[a.base + g0 + i] = a.dst[g0 + i];
      a.position[a.id[g0 + i]] = a.base + g0 + i;
    }
  const int64_t c = static_cast<int64_t>(blockIdx.x) * (a.slice / 16);
  const int bytes = static_cast<int>(min(static_cast<int64_t>(a.slice), (a.chunks - c) * 16));
  uint4* pool = (kv ? a.v : a.k) + (a.layer0 + lz) * a.layer_stride + c;
  uint4* stage = a.stage + (static_cast<int64_t>(lz) * 2 + kv) * a.chunks + c;
  const int64_t slot = static_cast<int64_t>(a.layers) * 2 * a.chunks;  // chunks per slot
  auto at = [&](int32_t i) { return i >= 0 ? pool + i * a.chunks : stage + ~i * slot; };
  const uint32_t bar = smem_addr(&full), base = smem_addr(buf);
  if (lane == 0) {
    mbar_init(bar, 1);
    mbar_init_fence();
    mbar_arrive_expect_tx(bar, n * bytes);
  }
  __syncwarp();
  for (int i = lane; i < n; i += 32)
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::
            "r"(base + i * a.slice),
        "l"(at(a.src[g0 + i])), "r"(bytes), "r"(bar)
        : "memory");
  // A copy that never lands (no legitimate wait takes two seconds) leaves the destinations alone,
  // and is given as long again before the CTA retires.
  if (!__all_sync(0xffffffffu, mbar_wait_short(bar, 0, a.err))) {
    mbar_wait_short(bar, 0, a.err);
    return;
  }
  __syncwarp();
  for (int i = lane; i < n; i += 32)
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(
                     at(a.dst[g0 + i])),
                 "r"(base + i * a.slice), "r"(bytes)
                 : "memory");
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
  asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

// A moved page's id is replaced, after a long list.  `position` is meaningful for moved pages only: any other entry
// holds whatever the workspace held, and is told apart by old_ids.
__global__ void __launch_bounds__(kThreads)
    rename_kernel(int32_t* tables, int64_t rows, int cols, int64_t stride, int64_t num_blocks, int n,
                  const int32_t* old_ids, const int32_t* new_ids, const int32_t* position) {
  const int64_t total = rows * cols;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < total;
       i += static_cast<int64_t>(gridDim.x) * kThreads) {
    int32_t* e = tables + i / cols * stride + i % cols;
    const int32_t id = *e;
    if (id < 0 || id >= num_blocks) continue;  // padding
    const int32_t p = position[id];
    if (p >= 0 && p < n && old_ids[p] == id) *e = new_ids[p];
  }
}

}  // namespace
}  // namespace pa

struct pa_move_plan {
  int64_t num_blocks = 0;
  std::vector<int32_t> src, dst, id;  // the moves in order; src: page, or ~slot
  std::vector<int32_t> staged;        // page of each workspace slot
  bool chained = false;               // some page is both left and entered
};

namespace {

// Fills `p` from the checked pairs; throws std::bad_alloc.
void make_plan(pa_move_plan* p, const int32_t* pairs, int64_t n) {
  const size_t nb = static_cast<size_t>(p->num_blocks);
  std::vector<int32_t> from(nb, -1), to(nb, -1), order(nb, -1);
  for (int64_t i = 0; i < n; ++i)
    if (pairs[2 * i] != pairs[2 * i + 1]) {
      to[pairs[2 * i]] = pairs[2 * i + 1];
      from[pairs[2 * i + 1]] = pairs[2 * i];
    }
  // the move into page x is recorded at order[x]
  auto emit = [&](int32_t x) {
    order[x] = static_cast<int32_t>(p->dst.size());
    p->id.push_back(from[x]);
    p->dst.push_back(x);
  };
  for (int64_t i = 0; i < n; ++i)  // chains, from the page that nothing leaves
    if (to[pairs[2 * i + 1]] < 0 && from[pairs[2 * i + 1]] >= 0)
      for (int32_t x = pairs[2 * i + 1]; x >= 0 && from[x] >= 0; x = from[x]) emit(x);
  for (int64_t i = 0; i < n; ++i)  // cycles
    for (int32_t x = pairs[2 * i + 1]; from[x] >= 0 && order[x] < 0; x = from[x]) emit(x);
  p->src = p->id;
  for (size_t j = 0; j < p->src.size(); ++j) {
    const int32_t i = order[p->id[j]];  // the move that overwrites this source
    if (i < 0) continue;
    p->chained = true;
    if (static_cast<size_t>(i) / pa::kGroup == j / pa::kGroup) continue;
    if (static_cast<size_t>(i) > j && static_cast<size_t>(i) / pa::kMaxMoves != j / pa::kMaxMoves)
      continue;  // a later launch
    p->src[j] = ~static_cast<int32_t>(p->staged.size());
    p->staged.push_back(p->id[j]);
  }
}

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

size_t rename_bytes(const pa_move_plan* p) {
  if (p->dst.size() <= static_cast<size_t>(pa::kFewMoves)) return 0;
  return 2 * up256(p->dst.size() * sizeof(int32_t)) +
         up256(static_cast<size_t>(p->num_blocks) * sizeof(int32_t));
}

// One layer [NB, Hkv, bs, d] of a pool given as such or as [L, NB, Hkv, bs, d].
int layers_of(const pa_tensor* x, const char* name, pa_tensor* layer, int64_t* num, int64_t* stride) {
  if (!x) return pa::fail(PA_ERR_INVALID_ARG, std::string(name) + " is NULL");
  if (x->ndim != 4 && x->ndim != 5)
    return pa::fail(PA_ERR_INVALID_ARG, std::string(name) + " must have rank 4 or 5");
  const int o = x->ndim - 4;
  *layer = *x;
  layer->ndim = 4;
  for (int i = 0; i < 4; ++i) {
    layer->shape[i] = x->shape[i + o];
    layer->stride[i] = x->stride[i + o];
  }
  *num = o ? x->shape[0] : 1;
  *stride = o ? x->stride[0] : 0;
  if (*num < 1 || *num > 32767)
    return pa::fail(PA_ERR_INVALID_ARG, std::string(name) + " must have 1 to 32767 layers");
  return PA_OK;
}

}  // namespace

extern "C" {

pa_move_plan* pa_move_plan_create(const int32_t* pairs, int64_t n, int64_t num_blocks) {
  using namespace pa;
  clear_last_error();
  if (n < 0 || (n > 0 && !pairs) || num_blocks < 0 || num_blocks > INT32_MAX) {
    fail(PA_ERR_INVALID_ARG, "move plan: NULL pairs or bad size");
    return nullptr;
  }
  pa_move_plan* p = nullptr;
  try {
    std::vector<uint8_t> seen(static_cast<size_t>(num_blocks), 0);
    for (int64_t i = 0; i < n; ++i)
      for (int e = 0; e < 2; ++e) {
        const int32_t b = pairs[2 * i + e];
        if (b < 0 || b >= num_blocks) {
          fail(PA_ERR_INVALID_ARG, "move plan: a block id is outside the pool");
          return nullptr;
        }
        if (seen[b] & (1 << e)) {
          fail(PA_ERR_INVALID_ARG, e ? "move plan: two moves into one block"
                                     : "move plan: two moves out of one block");
          return nullptr;
        }
        seen[b] |= 1 << e;
      }
    p = new pa_move_plan();
    p->num_blocks = num_blocks;
    make_plan(p, pairs, n);
    return p;
  } catch (...) {
    delete p;
    try {
      fail(PA_ERR_INVALID_ARG, "move plan: out of host memory");
    } catch (...) {
    }
    return nullptr;
  }
}

void pa_move_plan_destroy(pa_move_plan* plan) { delete plan; }

int64_t pa_move_plan_staged(const pa_move_plan* plan) {
  return plan ? static_cast<int64_t>(plan->staged.size()) : 0;
}

size_t pa_move_blocks_workspace_size(const pa_move_plan* plan, const pa_tensor* k_cache,
                                     int32_t layers, int32_t with_tables) {
  pa_tensor l;
  int64_t num, stride;
  if (!plan || layers < 1 || layers_of(k_cache, "k_cache", &l, &num, &stride)) return 0;
  const size_t page = static_cast<size_t>(l.shape[1] * l.shape[2] * l.shape[3]) *
                      (l.dtype == PA_F8E4M3 ? 1 : 2);
  return (with_tables && !plan->dst.empty() ? rename_bytes(plan) : 0) +
         plan->staged.size() * 2 * page * layers;
}

int pa_move_blocks(const pa_move_plan* plan, const pa_tensor* k_cache, const pa_tensor* v_cache,
                   const pa_tensor* block_tables, void* workspace, size_t workspace_bytes,
                   void* stream) {
  using namespace pa;
  clear_last_error();
  if (!plan) return fail(PA_ERR_INVALID_ARG, "plan is NULL");
  int rc;
  pa_tensor kl, vl;
  int64_t layers, vlayers, kstride, vstride;
  if ((rc = layers_of(k_cache, "k_cache", &kl, &layers, &kstride))) return rc;
  if ((rc = layers_of(v_cache, "v_cache", &vl, &vlayers, &vstride))) return rc;
  const bool fp8 = kl.dtype == PA_F8E4M3;
  if ((rc = check_pool(&kl, &vl, fp8 ? PA_F8E4M3 : pool_dtype16(&kl)))) return rc;
  if (layers != vlayers || kstride != vstride)
    return fail(PA_ERR_INVALID_ARG, "k_cache and v_cache layers differ");
  if (kl.shape[0] != plan->num_blocks)
    return fail(PA_ERR_INVALID_ARG, "the plan was made for a pool of " +
                                        std::to_string(plan->num_blocks) + " blocks");
  const int64_t page = kl.shape[1] * kl.shape[2] * kl.shape[3];  // values
  const int64_t per16 = fp8 ? 16 : 8;
  if (layers > 1 && (kstride < kl.shape[0] * page || kstride % per16 != 0))
    return fail(PA_ERR_INVALID_ARG, "layers must not overlap and must be 16-byte aligned");
  if (block_tables) {
    if ((rc = check_tensor(block_tables, "block_tables", PA_I32, 2))) return rc;
    if (block_tables->shape[1] > INT32_MAX ||
        (block_tables->shape[0] > 1 && block_tables->stride[0] < block_tables->shape[1]))
      return fail(PA_ERR_INVALID_ARG, "block_tables row stride must cover its columns");
  }
  const int64_t n = static_cast<int64_t>(plan->dst.size());
  if (n == 0) return PA_OK;
  // K's and V's layers may alternate in one buffer, but no two may overlap
  const int64_t k0 = reinterpret_cast<intptr_t>(kl.data), v0 = reinterpret_cast<intptr_t>(vl.data);
  const int64_t esize = fp8 ? 1 : 2, one = kl.shape[0] * page * esize, step = kstride * esize;
  const int64_t apart = k0 > v0 ? k0 - v0 : v0 - k0;
  if (apart < (layers - 1) * step + one) {
    const int64_t phase = layers > 1 ? apart % step : 0;
    if (layers == 1 || phase < one || step - phase < one)
      return fail(PA_ERR_INVALID_ARG, "k_cache and v_cache overlap");
  }

  const bool tables = block_tables && block_tables->shape[0] > 0 && block_tables->shape[1] > 0;
  const size_t fixed = tables ? rename_bytes(plan) : 0;
  const size_t slot = static_cast<size_t>(page) * 2 * (fp8 ? 1 : 2);  // K and V, one layer
  const size_t per_layer = plan->staged.size() * slot;
  const size_t need = fixed + per_layer;
  if (need > 0) {
    if (!workspace || workspace_bytes < need)
      return fail(PA_ERR_WORKSPACE, "workspace needs " + std::to_string(need) + " bytes");
    if (reinterpret_cast<uintptr_t>(workspace) & 255u)
      return fail(PA_ERR_WORKSPACE, "workspace must be 256-byte aligned");
  }
  // as many layers at once as the workspace stages
  int64_t batch = per_layer ? static_cast<int64_t>((workspace_bytes - fixed) / per_layer) : layers;
  batch = std::min<int64_t>(std::max<int64_t>(batch, 1), layers);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const bool few = n <= kFewMoves, listed = tables && !few;
  int32_t* old_ids = listed ? reinterpret_cast<int32_t*>(ws) : nullptr;
  int32_t* new_ids = listed ? reinterpret_cast<int32_t*>(ws + up256(n * sizeof(int32_t))) : nullptr;
  int32_t* position =
      listed ? reinterpret_cast<int32_t*>(ws + 2 * up256(n * sizeof(int32_t))) : nullptr;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  unsigned* err = nullptr;
  if ((e = error_word(stream, &err)) != cudaSuccess) return cuda_fail(e, "error word");
  auto run = [&](auto& a, int most) -> int {
    a.k = static_cast<uint4*>(kl.data);
    a.v = static_cast<uint4*>(vl.data);
    a.stage = reinterpret_cast<uint4*>(ws + fixed);
    a.layer_stride = kstride / per16;
    a.chunks = page / per16;
    a.old_ids = old_ids;
    a.new_ids = new_ids;
    a.err = err;
    a.group = plan->chained ? kGroup : kLooseGroup;
    a.slice = plan->chained ? kSlice : kLooseSlice;
    auto launch = [&](bool rename) {
      dim3 grid(static_cast<unsigned>((a.chunks * 16 + a.slice - 1) / a.slice),
                static_cast<unsigned>((a.n + a.group - 1) / a.group),
                static_cast<unsigned>(2 * a.layers));
      if (rename) {
        a.tables = static_cast<int32_t*>(block_tables->data);
        a.rows = block_tables->shape[0];
        a.cols = static_cast<int>(block_tables->shape[1]);
        a.stride = block_tables->stride[0];
        // Up to 8 entries a thread ride along (48 moves in a pool of 512 pages, 16 tables: 4.6 -> 2.9
        // us on the device and 8.8 -> 4.7 a call against a second launch and its workspace); longer
        // tables have a launch of their own.
        const int64_t total = a.rows * a.cols, ride = int64_t{8 * 32} * grid.x * grid.y;
        if (total <= ride) {
          grid.z += 1;
        } else if constexpr (std::is_same_v<std::decay_t<decltype(a)>, MoveArgs<kFewMoves>>) {
          const int64_t blocks = std::min<int64_t>((total + kThreads - 1) / kThreads, 152 * 8);
          rename_few_kernel<<<static_cast<unsigned>(blocks), kThreads, 0, st>>>(a);
          if ((e = cudaGetLastError()) != cudaSuccess) return e;
        }
      }
      move_kernel<<<grid, 32, a.group * a.slice, st>>>(a);  // 16 or 32 KB of shared memory
      return cudaGetLastError();
    };
    for (int64_t l0 = 0; l0 < layers; l0 += batch) {
      a.layer0 = static_cast<int>(l0);
      a.layers = static_cast<int>(std::min(batch, layers - l0));
      a.position = nullptr;
      const int64_t ns = static_cast<int64_t>(plan->staged.size());
      for (int64_t b = 0; b < ns; b += most) {
        a.n = static_cast<int>(std::min<int64_t>(most, ns - b));
        for (int i = 0; i < a.n; ++i) {
          a.src[i] = plan->staged[b + i];
          a.dst[i] = ~static_cast<int32_t>(b + i);
        }
        if ((e = launch(false)) != cudaSuccess) return cuda_fail(e, "move_blocks staging launch");
      }
      a.position = l0 == 0 ? position : nullptr;
      for (int64_t b = 0; b < n; b += most) {
        a.n = static_cast<int>(std::min<int64_t>(most, n - b));
        a.base = static_cast<int>(b);
        std::copy_n(plan->src.data() + b, a.n, a.src);
        std::copy_n(plan->dst.data() + b, a.n, a.dst);
        std::copy_n(plan->id.data() + b, a.n, a.id);
        if ((e = launch(tables && few && l0 == 0)) != cudaSuccess)
          return cuda_fail(e, "move_blocks launch");
      }
    }
    return PA_OK;
  };
  if (few) {
    MoveArgs<kFewMoves> a;
    if ((rc = run(a, kFewMoves))) return rc;
  } else {
    MoveArgs<kMaxMoves> a;
    if ((rc = run(a, kMaxMoves))) return rc;
  }
  if (listed) {
    const int64_t total = block_tables->shape[0] * block_tables->shape[1];
    const unsigned blocks = static_cast<unsigned>(
        std::min<int64_t>((total + kThreads - 1) / kThreads, 152 * 8));
    rename_kernel<<<blocks, kThreads, 0, st>>>(
        static_cast<int32_t*>(block_tables->data), block_tables->shape[0],
        static_cast<int>(block_tables->shape[1]), block_tables->stride[0], plan->num_blocks,
        static_cast<int>(n), old_ids, new_ids, position);
    if ((e = cudaGetLastError()) != cudaSuccess) return cuda_fail(e, "block table rename launch");
  }
  return PA_OK;
}

}  // extern "C"
