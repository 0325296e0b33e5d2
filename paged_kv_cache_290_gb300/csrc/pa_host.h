// Host-side helpers shared by the C ABI's translation units: status messages, argument checks,
// tensor maps of the pools, the side stream.  Defined in pa_api.cu.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>
#include <string>

#include "pa.h"

namespace pa {

// Sets the message pa_last_error() returns on this host thread; returns `code`.
int fail(int code, const std::string& msg);
int cuda_fail(cudaError_t e, const char* what);
void clear_last_error();

const char* dtype_name(int dt);
// Rank, dtype, non-negative shape and strides, unit innermost stride, non-null when non-empty.
int check_tensor(const pa_tensor* t, const char* name, int dtype, int ndim);
int check_contiguous(const pa_tensor* t, const char* name);
bool aligned16(const void* p);
// bfloat16 when the pool says so, else fp16.
int pool_dtype16(const pa_tensor* kc);
// Pools [NB, Hkv, bs, d] of the given dtype: shapes, contiguity, supported d and bs, alignment.
int check_pool(const pa_tensor* kc, const pa_tensor* vc, int dtype);
int check_scales(const pa_kv_scales* sc);

// The pool as a 2-D tensor map (16-row boxes; see pa_api.cu).
int make_pool_map(CUtensorMap* m, void* base, int64_t rows, int d, int dtype);

// A 16-bit pool [NB, Hkv, bs, d] as a 4-D tensor (64 values, bs rows, NB * Hkv tiles, d / 64
// column halves) with boxes of 64 values x 16 rows x 2 adjacent heads x all halves, 128-byte
// swizzle: one copy fetches 16 tokens of a pair of heads as [half][head][16 rows][128 B].
int make_pair_map(CUtensorMap* m, void* base, int64_t tiles, int bs, int d, int dtype);

cudaError_t device_sm_count(int* out);

// Runs `set` once per device for the static `done` it is given (a bit per device): for attributes
// of a kernel that stay set, whose call costs as much as a small launch.
template <typename F>
cudaError_t once_per_device(std::atomic<uint64_t>& done, F set) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? uint64_t{1} << dev : 0;
  if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
  if ((e = set()) == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
  return e;
}

// A side stream and two events per device and host thread, for work beside the caller's stream.
struct SideStream {
  cudaStream_t stream = nullptr;
  cudaEvent_t fork = nullptr, join = nullptr;
};
cudaError_t side_stream(SideStream** out);

// The bounded-wait limit of this host thread's calls (pa_set_wait_limit).
uint64_t wait_limit_ns();

}  // namespace pa
