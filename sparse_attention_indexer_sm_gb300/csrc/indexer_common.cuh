// Shared by the indexer's operators: types in and out, programmatic dependent
// launch, the launch call, and the way to the library's last CUDA error.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <climits>
#include <cstdint>

#include "indexer_ops.h"

namespace topk_gb300 {
// Records a CUDA error for topk_last_cuda_error and returns TOPK_ERR_CUDA (topk_api.cu).
int record_cuda_error(cudaError_t e);
}  // namespace topk_gb300

namespace indexer_gb300 {

// Each source that counts bad slots or pages gives its counter to indexer_guard_hits.
cudaError_t cache_guard_hits(unsigned int* hits);
cudaError_t reset_cache_guard_hits();
cudaError_t scores_guard_hits(unsigned int* hits);
cudaError_t reset_scores_guard_hits();

// Checks a cache's description (nothing in device memory is read).
inline bool cache_ok(const indexer_cache_t* c) {
  if (c == nullptr || c->num_pages < 0 || c->page_size < 1 || c->dim < 1 || c->dim > 65536) return false;
  if (c->num_pages > INT32_MAX / c->page_size) return false;
  if (c->num_pages == 0) return true;
  if (c->codes == nullptr || c->scales == nullptr) return false;
  if ((reinterpret_cast<uintptr_t>(c->scales) & 3u) != 0) return false;
  const int64_t nb = (c->dim + INDEXER_BLOCK - 1) / INDEXER_BLOCK;
  const bool tokens = c->page_size > 1, pages = c->num_pages > 1;
  return (!tokens || (c->code_token_stride >= c->dim && c->scale_token_stride >= nb)) &&
         (!pages || (c->code_page_stride >= c->dim && c->scale_page_stride >= nb));
}

// Division of numbers below 2^31 by a constant of the launch: n / d = (n * magic) >> (31 + shift).
struct Divisor {
  uint32_t d, magic, shift;
};

inline Divisor divisor(int64_t d) {
  Divisor r = {static_cast<uint32_t>(d), 0, 0};
  while ((int64_t(1) << r.shift) < d) ++r.shift;
  r.magic = static_cast<uint32_t>(((uint64_t(1) << (31 + r.shift)) + d - 1) / d);
  return r;
}

inline size_t dtype_bytes(int32_t dtype) { return dtype == INDEXER_FP32 ? 4u : 2u; }

// The SM count of the current device, asked once for each device.
inline cudaError_t sm_count(int* out) {
  static thread_local int known_device = -1, known_count = 0;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev != known_device) {
    e = cudaDeviceGetAttribute(&known_count, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    known_device = dev;
  }
  *out = known_count;
  return cudaSuccess;
}

template <typename... Args>
cudaError_t launch(void (*kernel)(Args...), unsigned grid, unsigned threads, size_t smem,
                   cudaStream_t stream, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, 1, 1);
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

inline int status_of(cudaError_t e) {
  return e == cudaSuccess ? TOPK_OK : topk_gb300::record_cuda_error(e);
}

#ifdef __CUDACC__

__device__ __forceinline__ uint32_t quotient(const Divisor& d, uint32_t n) {
  return static_cast<uint32_t>((static_cast<uint64_t>(n) * d.magic) >> 31 >> d.shift);
}

// Programmatic dependent launch: the next kernel of the stream may be scheduled from
// here on, and nothing of the previous one is read or overwritten before it has ended.
__device__ __forceinline__ void begin_after_prior_grids() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_float(__half v) { return __half2float(v); }
template <typename T> __device__ __forceinline__ T from_float(float v);
template <> __device__ __forceinline__ float from_float<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}
template <> __device__ __forceinline__ __half from_float<__half>(float v) { return __float2half_rn(v); }

// N consecutive values at once, through one access of their size (at most 16 bytes each)
template <typename T, int N> struct alignas(sizeof(T) * N < 16 ? sizeof(T) * N : 16) Pack {
  T v[N];
};

// 32 bytes in one access, on a boundary of 32.
__device__ __forceinline__ void store32(void* p, const uint32_t (&v)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]),
               "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

#endif  // __CUDACC__

}  // namespace indexer_gb300
