// Rows to e4m3 with a scale for each block of 128 columns: on their own, or written into
// a paged cache; and cache rows back in 16 or 32 bits.
//
// Bound by memory: each element is read once and written once.
// - Rounding. A code is the e4m3 value nearest to the real quotient x / scale. The fp32
//   quotient alone may have been rounded onto (or across) the middle between two codes, so
//   its remainder, which one fma gives exactly, is kept as a sticky last bit: the quotient
//   rounded to odd, which then rounds to e4m3 as the real one does. With a power of two as
//   the scale the quotient is exact already.
// - The split. Half a warp owns a block: 16 lanes of 8 values, the largest magnitude found
//   by four shuffles on the bit patterns, as integers, which order a NaN above everything.

#include <cuda_fp8.h>

#include "indexer_common.cuh"

namespace indexer_gb300 {
namespace {

constexpr int kThreads = 256;
constexpr int kBlockLanes = 16;                     // lanes of one block
constexpr int kLaneValues = INDEXER_BLOCK / kBlockLanes;  // values of one lane: 8
constexpr uint32_t kAmaxFloorBits = (127u - 64u) << 23;   // 2^-64
constexpr uint32_t kInfBits = 0x7f800000u;

// Slots outside the cache that were met (see indexer_guard_hits).
__device__ unsigned int g_guard_hits;

struct QuantParams {
  const void* x;
  uint8_t* codes;
  float* scales;
  const int32_t* slots;   // nullptr: row r goes to row r
  const float* weights;   // nullptr: scales as they are
  int64_t x_ts, x_hs;
  int64_t code_ps, code_ts, scale_ps, scale_ts;
  int64_t units;          // rows * blocks of a row
  int64_t capacity;       // slots of the cache
  int32_t heads, dim, blocks, page_size, pow2;
};

__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// x / scale rounded to odd: exact, or with its last bit set and between the same two
// 24-bit neighbours as the real quotient. `inv` is 1 / scale.
__device__ __forceinline__ float quotient_to_odd(float x, float scale, float inv) {
  float q = x * inv;
  q = fmaf(fmaf(-q, scale, x), inv, q);
  const float rest = fmaf(-q, scale, x);
  uint32_t bits = __float_as_uint(q);
  if (rest != 0.0f) {
    bits -= (bits ^ __float_as_uint(rest)) >> 31;  // the rest points to zero: the lower neighbour
    bits |= 1u;
  }
  return __uint_as_float(bits);
}

// VEC: a lane's values are 8 consecutive columns, loaded 16 bytes at a time and stored as 8
// bytes; otherwise columns lane, lane + 16, ... one by one.
template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads) quantise_kernel(const QuantParams p) {
  begin_after_prior_grids();
  const int lane = threadIdx.x % kBlockLanes;
  const T* x = static_cast<const T*>(p.x);
  const int64_t stride = static_cast<int64_t>(gridDim.x) * (kThreads / kBlockLanes);
  // both halves of a warp run the same number of rounds (the shuffles name the whole warp)
  const int64_t first = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) / kBlockLanes;
  for (int64_t u0 = first & ~int64_t(1); u0 < p.units; u0 += stride) {
    const int64_t u = u0 + (first & 1);
    const bool live = u < p.units;
    const int64_t row = live ? u / p.blocks : 0;
    const int kb = live ? static_cast<int>(u - row * p.blocks) : 0;
    const int64_t t = row / p.heads;
    const T* src = x + t * p.x_ts + (row - t * p.heads) * p.x_hs + kb * INDEXER_BLOCK;
    const int cols = live ? min(p.dim - kb * INDEXER_BLOCK, INDEXER_BLOCK) : 0;
    float v[kLaneValues];
    if constexpr (VEC) {
      constexpr int kV = 16 / sizeof(T);
      if (lane * kLaneValues < cols) {
#pragma unroll
        for (int i = 0; i < kLaneValues / kV; ++i) {
          const Pack<T, kV> a = *reinterpret_cast<const Pack<T, kV>*>(src + lane * kLaneValues + i * kV);
#pragma unroll
          for (int j = 0; j < kV; ++j) v[i * kV + j] = to_float(a.v[j]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < kLaneValues; ++i) v[i] = 0.0f;
      }
    } else {
#pragma unroll
      for (int i = 0; i < kLaneValues; ++i) {
        const int c = lane + i * kBlockLanes;
        v[i] = c < cols ? to_float(src[c]) : 0.0f;
      }
    }
    uint32_t top = kAmaxFloorBits;
#pragma unroll
    for (int i = 0; i < kLaneValues; ++i) top = max(top, __float_as_uint(v[i]) & 0x7fffffffu);
#pragma unroll
    for (int d = kBlockLanes / 2; d > 0; d /= 2) top = max(top, __shfl_xor_sync(0xffffffffu, top, d));
    if (!live) continue;

    int64_t slot = row;
    if (p.slots != nullptr) {
      slot = p.slots[row];
      if (slot < 0 || slot >= p.capacity) {
        if (slot != -1 && lane == 0 && kb == 0) atomicAdd(&g_guard_hits, 1u);
        continue;
      }
    }
    const int64_t page = slot / p.page_size, off = slot - page * p.page_size;
    uint8_t* code = p.codes + page * p.code_ps + off * p.code_ts + kb * INDEXER_BLOCK;

    float scale;
    uint32_t c8[kLaneValues / 2];
    if (top >= kInfBits) {
      scale = __uint_as_float(0x7fffffffu);
#pragma unroll
      for (int i = 0; i < kLaneValues / 2; ++i) c8[i] = 0x7f7fu;
    } else if (p.pow2) {
      // amax = m 2^e, 1 <= m < 2: 448 = 1.75 * 2^8, so 2^(e-8) while m <= 1.75, else 2^(e-7)
      const uint32_t e = (top >> 23) - 8u + ((top & 0x7fffffu) > 0x600000u ? 1u : 0u);
      scale = __uint_as_float(e << 23);
      const float inv = __uint_as_float((254u - e) << 23);
#pragma unroll
      for (int i = 0; i < kLaneValues / 2; ++i) c8[i] = e4m3x2(v[2 * i] * inv, v[2 * i + 1] * inv);
    } else {
      scale = __fdiv_rn(__uint_as_float(top), 448.0f);
      const float inv = __frcp_rn(scale);
#pragma unroll
      for (int i = 0; i < kLaneValues / 2; ++i)
        c8[i] = e4m3x2(quotient_to_odd(v[2 * i], scale, inv), quotient_to_odd(v[2 * i + 1], scale, inv));
    }
    if constexpr (VEC) {
      if (lane * kLaneValues < cols)
        *reinterpret_cast<uint2*>(code + lane * kLaneValues) =
            make_uint2(c8[0] | c8[1] << 16, c8[2] | c8[3] << 16);
    } else {
#pragma unroll
      for (int i = 0; i < kLaneValues; ++i) {
        const int c = lane + i * kBlockLanes;
        if (c < cols) code[c] = static_cast<uint8_t>(c8[i / 2] >> (8 * (i & 1)));
      }
    }
    if (lane == 0)
      p.scales[page * p.scale_ps + off * p.scale_ts + kb] =
          p.weights != nullptr ? p.weights[row] * scale : scale;
  }
}

struct ReadParams {
  const uint8_t* codes;
  const float* scales;
  const int32_t* slots;
  void* out;
  int64_t code_ps, code_ts, scale_ps, scale_ts;
  int64_t units;     // rows * items of a row
  int64_t capacity;
  int32_t dim, items, page_size;
};

// VEC: an item is 8 columns (8 bytes in, 16 or 32 out); otherwise one column.
template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads) read_kernel(const ReadParams p) {
  constexpr int kV = VEC ? 8 : 1;
  begin_after_prior_grids();
  T* out = static_cast<T*>(p.out);
  for (int64_t u = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; u < p.units;
       u += static_cast<int64_t>(gridDim.x) * kThreads) {
    const int64_t row = u / p.items;
    const int item = static_cast<int>(u - row * p.items);
    const int col = item * kV;
    const int64_t slot = p.slots[row];
    const bool inside = slot >= 0 && slot < p.capacity;
    if (!inside && slot != -1 && item == 0) atomicAdd(&g_guard_hits, 1u);
    float f = 0.0f;
    Pack<uint8_t, kV> c = {};
    if (inside) {
      const int64_t page = slot / p.page_size, off = slot - page * p.page_size;
      c = *reinterpret_cast<const Pack<uint8_t, kV>*>(p.codes + page * p.code_ps + off * p.code_ts + col);
      f = p.scales[page * p.scale_ps + off * p.scale_ts + col / INDEXER_BLOCK];
    }
    T y[kV];
#pragma unroll
    for (int i = 0; i < kV; ++i) {
      const __half_raw h = __nv_cvt_fp8_to_halfraw(c.v[i], __NV_E4M3);
      y[i] = from_float<T>(__half2float(__half(h)) * f);
    }
    constexpr int kS = kV * sizeof(T) < 16 ? kV : 16 / sizeof(T);
#pragma unroll
    for (int i = 0; i < kV / kS; ++i) {
      Pack<T, kS> o;
#pragma unroll
      for (int j = 0; j < kS; ++j) o.v[j] = y[i * kS + j];
      *reinterpret_cast<Pack<T, kS>*>(out + row * p.dim + col + i * kS) = o;
    }
  }
}

unsigned grid_for(int64_t threads, int sms) {
  const int64_t blocks = (threads + kThreads - 1) / kThreads, most = int64_t(sms) * 8;
  return static_cast<unsigned>(blocks < most ? blocks : most);
}

template <typename T>
cudaError_t launch_quantise(const QuantParams& p, bool vec, int sms, cudaStream_t stream) {
  const unsigned grid = grid_for((p.units + 1) / 2 * 2 * kBlockLanes, sms);
  return vec ? launch(quantise_kernel<T, true>, grid, kThreads, 0, stream, p)
             : launch(quantise_kernel<T, false>, grid, kThreads, 0, stream, p);
}

int run_quantise(QuantParams p, int32_t dtype, int64_t rows, cudaStream_t stream) {
  int sms = 0;
  cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return status_of(e);
  p.blocks = (p.dim + INDEXER_BLOCK - 1) / INDEXER_BLOCK;
  p.units = rows * p.blocks;
  // rows a constant step apart need no division
  if (p.heads > 1 && p.x_ts == p.heads * p.x_hs) {
    p.x_ts = p.x_hs;
    p.heads = 1;
  }
  const int64_t values = static_cast<int64_t>(16 / dtype_bytes(dtype));
  const bool vec = p.dim % kLaneValues == 0 && p.x_ts % values == 0 && p.x_hs % values == 0 &&
                   (reinterpret_cast<uintptr_t>(p.x) & 15u) == 0 &&
                   p.code_ts % 8 == 0 && p.code_ps % 8 == 0 &&
                   (reinterpret_cast<uintptr_t>(p.codes) & 7u) == 0;
  if (dtype == INDEXER_BF16) e = launch_quantise<__nv_bfloat16>(p, vec, sms, stream);
  else if (dtype == INDEXER_FP16) e = launch_quantise<__half>(p, vec, sms, stream);
  else e = launch_quantise<float>(p, vec, sms, stream);
  return status_of(e);
}

template <typename T>
cudaError_t launch_read(const ReadParams& p, bool vec, int sms, cudaStream_t stream) {
  const unsigned grid = grid_for(p.units, sms);
  return vec ? launch(read_kernel<T, true>, grid, kThreads, 0, stream, p)
             : launch(read_kernel<T, false>, grid, kThreads, 0, stream, p);
}

bool dtype_ok(int32_t dtype) { return dtype >= INDEXER_BF16 && dtype <= INDEXER_FP32; }

bool aligned(const void* p, size_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

}  // namespace

cudaError_t cache_guard_hits(unsigned int* hits) {
  return cudaMemcpyFromSymbol(hits, g_guard_hits, sizeof(unsigned int));
}

cudaError_t reset_cache_guard_hits() {
  const unsigned int zero = 0;
  return cudaMemcpyToSymbol(g_guard_hits, &zero, sizeof(unsigned int));
}

}  // namespace indexer_gb300

extern "C" {

size_t indexer_cache_bytes(void) { return sizeof(indexer_cache_t); }

int indexer_quantise(const void* x, int64_t x_token_stride, int64_t x_head_stride, int32_t dtype,
                     int64_t tokens, int32_t heads, int32_t dim, int32_t scale_format,
                     const float* weights, uint8_t* codes, float* scales, cudaStream_t stream) {
  using namespace indexer_gb300;
  if (!dtype_ok(dtype) || scale_format < INDEXER_SCALE_FP32 || scale_format > INDEXER_SCALE_POW2)
    return TOPK_ERR_INVALID_ARGUMENT;
  if (tokens < 0 || tokens > INT32_MAX || heads < 0 || dim < 1 || dim > 65536 || x_token_stride < 0 ||
      x_head_stride < 0 || (weights != nullptr && dim > INDEXER_BLOCK))
    return TOPK_ERR_INVALID_ARGUMENT;
  if (tokens == 0 || heads == 0) return TOPK_OK;
  if (x == nullptr || codes == nullptr || scales == nullptr || !aligned(x, dtype_bytes(dtype)) ||
      !aligned(scales, 4) || !aligned(weights, 4))
    return TOPK_ERR_INVALID_ARGUMENT;
  QuantParams p = {};
  p.x = x;
  p.codes = codes;
  p.scales = scales;
  p.weights = weights;
  p.x_ts = tokens > 1 ? x_token_stride : 0;
  p.x_hs = heads > 1 ? x_head_stride : 0;
  p.heads = heads;
  p.dim = dim;
  p.pow2 = scale_format == INDEXER_SCALE_POW2;
  p.page_size = 1;  // row r is page r: its own place in contiguous outputs
  p.code_ps = dim;
  p.scale_ps = (dim + INDEXER_BLOCK - 1) / INDEXER_BLOCK;
  return run_quantise(p, dtype, tokens * heads, stream);
}

int indexer_cache_write(const void* x, int64_t x_token_stride, int32_t dtype, int64_t tokens,
                        const int32_t* slots, int32_t scale_format, const indexer_cache_t* cache,
                        cudaStream_t stream) {
  using namespace indexer_gb300;
  if (!dtype_ok(dtype) || scale_format < INDEXER_SCALE_FP32 || scale_format > INDEXER_SCALE_POW2 ||
      !cache_ok(cache))
    return TOPK_ERR_INVALID_ARGUMENT;
  if (tokens < 0 || tokens > INT32_MAX || x_token_stride < 0) return TOPK_ERR_INVALID_ARGUMENT;
  if (tokens == 0) return TOPK_OK;
  if (x == nullptr || slots == nullptr || !aligned(x, dtype_bytes(dtype)) || !aligned(slots, 4))
    return TOPK_ERR_INVALID_ARGUMENT;
  QuantParams p = {};
  p.x = x;
  p.codes = cache->codes;
  p.scales = cache->scales;
  p.slots = slots;
  p.x_ts = tokens > 1 ? x_token_stride : 0;
  p.heads = 1;
  p.dim = cache->dim;
  p.pow2 = scale_format == INDEXER_SCALE_POW2;
  p.page_size = cache->page_size;
  p.code_ps = cache->num_pages > 1 ? cache->code_page_stride : 0;
  p.code_ts = cache->page_size > 1 ? cache->code_token_stride : 0;
  p.scale_ps = cache->scale_page_stride;
  p.scale_ts = cache->scale_token_stride;
  p.capacity = cache->num_pages * cache->page_size;
  return run_quantise(p, dtype, tokens, stream);
}

int indexer_cache_read(const indexer_cache_t* cache, const int32_t* slots, int64_t rows,
                       int32_t dtype, void* out, cudaStream_t stream) {
  using namespace indexer_gb300;
  if (!dtype_ok(dtype) || !cache_ok(cache) || rows < 0 || rows > INT64_MAX / 65536)
    return TOPK_ERR_INVALID_ARGUMENT;
  if (rows == 0) return TOPK_OK;
  if (slots == nullptr || out == nullptr || !aligned(slots, 4) || !aligned(out, dtype_bytes(dtype)))
    return TOPK_ERR_INVALID_ARGUMENT;
  int sms = 0;
  cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return status_of(e);
  ReadParams p = {};
  p.codes = cache->codes;
  p.scales = cache->scales;
  p.slots = slots;
  p.out = out;
  p.dim = cache->dim;
  p.page_size = cache->page_size;
  p.code_ps = cache->num_pages > 1 ? cache->code_page_stride : 0;
  p.code_ts = cache->page_size > 1 ? cache->code_token_stride : 0;
  p.scale_ps = cache->scale_page_stride;
  p.scale_ts = cache->scale_token_stride;
  p.capacity = cache->num_pages * cache->page_size;
  const bool vec = p.dim % 8 == 0 && p.code_ts % 8 == 0 && p.code_ps % 8 == 0 && aligned(p.codes, 8) &&
                   aligned(out, 16);
  p.items = vec ? p.dim / 8 : p.dim;
  p.units = rows * p.items;
  if (dtype == INDEXER_BF16) e = launch_read<__nv_bfloat16>(p, vec, sms, stream);
  else if (dtype == INDEXER_FP16) e = launch_read<__half>(p, vec, sms, stream);
  else e = launch_read<float>(p, vec, sms, stream);
  return status_of(e);
}

int indexer_guard_hits(uint64_t* hits) {
  using namespace indexer_gb300;
  if (hits == nullptr) return TOPK_ERR_INVALID_ARGUMENT;
  unsigned int a = 0, b = 0;
  cudaError_t e = cache_guard_hits(&a);
  if (e == cudaSuccess) e = scores_guard_hits(&b);
  if (e == cudaSuccess) *hits = static_cast<uint64_t>(a) + b;
  return status_of(e);
}

int indexer_reset_guard_hits(void) {
  using namespace indexer_gb300;
  cudaError_t e = reset_cache_guard_hits();
  if (e == cudaSuccess) e = reset_scores_guard_hits();
  return status_of(e);
}

}  // extern "C"
