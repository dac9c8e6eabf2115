// Rows to e4m3 with a scale for each block of 128 columns: on their own, or written into
// a paged cache; and cache rows back in 16 or 32 bits.
//
// Bound by memory: each element is read once and written once, so few operations may be spent on one.
// - Rounding. A code is the e4m3 value nearest to the real quotient x / scale. x times an approximate
//   1 / scale, a little too small and a little too large, gives two codes with one instruction for
//   each pair; where they agree, the code is that, and almost everywhere they do. Where they do not, a 16-bit
//   value lies on a border between codes up to the scale's own rounding, whose sign decides. A 32-bit
//   value's remainder, which one fma gives exactly, becomes a sticky last bit: the quotient rounded to
//   odd, which rounds to e4m3 as the real one does. With a power of two as the scale the quotient is exact.
// - The split. Eight lanes own a block, 16 values each: with sixteen lanes of 8 values what a lane does once a
//   block (its place, its scale) cost as much as its values, and the kernel was bound by instructions
//   (8192 x 64 rows of 128 in bf16: 60 us against 35). The largest magnitude is found on the bit patterns, as
//   integers, which order a NaN above everything. In 32 bits the same rows take 51 us, 97% of the copy rate; a
//   width that is no multiple of 8 is read and written value by value (rows of 63: 48 us, three times its
//   floor).
//   Reading back, a lane makes one 32-byte store of 16 or 8 columns (or 16-byte store of 8); eight CTAs an SM
//   hide the loads' latency, which four rows in flight in each of fewer lanes did not (524288 rows of 512 to
//   bf16: 131 against 203 us).

#include <cuda_fp8.h>

#include <cstring>
#include <initializer_list>

#include "indexer_common.cuh"

namespace indexer_gb300 {
namespace {

constexpr int kThreads = 256;
constexpr int kBlockLanes = 8;                            // lanes of one block
constexpr int kLaneValues = INDEXER_BLOCK / kBlockLanes;  // values of one lane: 16, in two pieces of 8 columns
constexpr int kPiece = 8;
constexpr int kPieces = kLaneValues / kPiece;
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
  uint32_t units;         // rows * blocks of a row
  uint32_t capacity;      // slots of the cache
  Divisor heads, blocks, page_size;
  int32_t dim, pow2;
};

__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// top / 448, correctly rounded (Markstein: a quotient from the correctly rounded reciprocal, corrected once by its
// exact remainder).
__device__ __forceinline__ float over_448(float top) {
  const float y = 1.0f / 448.0f, q = top * y;
  return fmaf(fmaf(-448.0f, q, top), y, q);
}

// 1 / scale to within a step: scales lie between 2^-73 and 2^120.
__device__ __forceinline__ float about_inverse(float scale) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(scale));
  return r;
}

// The bit pattern of the largest magnitude among a block's values, NaN above everything, as fp32.
template <typename T>
__device__ __forceinline__ uint32_t block_top(const uint32_t (&bits)[kLaneValues * sizeof(T) / 4]) {
  constexpr int kWords = kLaneValues * sizeof(T) / 4;
  constexpr uint32_t kAbs = sizeof(T) == 4 ? 0x7fffffffu : 0x7fff7fffu;
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < kWords; i += 2) {  // pairs of 16 bits order as integers too
    const uint32_t a = bits[i] & kAbs, b = bits[i + 1] & kAbs;
    if constexpr (sizeof(T) == 4) top = __vimax3_u32(top, a, b);
    else top = __vimax3_u16x2(top, a, b);
  }
#pragma unroll
  for (int d = kBlockLanes / 2; d > 0; d /= 2) {
    const uint32_t other = __shfl_xor_sync(0xffffffffu, top, d);
    if constexpr (sizeof(T) == 4) top = max(top, other);
    else top = __vmaxu2(top, other);
  }
  if constexpr (sizeof(T) == 4) {
    return top;
  } else {
    const unsigned short raw = static_cast<unsigned short>(max(top & 0xffffu, top >> 16));
    T v;
    memcpy(&v, &raw, 2);
    return __float_as_uint(to_float(v));
  }
}

// Codes of two values, as 16 bits, from their products with a number near 1 / scale.
__device__ __forceinline__ uint32_t codes_of(const float* v, float inv) { return e4m3x2(v[0] * inv, v[1] * inv); }

// VEC: a lane's pieces are 8 consecutive columns each, loaded 16 bytes at a time and stored as 8
// bytes; otherwise its columns are lane, lane + 8, ... one by one. SLOTS: row r goes to slots[r].
template <typename T, bool VEC, bool SLOTS>
__global__ void __launch_bounds__(kThreads) quantise_kernel(const QuantParams p) {
  constexpr int kWords = kLaneValues * sizeof(T) / 4, kPieceWords = kWords / kPieces;
  begin_after_prior_grids();
  const int lane = threadIdx.x % kBlockLanes;
  const T* x = static_cast<const T*>(p.x);
  // all groups of lanes of a warp run the same number of rounds (the shuffles name the whole warp)
  constexpr uint32_t kGroups = 32 / kBlockLanes;
  const uint32_t group = (blockIdx.x * kThreads + threadIdx.x) / kBlockLanes;
  for (uint32_t u0 = group / kGroups * kGroups; u0 < p.units; u0 += gridDim.x * (kThreads / kBlockLanes)) {
    uint32_t bits[kWords];
    const uint32_t u = u0 + group % kGroups;
    const bool live = u < p.units;
    const uint32_t row = live ? quotient(p.blocks, u) : 0;
    const uint32_t kb = live ? u - row * p.blocks.d : 0;
    const int cols = live ? min(p.dim - static_cast<int>(kb) * INDEXER_BLOCK, INDEXER_BLOCK) : 0;
    int32_t slot_id = -1;
    if constexpr (SLOTS) slot_id = live ? p.slots[row] : -1;  // on its way with the row
    const uint32_t t = SLOTS ? row : quotient(p.heads, row);  // a cache's rows have no heads
    const T* src = x + t * p.x_ts + (SLOTS ? 0 : (row - t * p.heads.d) * p.x_hs) + kb * INDEXER_BLOCK;
#pragma unroll
    for (int i = 0; i < kWords; ++i) bits[i] = 0;
    if constexpr (VEC) {
#pragma unroll
      for (int q = 0; q < kPieces; ++q) {
        const int c = (q * kBlockLanes + lane) * kPiece;
        if (c < cols) {
#pragma unroll
          for (int i = 0; i < kPieceWords / 4; ++i) {
            const uint4 a = reinterpret_cast<const uint4*>(src + c)[i];
            uint32_t* w = &bits[q * kPieceWords + 4 * i];
            w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
          }
        }
      }
    } else {
      T v[kLaneValues];
#pragma unroll
      for (int i = 0; i < kLaneValues; ++i) {
        const int c = lane + i * kBlockLanes;
        v[i] = c < cols ? src[c] : from_float<T>(0.0f);
      }
      memcpy(bits, v, sizeof(v));
    }
    const uint32_t top = max(block_top<T>(bits), kAmaxFloorBits);
    if (cols == 0) continue;
    uint8_t* code;
    float* scale_at;
    if constexpr (SLOTS) {
      const uint32_t slot = static_cast<uint32_t>(slot_id);
      if (slot >= p.capacity) {  // negative ones too
        if (slot_id != -1 && lane == 0 && kb == 0) atomicAdd(&g_guard_hits, 1u);
        continue;
      }
      const uint32_t page = quotient(p.page_size, slot), off = slot - page * p.page_size.d;
      code = p.codes + page * p.code_ps + off * p.code_ts + kb * INDEXER_BLOCK;
      scale_at = p.scales + page * p.scale_ps + off * p.scale_ts + kb;
    } else {
      code = p.codes + row * static_cast<int64_t>(p.dim) + kb * INDEXER_BLOCK;
      scale_at = p.scales + (row * static_cast<int64_t>(p.blocks.d) + kb);
    }

    T typed[kLaneValues];
    float v[kLaneValues], scale;
    memcpy(typed, bits, sizeof(typed));
#pragma unroll
    for (int i = 0; i < kLaneValues; ++i) v[i] = to_float(typed[i]);
    uint32_t c[kLaneValues / 4];  // four codes each
    if (top >= kInfBits) {
      scale = __uint_as_float(0x7fffffffu);
#pragma unroll
      for (int i = 0; i < kLaneValues / 4; ++i) c[i] = 0x7f7f7f7fu;
    } else if (p.pow2) {
      // amax = m 2^e, 1 <= m < 2: 448 = 1.75 * 2^8, so 2^(e-8) while m <= 1.75, else 2^(e-7)
      const uint32_t e = (top >> 23) - 8u + ((top & 0x7fffffu) > 0x600000u ? 1u : 0u);
      scale = __uint_as_float(e << 23);
      const float inv = __uint_as_float((254u - e) << 23);
#pragma unroll
      for (int i = 0; i < kLaneValues / 4; ++i) c[i] = codes_of(&v[4 * i], inv) | codes_of(&v[4 * i + 2], inv) << 16;
    } else {
      scale = over_448(__uint_as_float(top));
      // the two quotients enclose the real one by 2^-22 or more on each side
      const float inv = about_inverse(scale), low = inv * (1.0f - 0x1p-21f), high = inv * (1.0f + 0x1p-21f);
      // Of 16-bit values, x / amax has numerator and denominator below 2^11, a border between codes 2^5: it lies on
      // the border or 2^-16 of it away. So where the codes differ (by one, then), x * 448 / amax is on the border,
      // and x / scale is where the rounding of the scale has put it: above, below, or on it (to the even code).
      const float rest = fmaf(-448.0f, scale, __uint_as_float(top));
      [[maybe_unused]] const uint32_t up = rest > 0.0f ? 0x01010101u : 0u, even = rest == 0.0f ? 0x01010101u : 0u;
#pragma unroll
      for (int i = 0; i < kLaneValues / 4; ++i) {
        c[i] = codes_of(&v[4 * i], low) | codes_of(&v[4 * i + 2], low) << 16;
        const uint32_t differ = c[i] ^ (codes_of(&v[4 * i], high) | codes_of(&v[4 * i + 2], high) << 16);
        if constexpr (sizeof(T) == 2) {
          c[i] += differ & (up | (c[i] & even));
        } else if (differ != 0u) {
          c[i] = e4m3x2(quotient_to_odd(v[4 * i], scale, inv), quotient_to_odd(v[4 * i + 1], scale, inv)) |
                 e4m3x2(quotient_to_odd(v[4 * i + 2], scale, inv), quotient_to_odd(v[4 * i + 3], scale, inv)) << 16;
        }
      }
    }
    if constexpr (VEC) {
#pragma unroll
      for (int q = 0; q < kPieces; ++q) {
        const int col = (q * kBlockLanes + lane) * kPiece;
        if (col < cols) *reinterpret_cast<uint2*>(code + col) = make_uint2(c[2 * q], c[2 * q + 1]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < kLaneValues; ++i) {
        const int col = lane + i * kBlockLanes;
        if (col < cols) code[col] = static_cast<uint8_t>(c[i / 4] >> (8 * (i & 3)));
      }
    }
    if (lane == 0) {
      if constexpr (SLOTS) *scale_at = scale;
      else *scale_at = p.weights != nullptr ? p.weights[row] * scale : scale;
    }
  }
}

struct ReadParams {
  const uint8_t* codes;
  const float* scales;
  const int32_t* slots;
  void* out;
  int64_t code_ps, code_ts, scale_ps, scale_ts;
  uint32_t units;     // rows * items of a row
  uint32_t capacity;
  Divisor items, page_size;
  int32_t dim;
};

// An item is V columns of a row: V * sizeof(T) = 32 or 16 bytes of output in one store, or one column (V = 1).
template <typename T, int V>
__global__ void __launch_bounds__(kThreads, 8) read_kernel(const ReadParams p) {
  begin_after_prior_grids();
  T* out = static_cast<T*>(p.out);
  for (uint32_t u = blockIdx.x * kThreads + threadIdx.x; u < p.units; u += gridDim.x * kThreads) {
    const uint32_t row = quotient(p.items, u), col = (u - row * p.items.d) * V;
    const int32_t slot = p.slots[row];
    float f = 0.0f;
    Pack<uint8_t, V> c = {};
    if (static_cast<uint32_t>(slot) < p.capacity) {
      const uint32_t page = quotient(p.page_size, slot), off = slot - page * p.page_size.d;
      c = *reinterpret_cast<const Pack<uint8_t, V>*>(p.codes + page * p.code_ps + off * p.code_ts + col);
      f = p.scales[page * p.scale_ps + off * p.scale_ts + col / INDEXER_BLOCK];
    } else if (slot != -1 && col == 0) {
      atomicAdd(&g_guard_hits, 1u);
    }
    T* dst = out + static_cast<int64_t>(row) * p.dim + col;
    if constexpr (V == 1) {
      *dst = from_float<T>(__half2float(__half(__nv_cvt_fp8_to_halfraw(c.v[0], __NV_E4M3))) * f);
    } else {
      T y[V];
#pragma unroll
      for (int i = 0; i < V / 2; ++i) {
        const __nv_fp8x2_storage_t two = static_cast<__nv_fp8x2_storage_t>(c.v[2 * i] | c.v[2 * i + 1] << 8);
        const float2 v = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(two, __NV_E4M3)));
        y[2 * i] = from_float<T>(v.x * f);
        y[2 * i + 1] = from_float<T>(v.y * f);
      }
      if constexpr (V * sizeof(T) == 32) {
        uint32_t words[8];
        memcpy(words, y, sizeof(words));
        store32(dst, words);
      } else {
        uint4 words;
        memcpy(&words, y, sizeof(words));
        *reinterpret_cast<uint4*>(dst) = words;
      }
    }
  }
}

// Four times the CTAs that an SM holds, at most: enough rounds to even out uneven ones, few enough to keep a
// CTA's start cheap (65535 rows of 576 written: 23.3 us with one time, 22.1 with four, 23.4 with eight; 524288
// rows of 512 read: 140 us with two, 132 with four).
unsigned grid_for(int64_t threads, int sms) {
  const int64_t blocks = (threads + kThreads - 1) / kThreads, most = int64_t(sms) * 32;
  return static_cast<unsigned>(blocks < most ? blocks : most);
}

template <typename T>
cudaError_t launch_quantise(const QuantParams& p, bool vec, int sms, cudaStream_t stream) {
  constexpr int64_t kWarpUnits = 32 / kBlockLanes;
  const unsigned grid = grid_for((static_cast<int64_t>(p.units) + kWarpUnits - 1) / kWarpUnits * 32, sms);
  if (p.slots != nullptr)
    return vec ? launch(quantise_kernel<T, true, true>, grid, kThreads, 0, stream, p)
               : launch(quantise_kernel<T, false, true>, grid, kThreads, 0, stream, p);
  return vec ? launch(quantise_kernel<T, true, false>, grid, kThreads, 0, stream, p)
             : launch(quantise_kernel<T, false, false>, grid, kThreads, 0, stream, p);
}

// The kernels number rows' parts in 31 bits: longer calls are cut into launches of so many rows.
int64_t rows_of_launch(int64_t parts_of_row) { return (INT64_C(1) << 30) / parts_of_row; }

// heads: rows of a token (one slot, or `heads` rows in a row of the outputs).
int run_quantise(QuantParams p, int32_t dtype, int64_t tokens, int64_t heads, cudaStream_t stream) {
  int sms = 0;
  cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return status_of(e);
  const int64_t blocks = (p.dim + INDEXER_BLOCK - 1) / INDEXER_BLOCK;
  p.blocks = divisor(blocks);
  // rows a constant step apart need no division
  if (heads > 1 && p.x_ts == heads * p.x_hs && tokens * heads <= INT32_MAX) {
    tokens *= heads;
    p.x_ts = p.x_hs;
    heads = 1;
  }
  const int64_t values = static_cast<int64_t>(16 / dtype_bytes(dtype));
  const bool vec = p.dim % kPiece == 0 && p.x_ts % values == 0 && p.x_hs % values == 0 &&
                   (reinterpret_cast<uintptr_t>(p.x) & 15u) == 0 &&
                   p.code_ts % 8 == 0 && p.code_ps % 8 == 0 &&
                   (reinterpret_cast<uintptr_t>(p.codes) & 7u) == 0;
  if (heads > rows_of_launch(blocks)) return TOPK_ERR_INVALID_ARGUMENT;
  p.heads = divisor(heads);
  const int64_t step = rows_of_launch(blocks * heads);
  for (int64_t t = 0; t < tokens; t += step) {
    const int64_t n = tokens - t < step ? tokens - t : step;
    p.units = static_cast<uint32_t>(n * heads * blocks);
    if (dtype == INDEXER_BF16) e = launch_quantise<__nv_bfloat16>(p, vec, sms, stream);
    else if (dtype == INDEXER_FP16) e = launch_quantise<__half>(p, vec, sms, stream);
    else e = launch_quantise<float>(p, vec, sms, stream);
    if (e != cudaSuccess) return status_of(e);
    p.x = static_cast<const char*>(p.x) + n * p.x_ts * static_cast<int64_t>(dtype_bytes(dtype));
    if (p.slots != nullptr) {
      p.slots += n;
    } else {
      p.codes += n * heads * p.code_ts;
      p.scales += n * heads * p.scale_ts;
    }
    if (p.weights != nullptr) p.weights += n * heads;
  }
  return TOPK_OK;
}

template <typename T>
cudaError_t launch_read(const ReadParams& p, int columns, int sms, cudaStream_t stream) {
  const unsigned grid = grid_for(p.units, sms);
  constexpr int kWide = 32 / sizeof(T);
  if (columns == kWide) return launch(read_kernel<T, kWide>, grid, kThreads, 0, stream, p);
  if constexpr (kWide > 8) {
    if (columns == 8) return launch(read_kernel<T, 8>, grid, kThreads, 0, stream, p);
  }
  return launch(read_kernel<T, 1>, grid, kThreads, 0, stream, p);
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
  p.dim = dim;
  p.pow2 = scale_format == INDEXER_SCALE_POW2;
  p.code_ts = dim;  // contiguous outputs
  p.scale_ts = (dim + INDEXER_BLOCK - 1) / INDEXER_BLOCK;
  return run_quantise(p, dtype, tokens, heads, stream);
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
  p.dim = cache->dim;
  p.pow2 = scale_format == INDEXER_SCALE_POW2;
  p.page_size = divisor(cache->page_size);
  p.code_ps = cache->num_pages > 1 ? cache->code_page_stride : 0;
  p.code_ts = cache->page_size > 1 ? cache->code_token_stride : 0;
  p.scale_ps = cache->scale_page_stride;
  p.scale_ts = cache->scale_token_stride;
  p.capacity = static_cast<uint32_t>(cache->num_pages * cache->page_size);
  return run_quantise(p, dtype, tokens, 1, stream);
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
  p.page_size = divisor(cache->page_size);
  p.code_ps = cache->num_pages > 1 ? cache->code_page_stride : 0;
  p.code_ts = cache->page_size > 1 ? cache->code_token_stride : 0;
  p.scale_ps = cache->scale_page_stride;
  p.scale_ts = cache->scale_token_stride;
  p.capacity = static_cast<uint32_t>(cache->num_pages * cache->page_size);
  // Columns of an item: a 32-byte store where rows start on 32 bytes, or eight, or one (239616 rows of 200 to
  // bf16: eight 27 us, one 111).
  const int32_t wide = 32 / static_cast<int32_t>(dtype_bytes(dtype));
  auto fits = [&](int32_t n) {
    return p.dim % n == 0 && p.code_ts % n == 0 && p.code_ps % n == 0 && aligned(p.codes, n) &&
           aligned(out, n * dtype_bytes(dtype));
  };
  const int32_t columns = fits(wide) ? wide : fits(8) ? 8 : 1;
  const int32_t items = p.dim / columns;
  p.items = divisor(items);
  const int64_t step = rows_of_launch(items);
  for (int64_t r = 0; r < rows; r += step) {
    const int64_t n = rows - r < step ? rows - r : step;
    p.units = static_cast<uint32_t>(n * items);
    if (dtype == INDEXER_BF16) e = launch_read<__nv_bfloat16>(p, columns, sms, stream);
    else if (dtype == INDEXER_FP16) e = launch_read<__half>(p, columns, sms, stream);
    else e = launch_read<float>(p, columns, sms, stream);
    if (e != cudaSuccess) return status_of(e);
    p.slots += n;
    p.out = static_cast<char*>(p.out) + n * p.dim * static_cast<int64_t>(dtype_bytes(dtype));
  }
  return TOPK_OK;
}

int indexer_guard_hits(uint64_t* hits) {
  using namespace indexer_gb300;
  if (hits == nullptr) return TOPK_ERR_INVALID_ARGUMENT;
  // the copies below are ordered behind the default stream alone, not behind non-blocking ones
  cudaError_t e = cudaDeviceSynchronize();
  uint64_t sum = 0;
  for (const auto count : {cache_guard_hits, scores_guard_hits, rotary_guard_hits, append_guard_hits, attention_guard_hits}) {
    unsigned int n = 0;
    if (e == cudaSuccess) e = count(&n);
    sum += n;
  }
  if (e == cudaSuccess) *hits = sum;
  return status_of(e);
}

int indexer_reset_guard_hits(void) {
  using namespace indexer_gb300;
  cudaError_t e = cudaDeviceSynchronize();
  for (const auto reset : {reset_cache_guard_hits, reset_scores_guard_hits, reset_rotary_guard_hits, reset_append_guard_hits,
                           reset_attention_guard_hits})
    if (e == cudaSuccess) e = reset();
  return status_of(e);
}

}  // extern "C"
