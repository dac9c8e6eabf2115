// Rows appended to a paged cache of e4m3 codes with one scale for each block of tokens and head.
//
// A block's scale is the smallest power of two that brings its largest value to 448 or less. Tokens come a few at a time,
// so a block that has rows from before keeps its scale unless the new rows need a larger one; then the older codes
// are rounded once more, to old / new of what they were. That quotient is a power of two: codes that stay normal numbers
// lose nothing that the new rows' precision has, whereas a scale of 24 bits would move every one of them. A scale that something
// else has written may be any number: products and quotients are then rounded to odd before they become codes, which
// rounds them as the real ones.
//
// Bound by memory: rows are read once and codes written once. A warp, or the eight of a CTA, owns the part of one block
// and head that a call appends, holds its rows in registers (the first eight of a lane, or four; more than those are read
// again), agrees on the largest magnitude and writes. So nothing is exchanged between owners, and no order matters.
// An owner's rows are behind the lengths of its sequence, which it finds among all by steps of 32 at once; and its page and
// old scale are asked for with the rows.
// Measured: 41000 rows of 8 heads of 128 in bf16 onto eight sequences 26 us (127 MB: 19 us at the copy rate), a token on each
// of 256 sequences 4.5 us, a chain of four dependent loads (starts, lengths, page, scale and codes) around a launch. Rows that start
// on no 16-byte boundary are read value by value, and 16-bit ones spill some registers: 43 us (fp16 47) and 5.2 (5.9).

#include <cuda_fp8.h>

#include "indexer_common.cuh"

namespace indexer_gb300 {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kPiece = 8;                                // columns of a lane
constexpr uint32_t kAmaxFloorBits = (127u - 64u) << 23;  // 2^-64
constexpr uint32_t kInfBits = 0x7f800000u, kNanBits = 0x7fffffffu;

// Pages outside the cache and sequences that do not fit that were met (see indexer_guard_hits).
__device__ unsigned int g_guard_hits;

struct AppendParams {
  const void* x;
  const int32_t* starts;
  const int32_t* seq_lens;
  const int32_t* page_table;
  uint8_t* codes;
  float* scales;
  int64_t x_ts, x_hs, pt_stride;
  int64_t code_ps, code_ts, code_hs, scale_ps, scale_bs, scale_hs;
  int64_t num_pages, row_len;   // row_len: positions that the page table has
  uint32_t units, tokens;       // units: parts of blocks (see place) * heads
  Divisor block, page_blocks, heads, pieces;
  int32_t batch, dim;
};

__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// What one unit appends: `count` rows of x from `row` on, at offset `before` of a block of one page.
struct Place {
  uint32_t row, count, before;
  int64_t page;
  uint32_t page_block;  // of the page's blocks
};

// Sequence b's rows: whether they lie in x and its positions in the page table.
__device__ __forceinline__ bool sequence_at(const AppendParams& p, int b, uint32_t* start, uint32_t* count, int64_t* first) {
  const int32_t s = p.starts[b], e = p.starts[b + 1], len = p.seq_lens[b];
  *start = static_cast<uint32_t>(s);
  *count = static_cast<uint32_t>(e) - static_cast<uint32_t>(s);
  *first = static_cast<int64_t>(len) - *count;
  return s >= 0 && e >= s && static_cast<uint32_t>(e) <= p.tokens && *first >= 0 && len <= p.row_len;
}

// Sequence b has starts[b] / block + 2 b as the number of its first part: n rows touch at most n / block + 2 blocks.
__device__ __forceinline__ uint32_t first_part(const AppendParams& p, int b) {
  const int32_t s = p.starts[b];
  return quotient(p.block, static_cast<uint32_t>(max(s, 0))) + 2u * b;
}

__device__ __forceinline__ bool place(const AppendParams& p, uint32_t part, Place* at) {
  // the last sequence whose first part is not behind this one; by whole warps, each lane one place
  const int lane = threadIdx.x & 31;
  int low = 0, among = p.batch;
  while (among > 1) {
    const int step = (among + 31) / 32;
    const bool before = lane * step < among && first_part(p, low + lane * step) <= part;
    const int k = max(__popc(__ballot_sync(0xffffffffu, before)), 1) - 1;
    low += k * step;
    among = min(step, among - k * step);
  }
  uint32_t start, count;
  int64_t first;
  if (!sequence_at(p, low, &start, &count, &first) || count == 0) return false;
  const uint32_t in = part - first_part(p, low), position = static_cast<uint32_t>(first);
  const uint32_t first_block = quotient(p.block, position);
  const int64_t begin = (static_cast<int64_t>(first_block) + in) * p.block.d;  // of the block
  const int64_t from = begin > first ? begin : first, end = first + count;
  const int64_t to = begin + p.block.d < end ? begin + p.block.d : end;
  if (from >= to) return false;
  at->row = start + static_cast<uint32_t>(from - first);
  at->count = static_cast<uint32_t>(to - from);
  at->before = static_cast<uint32_t>(from - begin);
  const uint32_t block = first_block + in, entry = quotient(p.page_blocks, block);
  at->page = p.page_table[low * p.pt_stride + entry];
  at->page_block = block - entry * p.page_blocks.d;
  return true;
}

// 8 values of a lane: as they are, and the largest magnitude among them on the bit patterns, as integers, which order a
// NaN above everything.
template <typename T, bool VEC>
__device__ __forceinline__ void load_piece(const T* src, uint32_t (&bits)[kPiece * sizeof(T) / 4]) {
  if constexpr (VEC) {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(bits)) / 16; ++i) {
      const uint4 a = reinterpret_cast<const uint4*>(src)[i];
      bits[4 * i] = a.x, bits[4 * i + 1] = a.y, bits[4 * i + 2] = a.z, bits[4 * i + 3] = a.w;
    }
  } else {
    T v[kPiece];
#pragma unroll
    for (int i = 0; i < kPiece; ++i) v[i] = src[i];
    memcpy(bits, v, sizeof(v));
  }
}

template <typename T>
__device__ __forceinline__ uint32_t top_of(uint32_t top, const uint32_t (&bits)[kPiece * sizeof(T) / 4]) {
#pragma unroll
  for (int i = 0; i < static_cast<int>(sizeof(bits)) / 4; ++i) {
    if constexpr (sizeof(T) == 4) top = max(top, bits[i] & 0x7fffffffu);
    else top = __vmaxu2(top, bits[i] & 0x7fff7fffu);
  }
  return top;
}

// kJoin: warps of a unit. VEC: x's rows start on 16 bytes. kHeld: rows of a lane that stay in registers.
template <typename T, int kJoin, bool VEC>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 4 ? 2 : kJoin > 1 ? 5 : 3) append_kernel(const AppendParams p) {
  constexpr int kWords = kPiece * sizeof(T) / 4, kHeld = kJoin > 1 ? 4 : 8;
  __shared__ uint32_t tops[kWarps];
  begin_after_prior_grids();
  const uint32_t unit = kJoin == 1 ? blockIdx.x * kWarps + threadIdx.x / 32 : blockIdx.x;
  if (unit >= p.units) return;
  const int lane = threadIdx.x & 31, warp = kJoin == 1 ? 0 : threadIdx.x / 32;
  const uint32_t part = quotient(p.heads, unit), head = unit - part * p.heads.d;
  // each sequence is looked over once
  if (head == 0 && warp == 0 && part < static_cast<uint32_t>(p.batch)) {
    uint32_t start, count;
    int64_t first;
    if (!sequence_at(p, part, &start, &count, &first) && lane == 0) atomicAdd(&g_guard_hits, 1u);
  }
  Place at;
  if (!place(p, part, &at)) return;
  // a lane owns one piece of every kStep-th row
  const uint32_t rows_at_once = 32 / p.pieces.d, lane_row = quotient(p.pieces, lane);
  const bool in = lane_row < rows_at_once;
  const int col = static_cast<int>(lane - lane_row * p.pieces.d) * kPiece;
  const uint32_t first = warp * rows_at_once + lane_row, step = kJoin * rows_at_once;
  const T* src = static_cast<const T*>(p.x) + at.row * p.x_ts + head * p.x_hs + col;
  uint32_t held[kHeld][kWords], top = 0;
#pragma unroll
  for (int k = 0; k < kHeld; ++k) {
    const uint32_t r = first + k * step;
    if (in && r < at.count) {
      load_piece<T, VEC>(src + r * p.x_ts, held[k]);
    }
  }
  const bool there = at.page >= 0 && at.page < p.num_pages;
  uint8_t* code = p.codes + at.page * p.code_ps + static_cast<int64_t>(at.page_block * p.block.d) * p.code_ts +
                  head * p.code_hs + col;
  float* scale_at = p.scales + at.page * p.scale_ps + at.page_block * p.scale_bs + head * p.scale_hs;
  if (!there) {
    if (head == 0 && warp == 0 && lane == 0) atomicAdd(&g_guard_hits, 1u);
    return;
  }
  const float old = at.before > 0 ? *scale_at : 0.0f;
#pragma unroll
  for (int k = 0; k < kHeld; ++k)
    if (in && first + k * step < at.count) top = top_of<T>(top, held[k]);

  for (uint32_t r = first + kHeld * step; in && r < at.count; r += step) {
    uint32_t bits[kWords];
    load_piece<T, VEC>(src + r * p.x_ts, bits);
    top = top_of<T>(top, bits);
  }
  if constexpr (sizeof(T) == 2) {
    const unsigned short raw = static_cast<unsigned short>(max(top & 0xffffu, top >> 16));
    T v;
    memcpy(&v, &raw, 2);
    top = __float_as_uint(to_float(v));
  }
  top = __reduce_max_sync(0xffffffffu, top);
  if constexpr (kJoin > 1) {
    if (lane == 0) tops[warp] = top;
    __syncthreads();  // also: every warp has read the old scale
#pragma unroll
    for (int w = 0; w < kWarps; ++w) top = max(top, tops[w]);
  }

  // amax = m 2^e, 1 <= m < 2: 448 = 1.75 * 2^8, so 2^(e-8) while m <= 1.75, else 2^(e-7)
  const uint32_t floored = max(top, kAmaxFloorBits);
  const uint32_t e = (floored >> 23) - 8u + ((floored & 0x7fffffu) > 0x600000u ? 1u : 0u);
  uint32_t bits = top >= kInfBits ? kNanBits : e << 23;
  const uint32_t old_bits = __float_as_uint(old);
  if ((old_bits & 0x7fffffffu) > kInfBits) bits = kNanBits;
  else if (bits != kNanBits && old > __uint_as_float(bits)) bits = old_bits;
  const float scale = __uint_as_float(bits), inv = 1.0f / scale;
  const bool power = (bits & 0x7fffffu) == 0u || top >= kInfBits;  // x * inv is the quotient; or all is NaN
  if (at.before > 0 && bits != old_bits) {
    const float ratio = old / scale;
    for (uint32_t r = first; in && r < at.before; r += step) {
      uint2* const to = reinterpret_cast<uint2*>(code + r * p.code_ts);
      const uint2 was = *to;
      uint32_t now[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t w = i == 0 ? was.x : was.y;
        uint32_t y = 0;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w >> (16 * k)), __NV_E4M3);
          const float2 f = __half22float2(__half2(h));
          y |= e4m3x2(product_to_odd(f.x, ratio), product_to_odd(f.y, ratio)) << (16 * k);
        }
        now[i] = y;
      }
      *to = make_uint2(now[0], now[1]);
    }
  }
  code += at.before * p.code_ts;
  auto store = [&](uint32_t r, const uint32_t (&raw)[kWords]) {
    T typed[kPiece];
    memcpy(typed, raw, sizeof(typed));
    uint32_t c[2];
    if (power) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
        c[i] = e4m3x2(to_float(typed[4 * i]) * inv, to_float(typed[4 * i + 1]) * inv) |
               e4m3x2(to_float(typed[4 * i + 2]) * inv, to_float(typed[4 * i + 3]) * inv) << 16;
    } else {
      auto code = [&](int k) { return quotient_to_odd(to_float(typed[k]), scale, inv); };
#pragma unroll
      for (int i = 0; i < 2; ++i)
        c[i] = e4m3x2(code(4 * i), code(4 * i + 1)) | e4m3x2(code(4 * i + 2), code(4 * i + 3)) << 16;
    }
    *reinterpret_cast<uint2*>(code + r * p.code_ts) = make_uint2(c[0], c[1]);
  };
#pragma unroll
  for (int k = 0; k < kHeld; ++k) {
    const uint32_t r = first + k * step;
    if (in && r < at.count) store(r, held[k]);
  }
  for (uint32_t r = first + kHeld * step; in && r < at.count; r += step) {
    uint32_t again[kWords];
    load_piece<T, VEC>(src + r * p.x_ts, again);
    store(r, again);
  }
  __syncwarp();  // every lane has read the old scale
  if (warp == 0 && lane == 0) *scale_at = scale;
}

template <typename T, int kJoin>
cudaError_t launch_append(const AppendParams& p, bool vec, cudaStream_t stream) {
  const unsigned grid = kJoin == 1 ? (p.units + kWarps - 1) / kWarps : p.units;
  return vec ? launch(append_kernel<T, kJoin, true>, grid, kThreads, 0, stream, p)
             : launch(append_kernel<T, kJoin, false>, grid, kThreads, 0, stream, p);
}

bool aligned(const void* p, size_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

}  // namespace

cudaError_t append_guard_hits(unsigned int* hits) {
  return cudaMemcpyFromSymbol(hits, g_guard_hits, sizeof(unsigned int));
}

cudaError_t reset_append_guard_hits() {
  const unsigned int zero = 0;
  return cudaMemcpyToSymbol(g_guard_hits, &zero, sizeof(unsigned int));
}

}  // namespace indexer_gb300

extern "C" {

size_t indexer_block_cache_bytes(void) { return sizeof(indexer_block_cache_t); }

int indexer_cache_append(const void* x, int64_t x_token_stride, int64_t x_head_stride, int32_t dtype, int64_t tokens,
                         const int32_t* starts, const int32_t* seq_lens, const int32_t* page_table,
                         int64_t page_table_stride, int64_t table_pages, int32_t batch,
                         const indexer_block_cache_t* cache, cudaStream_t stream) {
  using namespace indexer_gb300;
  if (dtype < INDEXER_BF16 || dtype > INDEXER_FP32 || !block_cache_ok(cache)) return TOPK_ERR_INVALID_ARGUMENT;
  if (tokens < 0 || tokens > (INT64_C(1) << 30) || batch < 0 || batch > (1 << 28) || x_token_stride < 0 || x_head_stride < 0 ||
      table_pages < 0 || page_table_stride < 0 || (batch > 1 && page_table_stride < table_pages))
    return TOPK_ERR_INVALID_ARGUMENT;
  if (tokens == 0 || batch == 0) return TOPK_OK;
  if (x == nullptr || starts == nullptr || seq_lens == nullptr || (page_table == nullptr && table_pages > 0) ||
      !aligned(x, dtype_bytes(dtype)) || !aligned(starts, 4) || !aligned(seq_lens, 4) || !aligned(page_table, 4))
    return TOPK_ERR_INVALID_ARGUMENT;
  // the units are numbered in 31 bits
  const int64_t parts = tokens / cache->block + 2 * static_cast<int64_t>(batch);
  if (parts > INT32_MAX / cache->heads) return TOPK_ERR_INVALID_ARGUMENT;
  AppendParams p = {};
  p.x = x;
  p.starts = starts;
  p.seq_lens = seq_lens;
  p.page_table = page_table;
  p.codes = cache->codes;
  p.scales = cache->scales;
  p.x_ts = tokens > 1 ? x_token_stride : 0;
  p.x_hs = cache->heads > 1 ? x_head_stride : 0;
  p.pt_stride = batch > 1 ? page_table_stride : 0;
  p.code_ps = cache->code_page_stride;
  p.code_ts = cache->code_token_stride;
  p.code_hs = cache->code_head_stride;
  p.scale_ps = cache->scale_page_stride;
  p.scale_bs = cache->scale_block_stride;
  p.scale_hs = cache->scale_head_stride;
  p.num_pages = cache->num_pages;
  const int64_t positions = table_pages > INT32_MAX / cache->page_size ? INT32_MAX : table_pages * cache->page_size;
  p.row_len = positions;
  p.units = static_cast<uint32_t>(parts * cache->heads);
  p.tokens = static_cast<uint32_t>(tokens);
  p.block = divisor(cache->block);
  p.page_blocks = divisor(cache->page_size / cache->block);
  p.heads = divisor(cache->heads);
  p.pieces = divisor(cache->dim / kPiece);
  p.batch = batch;
  p.dim = cache->dim;
  const int64_t values = static_cast<int64_t>(16 / dtype_bytes(dtype));
  const bool vec = p.x_ts % values == 0 && p.x_hs % values == 0 && aligned(x, 16);
  // Eight warps where a block's new rows would be more than one warp holds.
  const int64_t mean = (tokens + batch - 1) / batch, rows = mean < cache->block ? mean : cache->block;
  const bool join = rows > 8 * (32 / (cache->dim / kPiece));
  cudaError_t e;
  if (dtype == INDEXER_BF16) e = join ? launch_append<__nv_bfloat16, kWarps>(p, vec, stream) : launch_append<__nv_bfloat16, 1>(p, vec, stream);
  else if (dtype == INDEXER_FP16) e = join ? launch_append<__half, kWarps>(p, vec, stream) : launch_append<__half, 1>(p, vec, stream);
  else e = join ? launch_append<float, kWarps>(p, vec, stream) : launch_append<float, 1>(p, vec, stream);
  return status_of(e);
}

}  // extern "C"
