// Shared by the kernels of attention over block-scaled caches: what a call is, how its work is shared out, small pieces
// of arithmetic.
#pragma once

#include "indexer_common.cuh"

namespace indexer_gb300 {

constexpr float kShift = 7.0f, kSlack = 8.0f;  // of weights, in powers of two: see indexer_attention.cu

// One of the two caches.
struct Side {
  const uint8_t* codes;
  const float* scales;
  int64_t code_hs, scale_hs;
  uint32_t code_ps, code_ts;    // in 16 bytes: a key's place takes one multiplication for each
  uint32_t scale_ps, scale_bs;
  Divisor block;
};

// What a span leaves to the second kernel: the tile that begins in it and goes on in the next ones, if there is one.
struct Cut {
  int64_t total;       // steps of the whole work
  int32_t slice, head, last, there;
};

struct AttendParams {
  Side side[2];              // keys, values
  const void* q;
  void* out;
  float* lse;                // may be NULL
  const int32_t* index;      // page table, or slots
  const int32_t* seq_lens;   // NULL: slots
  float* partial;
  Cut* cuts;
  int64_t index_stride, num_pages, capacity;
  Divisor page_size, group;  // group: query heads of a cache head
  int32_t lists, list_queries;  // rows of `index`, and the queries that share one
  int32_t tiles, slices;     // tiles of a list; of all lists
  int32_t kv_heads, heads, dim;
  int32_t row_len;           // positions or slots of a list
  int32_t fp16;              // q and out: fp16, else bf16
  int32_t whole_steps;       // the 16 keys of a step lie on one page
  int32_t fail;              // for tests: as if a wait of every CTA had run out (wide tiles)
  float scale;               // softmax_scale * log2(e)
};

// A step of the work and how much is left: tiles in turn, a tile's heads in turn, a head's steps.
struct Cursor {
  int64_t left;
  int32_t slice, list, head, step, steps, longest;
};

struct Spans {
  int64_t total;
  int64_t at[2];       // begin and end, in steps
  int32_t slice[2];
  int64_t rest[2];     // steps of the slice before it
};

__device__ __forceinline__ int32_t steps_of(int32_t len, int keys) { return len > keys ? (len + keys - 1) / keys : 1; }

// Keys that any query of a slice's tile of `rows` rows sees.
__device__ __forceinline__ int32_t longest_of(const AttendParams& p, int32_t slice, int rows, int first, int step) {
  if (p.seq_lens == nullptr) return p.row_len;
  const int32_t list = slice / p.tiles, r0 = (slice - list * p.tiles) * rows;
  const int32_t all = p.list_queries * static_cast<int32_t>(p.group.d);
  const int32_t n0 = quotient(p.group, r0), n1 = quotient(p.group, min(r0 + rows, all) - 1);
  int32_t longest = 0;
  for (int32_t n = n0 + first; n <= n1; n += step)
    longest = max(longest, p.seq_lens[static_cast<int64_t>(list) * p.list_queries + n]);
  return min(longest, p.row_len);
}

// This CTA's span of the work, which every CTA finds by adding up the same lengths. All threads call this; sums:
// a number for each warp.
template <int kRows, int kKeys>
__device__ __forceinline__ void find_span(const AttendParams& p, int64_t* sums, Spans& s) {
  const int64_t part = blockIdx.x, parts = gridDim.x;
  if (p.seq_lens == nullptr) {
    if (threadIdx.x < 2) {
      const int64_t each = static_cast<int64_t>(steps_of(p.row_len, kKeys)) * p.kv_heads, total = each * p.slices;
      const int e = threadIdx.x;
      s.total = total;
      s.at[e] = total * (part + e) / parts;
      s.slice[e] = static_cast<int32_t>(s.at[e] / each);
      s.rest[e] = s.at[e] - s.slice[e] * each;
    }
    __syncthreads();
    return;
  }
  const int threads = blockDim.x, lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  const int32_t per = (p.slices + threads - 1) / threads;
  const int32_t begin = min(static_cast<int32_t>(threadIdx.x) * per, p.slices), end = min(begin + per, p.slices);
  auto work_of = [&](int32_t k) {
    return static_cast<int64_t>(steps_of(longest_of(p, k, kRows, 0, 1), kKeys)) * p.kv_heads;
  };
  int64_t mine = 0;
  for (int32_t k = begin; k < end; ++k) mine += work_of(k);
  int64_t sum = mine;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const int64_t below = __shfl_up_sync(0xffffffffu, sum, d);
    if (lane >= d) sum += below;
  }
  if (lane == 31) sums[warp] = sum;
  __syncthreads();
  int64_t before = sum - mine, total = 0;
  for (int k = 0; k < threads / 32; ++k) {
    before += k < warp ? sums[k] : 0;
    total += sums[k];
  }
  if (threadIdx.x == 0) s.total = total;
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int64_t at = total * (part + e) / parts;
    if (at == total ? threadIdx.x == 0 : at >= before && at < before + mine) {
      s.at[e] = at;
      int32_t k = begin;
      int64_t rest = at - before;
      if (at == total) {
        k = p.slices, rest = 0;
      } else if (per > 1) {
        for (int64_t w = work_of(k); rest >= w; w = work_of(k)) rest -= w, ++k;
      }
      s.slice[e] = k;
      s.rest[e] = rest;
    }
  }
  __syncthreads();
}

__device__ __forceinline__ uint32_t halves_of(uint32_t two_codes) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(two_codes)));
  return r;
}

// 0x80 in each byte that is a NaN code.
__device__ __forceinline__ uint32_t nan_codes(uint32_t x) { return ((x & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u; }

__device__ __forceinline__ float exp2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

__device__ __forceinline__ float log2_fast(float x) {
  float r;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float inverse_fast(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// The larger one, NaN if either is.
__device__ __forceinline__ float max_or_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

__device__ __forceinline__ uint32_t smem_addr(const void* p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }

__device__ __forceinline__ void copy16(uint32_t to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t to, const void* from) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to), "l"(from) : "memory");
}

__device__ __forceinline__ void store_pair(void* out, int64_t at, bool fp16, float a, float b) {
  if (fp16) *reinterpret_cast<__half2*>(static_cast<__half*>(out) + at) = __floats2half2_rn(a, b);
  else *reinterpret_cast<__nv_bfloat162*>(static_cast<__nv_bfloat16*>(out) + at) = __floats2bfloat162_rn(a, b);
}

// log(sum of p) from the bound m and the sum of 2^(kShift - m) p.
__device__ __forceinline__ float log_sum(float bound, float sum) {
  const float none = __uint_as_float(0xff800000u);
  if (sum == 0.0f) return none;
  return bound == none ? sum : (bound - kShift + log2f(sum)) * 0.69314718055994530942f;
}

constexpr int kJoinRows = 8, kJoinThreads = 256;

// Joins the pieces of the tile of `rows` rows that begins in span blockIdx.x and goes on in the next ones, if there is one:
// 8 of its rows a CTA. A piece is [rows][kDim] sums, then bound and sum of weights of each row. All pieces' bounds are asked
// for at once, and a thread's part of all pieces' sums. Order: what four neighbouring values of a row's sums are the
// columns of.
template <int kDim, typename Order>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const __grid_constant__ AttendParams p, const int32_t spans, const int32_t rows) {
  extern __shared__ float2 parts[];  // [pieces][kJoinRows]; then shares in their first halves
  begin_after_prior_grids();
  const Cut cut = p.cuts[blockIdx.x];
  if (cut.there == 0) return;
  const int64_t floats = static_cast<int64_t>(rows) * (kDim + 2);
  const int32_t list = cut.slice / p.tiles, here = blockIdx.y * kJoinRows, r0 = (cut.slice - list * p.tiles) * rows + here;
  const int32_t group = static_cast<int32_t>(p.group.d), live = min(p.list_queries * group - r0, kJoinRows);
  if (live <= 0) return;
  const int32_t first = static_cast<int32_t>(blockIdx.x), pieces = cut.last - first + 1;
  const float none = __uint_as_float(0xff800000u);
  auto row_at = [&](int32_t r) {
    const int32_t n = quotient(p.group, r0 + r);
    return (static_cast<int64_t>(list) * p.list_queries + n) * p.heads + cut.head * group + (r0 + r - n * group);
  };
  auto piece_at = [&](int32_t k) { return p.partial + (2 * static_cast<int64_t>(first + k) + (k == 0 ? 1 : 0)) * floats; };
  // spans without steps have no piece: there are fewer steps than spans then, and some spans begin where they end
  const bool all = cut.total >= spans;
  for (int u = threadIdx.x; u < pieces * kJoinRows; u += kJoinThreads) {
    const int k = u / kJoinRows;
    float2 part = make_float2(none, 0.0f);
    if (all || cut.total * (first + k) / spans < cut.total * (first + k + 1) / spans)
      part = *reinterpret_cast<const float2*>(piece_at(k) + rows * kDim + 2 * (here + u % kJoinRows));
    else
      part.y = -1.0f;
    parts[u] = part;
  }
  __syncthreads();
  const int lane = threadIdx.x & 31, r = threadIdx.x / 32;  // a warp a row
  float top = none, total = 0.0f;
  for (int k = lane; k < pieces; k += 32) top = fmaxf(top, parts[k * kJoinRows + r].x);
#pragma unroll
  for (int d = 16; d > 0; d /= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
  for (int k = lane; k < pieces; k += 32) {
    float2& part = parts[k * kJoinRows + r];
    const bool any = part.y != -1.0f;  // a sum of weights is not negative
    const float f = part.x == none ? 1.0f : exp2_fast(part.x - top);
    total += any ? part.y * f : 0.0f;
    part.x = any ? f : -1.0f;  // (a share may round to 0: a NaN among its piece's sums still counts)
  }
#pragma unroll
  for (int d = 16; d > 0; d /= 2) total += __shfl_xor_sync(0xffffffffu, total, d);
  const float over = total == 0.0f ? 0.0f : 1.0f / total;
  if (p.lse != nullptr && lane == 0 && r < live) p.lse[row_at(r)] = log_sum(top, total);
  __syncwarp();
  if (r >= live) return;
  const int64_t out = row_at(r) * p.dim;
#pragma unroll
  for (int q = 0; q < (kDim + 127) / 128; ++q) {
    const int at = (q * 32 + lane) * 4;
    if (at >= kDim) break;
    float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    const float* const base = p.partial + static_cast<int64_t>(here + r) * kDim + at;
#pragma unroll 4
    for (int32_t k = 0; k < pieces; ++k) {
      const float f = parts[k * kJoinRows + r].x;
      if (f >= 0.0f) {  // else there is no piece
        const float4 v = *reinterpret_cast<const float4*>(base + (2 * static_cast<int64_t>(first + k) + (k == 0 ? 1 : 0)) * floats);
        sum[0] = fmaf(v.x, f, sum[0]), sum[1] = fmaf(v.y, f, sum[1]), sum[2] = fmaf(v.z, f, sum[2]), sum[3] = fmaf(v.w, f, sum[3]);
      }
    }
    const int a = Order::column(at), b = Order::column(at + 2);
    if (a < p.dim) store_pair(p.out, out + a, p.fp16 != 0, sum[0] * over, sum[1] * over);
    if (b < p.dim) store_pair(p.out, out + b, p.fp16 != 0, sum[2] * over, sum[3] * over);
  }
}

template <int kDim, typename Order>
cudaError_t launch_join(const AttendParams& p, int spans, int rows, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(spans - 1, (rows + kJoinRows - 1) / kJoinRows, 1);
  cfg.blockDim = dim3(kJoinThreads, 1, 1);
  cfg.dynamicSmemBytes = static_cast<size_t>(spans) * kJoinRows * 8;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, join_kernel<kDim, Order>, p, static_cast<int32_t>(spans), static_cast<int32_t>(rows));
}

// Attention of more query rows on the same keys than a warp takes, for heads of more than 64 columns (padded to 128):
// indexer_attention_wide.cu. Rows of a tile, and the call.
int wide_rows(int64_t rows);
cudaError_t launch_wide_attention(AttendParams p, int sms, cudaStream_t stream);
cudaError_t wide_attention_guard_hits(unsigned int* hits);
cudaError_t reset_wide_attention_guard_hits();

}  // namespace indexer_gb300
