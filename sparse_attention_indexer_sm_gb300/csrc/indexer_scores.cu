// The indexer's scores over a paged cache of e4m3 keys:
//   score[j] = scale_j * sum_h weight_h * max(q_h . k_j, 0)
// A thread owns a key and keeps its 128 values in registers, as pairs of halves (exact);
// the queries' heads pass by in shared memory. Products and sums are in fp32.

#include <cuda_fp8.h>

#include "indexer_common.cuh"

namespace indexer_gb300 {
namespace {

constexpr int kTile = 128;  // keys of a CTA, one for each thread
constexpr int kDim = INDEXER_SCORE_DIM;

__device__ unsigned int g_guard_hits;

struct ScoresParams {
  const uint8_t* q;
  const float* weights;
  const uint8_t* codes;
  const float* scales;
  const int32_t* page_table;
  const int32_t* seq_lens;
  float* out;
  int64_t num_pages, code_ps, code_ts, scale_ps, scale_ts, pt_stride, row_len;
  int64_t tiles;
  int32_t page_size, batch, queries, heads;
};

__device__ __forceinline__ float2 e4m3_pair(uint16_t c) {
  return __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(c, __NV_E4M3)));
}

__global__ void __launch_bounds__(kTile) scores_kernel(const ScoresParams p) {
  __shared__ __align__(16) float2 qs[INDEXER_MAX_HEADS * kDim / 2 / 4];  // a quarter of the heads at once
  __shared__ float ws[INDEXER_MAX_HEADS];
  begin_after_prior_grids();
  const int64_t rows = static_cast<int64_t>(p.batch) * p.queries;
  for (int64_t u = blockIdx.x; u < rows * p.tiles; u += gridDim.x) {
    const int64_t row = u / p.tiles, j = (u - row * p.tiles) * kTile + threadIdx.x;
    const int64_t b = row / p.queries;
    const int64_t len = max(min(static_cast<int64_t>(p.seq_lens[row]), p.row_len), int64_t(0));
    float acc = 0.0f, scale = 0.0f;
    bool live = j < len;
    uint16_t k[kDim / 2];
    if (live) {
      const int64_t page = p.page_table[b * p.pt_stride + j / p.page_size], off = j % p.page_size;
      if (page < 0 || page >= p.num_pages) {
        atomicAdd(&g_guard_hits, 1u);
        live = false;
      } else {
        const uint4* src = reinterpret_cast<const uint4*>(p.codes + page * p.code_ps + off * p.code_ts);
#pragma unroll
        for (int i = 0; i < kDim / 16; ++i) *reinterpret_cast<uint4*>(&k[8 * i]) = src[i];
        scale = p.scales[page * p.scale_ps + off * p.scale_ts];
      }
    }
    constexpr int kQuarter = INDEXER_MAX_HEADS / 4;
    for (int h0 = 0; h0 < p.heads; h0 += kQuarter) {
      const int hn = min(kQuarter, p.heads - h0);
      __syncthreads();
      const uint16_t* q = reinterpret_cast<const uint16_t*>(p.q + (row * p.heads + h0) * kDim);
      for (int i = threadIdx.x; i < hn * kDim / 2; i += kTile) qs[i] = e4m3_pair(q[i]);
      for (int i = threadIdx.x; i < hn; i += kTile) ws[i] = p.weights[row * p.heads + h0 + i];
      __syncthreads();
      if (live) {
        for (int h = 0; h < hn; ++h) {
          float dot = 0.0f;
#pragma unroll
          for (int i = 0; i < kDim / 2; ++i) {
            const float2 a = e4m3_pair(k[i]), c = qs[h * (kDim / 2) + i];
            dot = fmaf(a.x, c.x, dot);
            dot = fmaf(a.y, c.y, dot);
          }
          acc = fmaf(ws[h], fmaxf(dot, 0.0f), acc);
        }
      }
    }
    if (j < p.row_len) p.out[row * p.row_len + j] = live ? acc * scale : __int_as_float(0xff800000);
  }
}

}  // namespace

cudaError_t scores_guard_hits(unsigned int* hits) {
  return cudaMemcpyFromSymbol(hits, g_guard_hits, sizeof(unsigned int));
}

cudaError_t reset_scores_guard_hits() {
  const unsigned int zero = 0;
  return cudaMemcpyToSymbol(g_guard_hits, &zero, sizeof(unsigned int));
}

}  // namespace indexer_gb300

extern "C" int indexer_scores(const uint8_t* q, const float* weights, const indexer_cache_t* cache,
                              const int32_t* page_table, int64_t page_table_stride,
                              const int32_t* seq_lens, int32_t batch, int32_t queries, int32_t heads,
                              int64_t row_len, float* out, cudaStream_t stream) {
  using namespace indexer_gb300;
  if (!cache_ok(cache) || cache->dim != INDEXER_SCORE_DIM) return TOPK_ERR_INVALID_ARGUMENT;
  if (batch < 0 || queries < 0 || heads < 1 || heads > INDEXER_MAX_HEADS || row_len < 1 ||
      row_len > INT32_MAX || static_cast<int64_t>(batch) * queries > INT32_MAX)
    return TOPK_ERR_INVALID_ARGUMENT;
  if (batch == 0 || queries == 0) return TOPK_OK;
  if (q == nullptr || weights == nullptr || page_table == nullptr || seq_lens == nullptr || out == nullptr)
    return TOPK_ERR_INVALID_ARGUMENT;
  const int64_t pages = (row_len + cache->page_size - 1) / cache->page_size;
  if (page_table_stride < (batch > 1 ? pages : 1)) return TOPK_ERR_INVALID_ARGUMENT;
  const uintptr_t low = reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(cache->codes) |
                        static_cast<uintptr_t>(cache->page_size > 1 ? cache->code_token_stride : 0) |
                        static_cast<uintptr_t>(cache->num_pages > 1 ? cache->code_page_stride : 0);
  const uintptr_t low4 = reinterpret_cast<uintptr_t>(weights) | reinterpret_cast<uintptr_t>(page_table) |
                         reinterpret_cast<uintptr_t>(seq_lens) | reinterpret_cast<uintptr_t>(out);
  if ((low & 15u) != 0 || (low4 & 3u) != 0) return TOPK_ERR_INVALID_ARGUMENT;
  int sms = 0;
  cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return status_of(e);
  ScoresParams p = {};
  p.q = q;
  p.weights = weights;
  p.codes = cache->codes;
  p.scales = cache->scales;
  p.page_table = page_table;
  p.seq_lens = seq_lens;
  p.out = out;
  p.num_pages = cache->num_pages;
  p.code_ps = cache->code_page_stride;
  p.code_ts = cache->code_token_stride;
  p.scale_ps = cache->scale_page_stride;
  p.scale_ts = cache->scale_token_stride;
  p.pt_stride = page_table_stride;
  p.row_len = row_len;
  p.tiles = (row_len + kTile - 1) / kTile;
  p.page_size = cache->page_size;
  p.batch = batch;
  p.queries = queries;
  p.heads = heads;
  const int64_t units = static_cast<int64_t>(batch) * queries * p.tiles, most = int64_t(sms) * 8;
  e = launch(scores_kernel, static_cast<unsigned>(units < most ? units : most), kTile, 0, stream, p);
  return status_of(e);
}
